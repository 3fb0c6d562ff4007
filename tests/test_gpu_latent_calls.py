"""Latent attention: calls that the contract allows and the other tests do not make. Tolerances as in tests/latent_reference.py."""
import math

import pytest
import torch

import attention_reference as ref
import latent_reference as lref
from test_gpu_latent import BF, HF, World, check_rows, expand_world, ints, starts

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from expert_slot_cache_device_gb300 import build

    build.build()


def test_expanded_bounds_of_any_size():
    """Bounds that a constructor takes serve every call: they are cut to the tokens and rows there are."""
    from expert_slot_cache_device_gb300.latent_cache import ExpandedBatch

    _, q, k, key, v, cu_q, cu_kv = expand_world([30, 200], [500, 200], 2, 64, 32, BF)
    for most in (2 ** 30 + 1, 2 ** 31 - 1):
        b = ExpandedBatch(ints(cu_q), ints(cu_kv), most, most)
        lse = torch.zeros((q.shape[0], 2), device="cuda")
        out = b.attend(q, k, key, v, lse=lse)
        assert b.status() == 0
        for i in range(2):
            t, r = slice(cu_q[i], cu_q[i + 1]), slice(cu_kv[i], cu_kv[i + 1])
            o, z, ot, zt = lref.expanded(q[t].cpu(), k[r].cpu(), key[r].cpu(), v[r].cpu(), 96 ** -0.5, True)
            check_rows(i, out[t], o, ot, lse[t], z, zt)


@pytest.mark.parametrize("owner", ["latent", "paged"])
def test_a_token_that_two_sequences_claim_goes_to_one_of_them(owner):
    """Offsets that fall back are recorded; a token that lies in two ranges then is written to its slot of one of the two
    sequences, not to a slot of one through the other's pages."""
    from expert_slot_cache_device_gb300 import ftmoe as F
    from expert_slot_cache_device_gb300.kv_cache import KVBatch, PagedKVCache, Rotary
    from expert_slot_cache_device_gb300.latent_cache import LatentCache

    n, ahead, page, last = 4096, 512, 16, 40
    own, wide = n // page, (n + ahead) // page
    table = torch.full((last + 1, wide), -1, dtype=torch.int32)
    table[0] = torch.arange(wide)  # the last pages are not sequence 0's by its length
    table[last] = torch.arange(wide, 2 * wide)
    lens = [n] + [0] * (last - 1) + [n + ahead]
    batch = KVBatch(table.cuda(), ints(lens), ints([0] + [n] * (last - 1) + [0, n]), n, n + ahead)
    g = torch.Generator().manual_seed(3)
    pos = torch.zeros(n, dtype=torch.int32, device="cuda")
    if owner == "latent":
        cache = LatentCache(2 * wide, page, 128, 16, BF)
        cache.pages.fill_(7.0)
        x = torch.randn((n, 128), generator=g).to(BF)
        cache.append(batch, Rotary(16), x.cuda(), torch.zeros((n, 16), dtype=BF, device="cuda"), pos)
        got = cache.pages[..., :128]
    else:
        cache = PagedKVCache(2 * wide, page, 1, 64, BF)
        cache.v_pages.fill_(7.0)
        x = torch.randn((n, 64), generator=g).to(BF)
        cache.append(batch, Rotary(64), None, torch.zeros((n, 1, 64), dtype=BF, device="cuda"), x[:, None].cuda(), pos)
        got = cache.v_pages[:, :, 0]
    assert cache.status() == F.ERR_STATE
    got = got.cpu().flatten(0, 1)
    first, second = got[:n + ahead], got[n + ahead:]
    assert (first[n:] == 7).all() and (second[:ahead] == 7).all()
    mine = torch.stack([(a == x).all(1) for a in (first[:n], second[ahead:])])
    none = torch.stack([(a == 7).all(1) for a in (first[:n], second[ahead:])])
    assert ((mine[0] & none[1]) | (none[0] & mine[1])).all()
