"""Latent attention: calls that the contract allows and the other tests do not make. Tolerances as in tests/latent_reference.py."""
import math

import pytest
import torch

import attention_reference as ref
import latent_reference as lref
from test_gpu_latent import BF, HF, World, check_attend, check_rows, expand_world, ints, starts

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
