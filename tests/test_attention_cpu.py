"""The attention half without a GPU: what the library and the owners refuse before anything is
enqueued, and the rotary frequencies."""
import ctypes
import math

import pytest
import torch

from expert_slot_cache_device_gb300 import build as B
from expert_slot_cache_device_gb300 import ftmoe as F
from expert_slot_cache_device_gb300.kv_cache import KVBatch, PagedKVCache, Rotary, rotary_frequencies
from expert_slot_cache_device_gb300.w4 import W4Weights


@pytest.fixture(scope="module", autouse=True)
def _lib():
    B.build()
    F.lib()


A = 1 << 20  # an aligned address; nothing is launched


def cache(**kw):
    d = dict(d_k=A, d_v=A, k_page=16 * 2 * 64, k_slot=2 * 64, k_head=64, v_page=16 * 2 * 64, v_slot=2 * 64, v_head=64,
             dtype=F.DT_BF16, num_pages=4, page_size=16, kv_heads=2, head_dim=64, d_status=None)
    d.update(kw)
    return F.KVCacheView(**d)


def batch(**kw):
    d = dict(d_block_table=A, table_stride=4, d_kv_lens=A, d_cu_q=A, batch=2, tokens=2, max_q=1, max_kv=64, max_pages=4)
    d.update(kw)
    return F.KVBatchView(**d)


def rows(**kw):
    d = dict(d=A, token=256, head=64)
    d.update(kw)
    return F.RowsView(**d)


R = ctypes.byref


def refused(code, call, *args):
    with pytest.raises(F.FtmoeError) as e:
        call(*args)
    assert e.value.code == code
    assert str(e.value)


BAD_CACHE = [dict(d_k=None), dict(d_v=A + 2), dict(page_size=8), dict(page_size=48), dict(page_size=512), dict(num_pages=0),
             dict(kv_heads=0), dict(head_dim=72), dict(head_dim=272), dict(k_slot=0), dict(v_head=65), dict(k_page=-8)]
BAD_BATCH = [dict(d_block_table=None), dict(d_kv_lens=None), dict(d_cu_q=None), dict(batch=-1), dict(tokens=-1), dict(max_q=-1),
             dict(max_kv=65), dict(max_kv=-1), dict(table_stride=3), dict(batch=65536)]


def attend(c, b, q=None, heads=4, scale=0.1, window=0, causal=True, out=None, mass=None, mh=64, ws=None, nb=0):
    F.ftmoe_paged_attention(R(c), R(b), R(q or rows()), heads, scale, window, causal, None, R(out or rows()), None, mass, 128,
                            mh, ws, nb, 0)


def test_attention_refusals():
    for bad in BAD_CACHE:
        refused(F.ERR_INVALID_ARG, attend, cache(**bad), batch())
    for bad in BAD_BATCH:
        refused(F.ERR_INVALID_ARG, attend, cache(), batch(**bad))
    refused(F.ERR_FORMAT, attend, cache(dtype=F.DT_F32), batch())
    refused(F.ERR_FORMAT, attend, cache(head_dim=96), batch())
    refused(F.ERR_FORMAT, lambda: attend(cache(), batch(), heads=2 * 129))
    for kw in (dict(heads=3), dict(heads=0), dict(scale=0.0), dict(scale=-1.0), dict(scale=math.nan), dict(scale=math.inf),
               dict(window=-1), dict(window=4, causal=False), dict(q=rows(d=A + 8)), dict(q=rows(token=100)),
               dict(out=rows(head=8)), dict(out=rows(d=None)), dict(mass=A, mh=63)):
        refused(F.ERR_INVALID_ARG, lambda: attend(cache(), batch(), **kw))
    with pytest.raises(F.FtmoeError):
        F.ftmoe_paged_attention(None, R(batch()), R(rows()), 4, 0.1, 0, True, None, R(rows()), None, None, 0, 0, None, 0, 0)
    # nothing to do is not an error, and needs no device
    attend(cache(), batch(tokens=0))
    attend(cache(), batch(batch=0))
    attend(cache(), batch(max_q=0))


def test_append_refusals():
    def call(c=None, b=None, rot=None, q=None, qo=None, heads=4, k=None, v=None, pos=A):
        F.ftmoe_rope_append(R(c or cache()), R(b or batch()), R(rot or F.RotaryView(A, 64, 0, 1.0)), R(q or rows()),
                            R(qo or rows()), heads, R(k or rows()), R(v or rows()), pos, 0)

    for bad in BAD_CACHE:
        refused(F.ERR_INVALID_ARG, call, cache(**bad))
    for bad in BAD_BATCH:
        refused(F.ERR_INVALID_ARG, call, cache(), batch(**bad))
    for kw in (dict(rot=F.RotaryView(A, 24, 0, 1.0)), dict(rot=F.RotaryView(A, 80, 0, 1.0)), dict(rot=F.RotaryView(None, 64, 0, 1.0)),
               dict(rot=F.RotaryView(A + 4, 64, 0, 1.0)), dict(rot=F.RotaryView(A, 64, 0, math.nan)), dict(heads=-1),
               dict(q=rows(d=A + 4)), dict(qo=rows(token=12)), dict(k=rows(head=4)), dict(k=rows(head=32)), dict(v=rows(d=None)),
               dict(pos=None)):
        refused(F.ERR_INVALID_ARG, lambda: call(**kw))
    call(b=batch(tokens=0))


def test_evict_refusals():
    def call(c=None, b=None, mass=A, mh=64, budget=32, recent=4, table=A, stride=2, kept=A, nm=A, nl=A):
        F.ftmoe_kv_evict(R(c or cache()), R(b or batch()), mass, 128, mh, budget, recent, table, stride, kept, nm, nl, 0)

    for bad in BAD_CACHE:
        refused(F.ERR_INVALID_ARG, call, cache(**bad))
    for kw in (dict(mass=None), dict(mh=63), dict(budget=0), dict(recent=-1), dict(recent=33), dict(table=None), dict(stride=1),
               dict(kept=None), dict(nm=None), dict(nl=None)):
        refused(F.ERR_INVALID_ARG, lambda: call(**kw))
    call(b=batch(batch=0))


def test_w4_refusals():
    for n, k, g, code in ((0, 128, 128, -1), (16, 0, 64, -1), (16, 96, 64, -1), (16, 128, 16, -5), (16, 256, 256, -5)):
        refused(code, F.ftmoe_w4_packed_bytes, n, k, g, False)
    assert F.ftmoe_w4_packed_bytes(17, 96, 32, True) == 2 * 2 * 512 + 2 * 4 * 48
    nb = F.ftmoe_w4_packed_bytes(16, 128, 64, False)
    refused(F.ERR_INVALID_ARG, F.ftmoe_w4_pack, A, A, None, 16, 128, 64, A, nb - 1, 0)
    refused(F.ERR_INVALID_ARG, F.ftmoe_w4_pack, A, A, None, 16, 128, 64, A + 16, nb, 0)
    refused(F.ERR_INVALID_ARG, F.ftmoe_w4_pack, None, A, None, 16, 128, 64, A, nb, 0)
    ok = [A, 16, 128, 64, False, F.DT_BF16, A, 128, 3, A, 16, 0]
    for at, value, code in ((0, None, -1), (0, A + 128, -1), (5, F.DT_F32, -5), (6, A + 2, -1), (7, 120, -1), (7, 132, -1), (8, -1, -1),
                            (9, None, -1), (10, 15, -1)):
        args = list(ok)
        args[at] = value
        refused(code, F.ftmoe_w4_matvec, *args)
    ok[8] = 0
    F.ftmoe_w4_matvec(*ok)  # no tokens: nothing to do


def test_owners_refuse_host_tensors_and_wrong_shapes():
    t = torch.zeros((2, 4), dtype=torch.int32)
    for args in ((t, t[:, 0], torch.zeros(3, dtype=torch.int32)), (t.float(), t[:, 0], t[0])):
        with pytest.raises(ValueError):
            KVBatch(*args, max_q=1, max_kv=1)
    with pytest.raises(ValueError):
        PagedKVCache(4, 16, 2, 64, torch.float32)
    with pytest.raises(ValueError):
        PagedKVCache(4, 16, 2, 64, k_pages=torch.zeros((4, 16, 2, 64), dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        W4Weights(torch.zeros((4, 64), dtype=torch.uint8), torch.zeros((4, 1)))
    for kw in (dict(rot_dim=24), dict(rot_dim=80), dict(rot_dim=0), dict(layout="pairs"), dict(base=1.0),
               dict(scaling=dict(kind="other", factor=2.0)), dict(scaling=dict(kind="linear")),
               dict(scaling=dict(kind="linear", factor=0.0)), dict(scaling=dict(kind="yarn", factor=2.0)),
               dict(scaling=dict(kind="linear", factor=2.0, low=1)),
               dict(scaling=dict(kind="banded", factor=2.0, original=100, low=4, high=4))):
        with pytest.raises(ValueError):
            Rotary(64, device="cpu", **kw)


def test_rotary_frequencies():
    f, m = rotary_frequencies(64)
    for i in (0, 7, 31):
        assert float(f[i]) == pytest.approx(10000.0 ** (-2 * i / 64), rel=1e-14)
    assert m == 1.0
    assert torch.equal(rotary_frequencies(64, scaling=dict(kind="linear", factor=4.0))[0], f / 4)
    # a changed base leaves the fastest pair and divides the slowest by the factor
    g, _ = rotary_frequencies(64, scaling=dict(kind="base", factor=4.0))
    assert float(g[0]) == 1.0 and float(g[31] * 4 / f[31]) == pytest.approx(1.0, rel=1e-12)
    y, m = rotary_frequencies(128, 1e6, dict(kind="yarn", factor=8.0, original=4096))
    f, _ = rotary_frequencies(128, 1e6)
    turns = 4096 * f / (2 * math.pi)
    assert torch.equal(y[turns > 40], f[turns > 40]) and torch.allclose(y[turns < 0.8], f[turns < 0.8] / 8, rtol=1e-14)
    assert ((y <= f) & (y >= f / 8 * (1 - 1e-14))).all() and m == pytest.approx(0.1 * math.log(8) + 1)
    assert rotary_frequencies(128, scaling=dict(kind="yarn", factor=8.0, original=4096, attention_factor=1.5))[1] == 1.5
    b, m = rotary_frequencies(128, 5e5, dict(kind="banded", factor=8.0, original=8192))
    f, _ = rotary_frequencies(128, 5e5)
    r = 8192 * f / (2 * math.pi)
    assert torch.allclose(b[r > 4], f[r > 4], rtol=1e-14) and torch.allclose(b[r < 1], f[r < 1] / 8, rtol=1e-14)
    mid = (r > 1) & (r < 4)
    a = (r[mid] - 1) / 3
    assert mid.any() and torch.allclose(b[mid], (1 - a) * f[mid] / 8 + a * f[mid], rtol=1e-12) and m == 1.0
    plan = Rotary(128, 64, scaling=dict(kind="linear", factor=3.0), device="cpu")
    both = plan.freq.double().sum(-1) * 2 * math.pi
    want = rotary_frequencies(64, scaling=dict(kind="linear", factor=3.0))[0]
    assert torch.allclose(both, want, rtol=2.0 ** -45)
