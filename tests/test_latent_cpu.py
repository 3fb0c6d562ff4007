"""Latent attention without a GPU: what the library and the owners refuse before anything is
enqueued, and the 8-bit reference."""
import math

import pytest
import torch

import latent_reference as lref
from expert_slot_cache_device_gb300 import ftmoe as F
from expert_slot_cache_device_gb300.latent_cache import ExpandedBatch, LatentCache, row_bytes
from test_attention_cpu import A, BAD_BATCH, R, _lib, batch, refused, rows  # noqa: F401


def cache(**kw):
    d = dict(d_pages=A, page_stride=16 * 1152, slot_stride=1152, dtype=F.DT_BF16, bits=16, num_pages=4, page_size=16, latent=512, rope=64,
             d_status=None)
    d.update(kw)
    return F.LatentCacheView(**d)


BAD_CACHE = [dict(d_pages=None), dict(d_pages=A + 8), dict(page_size=8), dict(page_size=48), dict(page_size=512), dict(num_pages=0),
             dict(slot_stride=1136), dict(slot_stride=1160), dict(page_stride=0), dict(page_stride=24), dict(page_stride=-16)]
BAD_FORMAT = [dict(dtype=F.DT_F32), dict(bits=4), dict(bits=0), dict(latent=0), dict(latent=64), dict(latent=576), dict(latent=192), dict(rope=0),
              dict(rope=24), dict(rope=80)]


def test_append_refusals():
    def call(c=None, b=None, rot=None, lat=A, ls=512, key=A, ks=64, w=A, eps=1e-6, q=None, qo=None, heads=4, pos=A):
        F.ftmoe_latent_append(R(c or cache()), R(b or batch()), R(rot or F.RotaryView(A, 64, 0, 1.0)), lat, ls, key, ks, w, eps,
                              R(q or rows()), R(qo or rows()), heads, pos, 0)

    for bad in BAD_CACHE:
        refused(F.ERR_INVALID_ARG, call, cache(**bad))
    for bad in BAD_FORMAT:
        refused(F.ERR_FORMAT, call, cache(**bad))
    for bad in BAD_BATCH:
        refused(F.ERR_INVALID_ARG, call, cache(), batch(**bad))
    for kw in (dict(rot=F.RotaryView(A, 32, 0, 1.0)), dict(rot=F.RotaryView(None, 64, 0, 1.0)), dict(rot=F.RotaryView(A + 4, 64, 0, 1.0)),
               dict(rot=F.RotaryView(A, 64, 0, math.nan)), dict(lat=None), dict(lat=A + 8), dict(ls=508), dict(ls=504), dict(key=None),
               dict(key=A + 2), dict(ks=60), dict(ks=56), dict(w=A + 4), dict(eps=-1.0), dict(eps=math.nan), dict(eps=math.inf),
               dict(heads=-1), dict(heads=65536), dict(q=rows(d=A + 4)), dict(qo=rows(token=12)), dict(qo=rows(token=512)),
               dict(q=rows(head=32)), dict(pos=None)):
        refused(F.ERR_INVALID_ARG, lambda: call(**kw))
    call(b=batch(tokens=0))
    call(b=batch(batch=0))
    with pytest.raises(F.FtmoeError):
        F.ftmoe_latent_append(None, R(batch()), R(F.RotaryView(A, 64, 0, 1.0)), A, 512, A, 64, A, 0.0, None, None, 0, A, 0)


def test_read_refusals():
    def call(c=None, b=None, cu=A, n=64, out=A, stride=576):
        F.ftmoe_latent_read(R(c or cache()), R(b or batch()), cu, n, out, stride, 0)

    for bad in BAD_CACHE:
        refused(F.ERR_INVALID_ARG, call, cache(**bad))
    for bad in BAD_FORMAT:
        refused(F.ERR_FORMAT, call, cache(**bad))
    for bad in BAD_BATCH:
        refused(F.ERR_INVALID_ARG, call, cache(), batch(**bad))
    for kw in (dict(cu=None), dict(n=-1), dict(out=None), dict(out=A + 8), dict(stride=568), dict(stride=580)):
        refused(F.ERR_INVALID_ARG, lambda: call(**kw))
    call(n=0)
    call(b=batch(batch=0))
    call(b=batch(max_kv=0))


def test_attend_refusals():
    wide = rows(token=4 * 576, head=576)

    def call(c=None, b=None, q=wide, qr=wide, heads=4, scale=0.1, out=wide, ws=None, nb=0):
        F.ftmoe_latent_attention(R(c or cache()), R(b or batch()), R(q), R(qr), heads, scale, True, R(out), None, ws, nb, 0)

    for bad in BAD_CACHE:
        refused(F.ERR_INVALID_ARG, call, cache(**bad))
    for bad in BAD_FORMAT:
        refused(F.ERR_FORMAT, call, cache(**bad))
    for bad in BAD_BATCH:
        refused(F.ERR_INVALID_ARG, call, cache(), batch(**bad))
    for kw in (dict(heads=0), dict(heads=-3), dict(heads=65536), dict(scale=0.0), dict(scale=-1.0), dict(scale=math.nan), dict(scale=math.inf),
               dict(q=rows(token=4 * 576, head=504)), dict(q=rows(d=None)), dict(qr=rows(head=56)), dict(out=rows(d=A + 8)),
               dict(out=rows(token=8 * 576, head=576)), dict(b=batch(tokens=1 << 20), heads=2048)):
        refused(F.ERR_INVALID_ARG, lambda: call(**kw))
    call(b=batch(tokens=0))
    call(b=batch(batch=0))
    call(b=batch(max_q=0))
    with pytest.raises(F.FtmoeError):
        F.ftmoe_latent_attention_workspace_bytes(None, R(batch()), 4, True)


def row_batch(**kw):
    d = dict(d_cu_q=A, d_cu_kv=A, batch=2, tokens=4, rows=64, max_q=2, max_kv=32, d_status=None)
    d.update(kw)
    return F.RowBatchView(**d)


def test_expanded_refusals():
    wide = rows(token=4 * 192, head=192)

    def call(b=None, dt=F.DT_BF16, heads=4, nope=128, rope=64, vd=128, q=wide, k=wide, key=A, ks=64, v=wide, scale=0.1, out=wide):
        F.ftmoe_expanded_attention(R(b or row_batch()), dt, heads, nope, rope, vd, R(q), R(k), key, ks, R(v), scale, True, R(out), None, None, 0, 0)

    for kw in (dict(d_cu_q=None), dict(d_cu_kv=None), dict(batch=-1), dict(batch=65536), dict(tokens=-1), dict(rows=-1), dict(max_q=-1),
               dict(max_kv=-1), dict(max_kv=(1 << 30) + 1)):
        refused(F.ERR_INVALID_ARG, lambda: call(row_batch(**kw)))
    for kw in (dict(dt=F.DT_F32), dict(nope=96), dict(nope=64), dict(vd=64), dict(nope=0, vd=0), dict(rope=0), dict(rope=8), dict(rope=72)):
        refused(F.ERR_FORMAT, lambda: call(**kw))
    for kw in (dict(heads=0), dict(heads=65536), dict(scale=0.0), dict(scale=math.inf), dict(q=rows(head=128)), dict(k=rows(head=64)), dict(v=rows(d=A + 4)),
               dict(out=rows(d=None)), dict(key=None), dict(key=A + 2), dict(ks=56), dict(ks=68)):
        refused(F.ERR_INVALID_ARG, lambda: call(**kw))
    call(row_batch(tokens=0))
    call(row_batch(batch=0))
    call(row_batch(max_q=0))


def test_owners_refuse():
    for kw in (dict(latent=500), dict(latent=640), dict(rope=8), dict(rope=128), dict(bits=4), dict(dtype=torch.float32)):
        with pytest.raises(ValueError):
            LatentCache(**dict(dict(num_pages=2, page_size=16, latent=512, rope=64, device="cpu"), **kw))
    with pytest.raises(ValueError):  # pages on the host
        LatentCache(2, 16, 512, 64, pages=torch.zeros((2, 16, 576), dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        ExpandedBatch(torch.zeros(3, dtype=torch.int32), torch.zeros(3, dtype=torch.int32), 1, 1)
    for latent, rope in ((128, 16), (256, 32), (384, 64), (512, 64)):
        for bits in (16, 8):
            assert row_bytes(latent, rope, bits) == lref.row_bytes(latent, rope, bits)
            assert row_bytes(latent, rope, bits) % 16 == 0


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
def test_reference_of_8_bits(dt):
    """The reference against torch's e4m3 type, and its round trip."""
    g = torch.Generator().manual_seed(5)
    y = (torch.randn((64, 128), generator=g) * torch.exp2(torch.randint(-20, 14, (64, 1), generator=g).float())).to(dt)
    y[0], y[1, :32] = 0, 448.0
    codes, powers, _ = lref.encode(y)
    x = y.double().clamp(-61440, 61440) if dt == torch.float16 else y.double()
    want = (x.view(64, 4, 32) / torch.exp2(powers.double() - 127)[..., None]).float().to(torch.float8_e4m3fn)
    assert torch.equal(codes, want.view(torch.uint8).view(64, 128))
    back = lref.decode(codes, powers, dt)
    top = x.view(64, 4, 32).abs().amax(2).repeat_interleave(32, 1)
    assert ((back - x).abs() <= 2.0 ** -4 * x.abs() + top * 2.0 ** -17 + 2.0 ** -25).all() and torch.isfinite(back).all()
    assert (powers[0] == 0).all() and powers[1, 0] == 127
