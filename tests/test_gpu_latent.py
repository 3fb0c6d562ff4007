"""Latent attention on the GPU against plain implementations in 64 bits: the write to the cache in 16
and 8 bits, its reading back, absorbed and expanded attention with their log-sum-exps.
Tolerances are what the stated roundings may move a result by (tests/latent_reference.py)."""
import math

import pytest
import torch

import attention_reference as ref
import latent_reference as lref

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]
BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _built():
    from expert_slot_cache_device_gb300 import build

    build.build()


def ints(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


def starts(lens):
    return [sum(lens[:i]) for i in range(len(lens) + 1)]


class World:
    """A latent cache full of tokens, a batch with random pages, and the plain values."""

    def __init__(self, q_lens, kv_lens, latent=512, rope=64, page=16, dtype=BF, bits=16, seed=0, gap=0, slack=0):
        from expert_slot_cache_device_gb300.kv_cache import KVBatch
        from expert_slot_cache_device_gb300.latent_cache import LatentCache

        g = self.gen = torch.Generator().manual_seed(seed)
        self.q_lens, self.kv_lens, self.page, self.latent, self.rope, self.dtype, self.bits = q_lens, kv_lens, page, latent, rope, dtype, bits
        need = [-(-n // page) for n in kv_lens]
        pages = sum(need) + 2
        perm = torch.randperm(pages, generator=g)
        self.table = torch.full((len(kv_lens), max(need + [1]) + 1), -(1 << 30), dtype=torch.int32)  # entries that no call needs are junk
        row = lref.row_bytes(latent, rope, bits)
        raw = torch.full((pages, page, row + gap), 255, dtype=torch.uint8)  # slots never written: NaN in every type
        self.c, self.key, self.stored = [], [], []
        at = 0
        for i, (n, m) in enumerate(zip(kv_lens, need)):
            self.table[i, :m] = perm[at:at + m].to(torch.int32)
            at += m
            c, key = torch.randn((n, latent), generator=g).to(dtype), torch.randn((n, rope), generator=g).to(dtype)
            if bits == 8 and n:
                codes, powers, _ = lref.encode(c)
                c, rows = lref.decode(codes, powers, dtype).to(dtype), lref.pack(codes, powers, key)
            else:
                rows = torch.cat([c, key], 1).view(torch.uint8) if n else torch.zeros((0, row), dtype=torch.uint8)
            p, r = ref.cells(self.table[i], page, n)
            raw[p, r, :row] = rows
            self.c.append(c)
            self.key.append(key)
            self.stored.append(rows)
        self.raw = raw.cuda()
        view = self.raw[..., :row] if bits == 8 else self.raw.view(dtype)[..., :latent + rope]
        self.cache = LatentCache(pages, page, latent, rope, dtype, bits, pages=view)
        self.cu = starts(q_lens)
        self.tokens = self.cu[-1] + slack
        self.batch = KVBatch(self.table.cuda(), ints(kv_lens), ints(self.cu), max_q=max(q_lens), max_kv=max(kv_lens))

    def cells(self, i):
        """Bytes of sequence i's slots as they are on the device."""
        p, r = ref.cells(self.table[i], self.page, self.kv_lens[i])
        return self.raw.cpu()[p, r]

    def queries(self, heads):
        """Slices of a wider projection."""
        wide = torch.randn((self.tokens, heads + 1, self.latent + 2 * self.rope), generator=self.gen).to(self.dtype).cuda()
        return wide[:, 1:, :self.latent], wide[:, 1:, self.latent + self.rope:]


# ---------------------------------------------------------------- write and reading back
STORE = [
    # q_lens, kv_lens, heads, latent, rope, page, dtype, bits, layout
    ([1], [1], 1, 512, 64, 16, BF, 16, "interleaved"),
    ([1, 1, 1], [5, 64, 33], 16, 512, 64, 64, BF, 8, "half"),
    ([3, 0, 40], [3, 7, 41], 0, 256, 32, 16, HF, 16, "half"),
    ([17, 2], [60, 300], 5, 128, 16, 32, HF, 8, "interleaved"),
    ([90], [1000], 128, 384, 48, 128, BF, 8, "interleaved"),
    ([130, 1, 64], [130, 1, 500], 3, 512, 64, 256, HF, 8, "half"),
    ([9, 4], [6, 4], 2, 256, 64, 16, BF, 16, "interleaved"),  # more new tokens than slots: the first have none
]


def store(w, heads, layout, weight, scaling=None, c=None, inplace=False):
    from expert_slot_cache_device_gb300.kv_cache import Rotary, rotary_frequencies

    rotary = Rotary(w.rope, layout=layout, scaling=scaling)
    n = w.tokens
    down = (torch.randn((n, w.latent + w.rope + 8), generator=w.gen) * 3).to(w.dtype)
    if c is not None:
        down[:, :w.latent] = c
    down = down.cuda()
    c, key = down[:, :w.latent], down[:, w.latent:w.latent + w.rope]
    pos = torch.randint(0, 1 << 20, (n,), generator=w.gen).to(torch.int32).cuda()
    q = torch.randn((n, max(heads, 1), 2 * w.rope), generator=w.gen).to(w.dtype).cuda()[:, :heads, w.rope:]
    q0 = q.clone()
    out = (q if inplace else torch.full((n, heads, w.rope), 7.0, dtype=w.dtype, device="cuda")) if heads else None
    got = w.cache.append(w.batch, rotary, c, key, pos, weight=weight, eps=1e-5, q_rope=q if heads else None, q_out=out)
    torch.cuda.synchronize()
    return c.cpu(), key.cpu(), pos.cpu(), q0.cpu(), got, rotary_frequencies(w.rope, scaling=scaling)


def check_turned(got, x, pos, freq, factor, layout):
    """As the rotary test of the paged cache: one rounding, and fp32 angles and products."""
    dt, rot = x.dtype, x.shape[-1]
    want = ref.rotate(x, pos, freq, factor, rot, layout)
    pair = x.double().abs().amax(-1, keepdim=True)
    tol = ref.U[dt] * want.abs() + factor * pair * 2.0 ** -19 + 2.0 ** -25
    assert ((got.double().cpu() - want).abs() <= tol).all()


@pytest.mark.parametrize("q_lens,kv_lens,heads,latent,rope,page,dt,bits,layout", STORE)
@pytest.mark.parametrize("gap", [0, 48])
def test_append(q_lens, kv_lens, heads, latent, rope, page, dt, bits, layout, gap):
    scaling = dict(kind="yarn", factor=8.0, original=4096) if gap else None
    w = World(q_lens, kv_lens, latent, rope, page, dt, bits, seed=heads, gap=gap, slack=2)
    weight = (torch.rand(latent, generator=w.gen) + 0.5).to(dt)
    before = [w.cells(i) for i in range(len(kv_lens))]
    c, key, pos, q, got, (freq, factor) = store(w, heads, layout, weight.cuda(), scaling)
    assert w.cache.status() == 0
    row = lref.row_bytes(latent, rope, bits)
    y, tol = lref.norm(c, weight, 1e-5)
    for i, (m, n) in enumerate(zip(q_lens, kv_lens)):
        have = w.cells(i)
        a = max(n - m, 0)
        assert torch.equal(have[:a], before[i][:a]) and torch.equal(have[:, row:], before[i][:, row:])
        if n == a:
            continue
        t = slice(w.cu[i] + m - (n - a), w.cu[i] + m)
        new = have[a:, :row].contiguous()
        check_turned(new[:, row - 2 * rope:].contiguous().view(dt)[:, None], key[t][:, None], pos[t], freq, factor, layout)
        if bits == 16:
            d = (new[:, :2 * latent].contiguous().view(dt).double() - y[t]).abs()
            assert (d <= tol[t]).all(), float((d / tol[t]).max())
        else:  # a power of two that one step of the rounding to 16 bits may move, and half a step of the codes
            v = lref.decode(new[:, :latent], new[:, latent:latent + latent // 32], dt)
            top = y[t].view(n - a, -1, 32).abs().amax(2).repeat_interleave(32, 1)
            assert ((v - y[t]).abs() <= 2.0 ** -4 * (y[t].abs() + tol[t]) + tol[t] + top * 2.0 ** -16).all()
    if heads:
        check_turned(got[:w.cu[-1]], q[:w.cu[-1]], pos[:w.cu[-1]], freq, factor, layout)
        assert (got[w.cu[-1]:] == 7).all()  # rows behind the last sequence
    for i in range(w.raw.shape[0]):  # pages that no sequence has
        if i not in set(w.table.flatten().tolist()):
            assert (w.raw[i] == 255).all()


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("latent", [128, 512])
def test_codes_are_those_of_the_definition(dt, latent):
    """Without a norm the codes are a function of the inputs: bit by bit, at every size of values, zeros, ties, the
    largest values, infinities and NaN."""
    n = 70
    w = World([n], [n], latent, 64, 16, dt, 8, seed=latent)
    g = w.gen
    c = torch.randn((n, latent), generator=g) * torch.exp2(torch.randint(-40 if dt == BF else -24, 100 if dt == BF else 12, (n, 1), generator=g).float())
    c = c.to(dt)
    c[0], c[1] = 0, -0.0
    c[2, :32], c[2, 32:64], c[2, 64:96] = 448.0, 450.0, torch.arange(32) - 16.0
    c[3] = torch.finfo(dt).max
    c[4] = torch.finfo(dt).smallest_normal / 8
    c[5] = (torch.arange(latent) % 64 * 0.0625 + 0.03125 + 1).to(dt)  # halfway between codes
    c[6, 5], c[7, 40], c[8, 70] = math.inf, -math.inf, math.nan
    got_c, *_ = store(w, 0, "half", None, c=c)
    codes, powers, bad = lref.encode(got_c)
    have = w.cells(0)
    assert torch.equal(have[:, latent:latent + latent // 32], powers)
    keep = ~bad.repeat_interleave(32, 1)
    assert torch.equal(have[:, :latent][keep], codes[keep])
    rows = w.cache.read(w.batch, ints([0, n]), rows=n)[:, :latent]
    want = lref.decode(codes, powers, dt)
    want[~keep] = math.nan
    assert torch.equal(rows.double().cpu().nan_to_num(12345.0, 1e39, -1e39), want.nan_to_num(12345.0, 1e39, -1e39))
    assert torch.isfinite(want[keep]).all()


def test_8_bits_hold_the_16_bit_norm():
    """The codes are those of the normalised latents as the 16-bit cache holds them."""
    n = 200
    a, b = (World([n], [n], 512, 64, 64, BF, bits, seed=4) for bits in (16, 8))
    weight = (torch.rand(512, generator=a.gen) + 0.5).to(BF).cuda()
    c = torch.randn((n, 512), generator=a.gen).to(BF)
    for w in (a, b):
        store(w, 0, "half", weight, c=c)
    codes, powers, _ = lref.encode(a.cells(0)[:, :1024].contiguous().view(BF))
    assert torch.equal(b.cells(0)[:, :512], codes) and torch.equal(b.cells(0)[:, 512:528], powers)


def test_append_over_its_queries():
    a, b = (World([5, 1], [9, 30], 256, 32, 16, BF, 16, seed=6) for _ in range(2))
    got = [store(w, 7, "interleaved", None, inplace=x) for w, x in ((a, False), (b, True))]
    assert torch.equal(got[0][4], got[1][4]) and torch.equal(a.cells(1), b.cells(1))


@pytest.mark.parametrize("q_lens,kv_lens,heads,latent,rope,page,dt,bits,layout", STORE)
@pytest.mark.parametrize("gap", [0, 16])
def test_read(q_lens, kv_lens, heads, latent, rope, page, dt, bits, layout, gap):
    w = World(q_lens, kv_lens, latent, rope, page, dt, bits, seed=heads, gap=gap)
    cu = starts(kv_lens)
    buf = torch.full((cu[-1] + 3, latent + rope + 8), 7.0, dtype=dt, device="cuda")
    out = w.cache.read(w.batch, ints(cu), out=buf[:, :latent + rope])
    torch.cuda.synchronize()
    assert w.cache.status() == 0 and out.data_ptr() == buf.data_ptr()
    want = torch.cat([torch.cat([c, k], 1) for c, k in zip(w.c, w.key)])
    assert torch.equal(out[:cu[-1]].cpu(), want)
    assert (buf[cu[-1]:] == 7).all() and (buf[:, latent + rope:] == 7).all()


def test_read_of_other_rows_than_cached_is_recorded():
    from expert_slot_cache_device_gb300 import ftmoe as F

    w = World([1, 1, 1], [20, 30, 40], 128, 16, 16, BF, 16)
    out = torch.full((90, 144), 7.0, dtype=BF, device="cuda")
    w.cache.read(w.batch, ints([0, 10, 50, 90]), out=out)  # ten rows for twenty tokens, forty for thirty
    torch.cuda.synchronize()
    assert w.cache.status() == F.ERR_STATE
    full = [torch.cat([c, k], 1) for c, k in zip(w.c, w.key)]
    assert torch.equal(out[:10].cpu(), full[0][:10]) and torch.equal(out[10:40].cpu(), full[1]) and (out[40:50] == 7).all()
    assert torch.equal(out[50:].cpu(), full[2])
    w.cache.reset_status()
    w.cache.read(w.batch, ints([-5, 1000, 20, 60]), out=out.fill_(7.0))
    torch.cuda.synchronize()
    assert w.cache.status() == F.ERR_STATE


# ---------------------------------------------------------------- absorbed attention
ATTEND = [
    # q_lens, kv_lens, heads, latent, rope, page, dtype, bits
    ([1], [1], 1, 512, 64, 16, BF, 16),
    ([1, 1, 1], [0, 17, 64], 16, 512, 64, 16, BF, 16),
    ([1] * 6, [1, 63, 64, 65, 129, 700], 20, 256, 32, 32, HF, 16),
    ([1] * 3, [5000, 1, 2049], 128, 512, 64, 64, BF, 16),
    ([1] * 4, [333, 1, 64, 65], 100, 384, 48, 16, HF, 16),
    ([1] * 5, [900, 130, 64, 1, 31], 32, 512, 64, 64, BF, 8),
    ([1] * 2, [333, 4100], 16, 512, 64, 16, HF, 8),
    ([1], [20000], 7, 512, 64, 128, BF, 16),
    ([1], [9000], 65, 128, 16, 256, BF, 8),
    ([4, 4, 3], [900, 5, 64], 16, 512, 64, 16, BF, 16),
    ([2, 0, 5], [130, 12, 700], 24, 256, 64, 32, HF, 8),
    ([8, 1], [2300, 40], 128, 512, 64, 64, BF, 16),
    ([70, 9, 130], [600, 9, 131], 5, 128, 32, 16, BF, 16),
    ([200], [200], 20, 512, 64, 16, HF, 16),
    ([20, 3], [7, 3], 6, 256, 16, 16, BF, 16),    # more new tokens than cached ones: rows that see nothing
    ([5, 2], [2, 0], 130, 512, 64, 32, BF, 8),
    ([1] * 150, [(37 * i) % 301 for i in range(150)], 3, 128, 16, 16, BF, 16),  # more sequences than SMs
    ([1] * 300, [(53 * i) % 97 for i in range(300)], 64, 256, 64, 16, HF, 8),
]


def check_attend(w, heads, scale=None, causal=True, want_lse=True):
    q, qr = w.queries(heads)
    scale = scale or (w.latent // 4 + w.rope) ** -0.5
    out = torch.full((w.tokens, heads, w.latent), 7.0, dtype=w.dtype, device="cuda")
    lse = torch.full((w.tokens, heads), 7.0, device="cuda") if want_lse else None
    w.cache.attend(w.batch, q, qr, scale, causal=causal, out=out, lse=lse)
    torch.cuda.synchronize()
    assert w.cache.status() == 0
    for i in range(len(w.kv_lens)):
        part = slice(w.cu[i], w.cu[i + 1])
        o, z, ot, zt = lref.absorbed(q[part].cpu(), qr[part].cpu(), w.c[i], w.key[i], scale, causal)
        check_rows(i, out[part], o, ot, lse[part] if want_lse else None, z, zt)
    assert (out[w.cu[-1]:] == 7).all()
    return out, lse


def check_rows(i, out, o, ot, lse, z, zt):
    d = (out.double().cpu() - o).abs()
    assert (d <= ot).all(), (i, "out", float((d / ot).max()))
    if lse is not None:
        none = z == -math.inf
        assert torch.equal(lse.cpu() == -math.inf, none)
        d = torch.where(none, 0.0, (lse.double().cpu() - z).abs())
        assert (d <= zt + 1e-12).all(), (i, "lse", float((d / (zt + 1e-12)).max()))


@pytest.mark.parametrize("q_lens,kv_lens,heads,latent,rope,page,dt,bits", ATTEND)
def test_attend(q_lens, kv_lens, heads, latent, rope, page, dt, bits):
    w = World(q_lens, kv_lens, latent, rope, page, dt, bits, seed=heads, slack=1)
    check_attend(w, heads)


@pytest.mark.parametrize("q_lens,kv_lens,heads,bits", [([5, 3, 2], [64, 1, 0], 12, 16), ([70, 9], [300, 5], 4, 8), ([1, 1], [900, 64], 128, 16)])
def test_attend_without_causality(q_lens, kv_lens, heads, bits):
    check_attend(World(q_lens, kv_lens, 256, 32, 16, BF, bits, seed=3), heads, causal=False, want_lse=False)


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("dt", [BF, HF])
def test_attend_with_far_scores(bits, dt):
    """Scores of thousands (one slot takes all), growing along the cache and falling along it."""
    n = 700
    for ends in ((0.01, 8.0), (8.0, 0.01)):
        w = World([1, 2], [n, 130], 256, 32, 16, dt, bits, seed=9, gap=16)
        check_attend(w, 20, scale=4.0)
        # the latents grow or shrink along the cache: the maximum moves with each tile
        size = torch.linspace(*ends, n).to(dt)
        c = (torch.ones(n, 256, dtype=dt) * size[:, None]).to(dt)
        if bits == 16:
            rows = torch.cat([c, w.key[0]], 1).view(torch.uint8)
        else:
            codes, powers, _ = lref.encode(c)
            c, rows = lref.decode(codes, powers, dt).to(dt), lref.pack(codes, powers, w.key[0])
        p, r = ref.cells(w.table[0], w.page, n)
        w.raw[p.cuda(), r.cuda(), :rows.shape[1]] = rows.cuda()
        w.c[0] = c
        check_attend(w, 20, scale=1.0)


def test_attend_over_its_queries_and_strides():
    for q_lens, kv_lens, heads, bits in (([1, 1, 4], [700, 5, 64], 16, 16), ([2, 1], [9000, 4000], 70, 8)):
        w = World(q_lens, kv_lens, 512, 64, 16, BF, bits, seed=1, gap=32)
        out, _ = check_attend(w, heads)
        q, qr = w.queries(heads)
        want = w.cache.attend(w.batch, q, qr, 0.1)
        got = w.cache.attend(w.batch, q, qr, 0.1, out=q)
        assert got is q and torch.equal(got, want)


def test_bad_pages_and_lengths_are_recorded():
    from expert_slot_cache_device_gb300 import ftmoe as F
    from expert_slot_cache_device_gb300.kv_cache import KVBatch

    for bits in (16, 8):
        w = World([1, 1], [100, 90], 256, 64, 16, BF, bits)
        q, qr = w.queries(10)
        good = w.cache.attend(w.batch, q, qr, 0.1).clone()
        for page in (-1, 1 << 30, w.raw.shape[0]):
            table = w.table.clone()
            table[0, 3] = page
            b = KVBatch(table.cuda(), ints(w.kv_lens), ints(w.cu), 1, 100)
            out = w.cache.attend(b, q, qr, 0.1)
            torch.cuda.synchronize()
            assert w.cache.status() == F.ERR_ID_RANGE and torch.equal(out[1], good[1])
            w.cache.reset_status()
            rows = torch.full((190, 320), 7.0, dtype=BF, device="cuda")
            w.cache.read(b, ints([0, 100, 190]), out=rows)
            assert w.cache.status() == F.ERR_ID_RANGE and (rows[48:64] == 7).all() and torch.equal(rows[64:100].cpu(), torch.cat([w.c[0], w.key[0]], 1)[64:])
            w.cache.reset_status()
        for lens, cu in (([101, 90], w.cu), ([100, -4], w.cu), (w.kv_lens, [0, 3, 2]), (w.kv_lens, [0, 2, 2])):
            w.cache.attend(KVBatch(w.table.cuda(), ints(lens), ints(cu), 1, 100), q, qr, 0.1)
            assert w.cache.status() == F.ERR_STATE
            w.cache.reset_status()


# ---------------------------------------------------------------- expanded attention
EXPAND = [
    # q_lens, kv_lens, heads, nope, rope, dtype
    ([1], [1], 1, 128, 64, BF),
    ([1, 1, 3], [0, 17, 64], 4, 64, 32, BF),
    ([5, 130, 1], [40, 131, 129], 3, 128, 64, HF),
    ([257], [257], 2, 128, 64, BF),
    ([300, 7, 64], [900, 7, 65], 5, 64, 64, HF),
    ([64, 300], [2000, 300], 3, 128, 16, BF),
    ([20, 300], [7, 170], 2, 128, 64, BF),        # more new tokens than rows
    ([40, 0, 9], [5000, 30, 4100], 2, 64, 48, BF),
    ([700], [700], 9, 128, 64, HF),
    ([128, 256, 129], [128, 256, 129], 8, 64, 16, BF),
    ([3] * 200, [(31 * i) % 150 for i in range(200)], 2, 64, 32, BF),
]


def expand_world(q_lens, kv_lens, heads, nope, rope, dt, seed=0):
    from expert_slot_cache_device_gb300.latent_cache import ExpandedBatch

    g = torch.Generator().manual_seed(seed)
    cu_q, cu_kv = starts(q_lens), starts(kv_lens)
    n, m = cu_q[-1] + 1, cu_kv[-1] + 2
    mk = lambda *s: torch.randn(s, generator=g).to(dt)  # noqa: E731
    q, kv, low = mk(n, heads + 1, nope + rope + 8) * 1.5, mk(m, heads, 2 * nope), mk(m, 128 + rope)
    kv[cu_kv[-1]:], low[cu_kv[-1]:] = math.nan, math.nan  # rows that no sequence has
    if m > 2 and kv_lens[0] and q_lens[0] == 0:
        kv[:kv_lens[0]] = math.nan
    q, kv, low = q.cuda(), kv.cuda(), low.cuda()
    b = ExpandedBatch(ints(cu_q), ints(cu_kv), max(q_lens), max(kv_lens))
    return b, q[:, 1:, 8:], kv[..., :nope], low[:, 128:], kv[..., nope:], cu_q, cu_kv


def check_expand(q_lens, kv_lens, heads, nope, rope, dt, causal=True, scale=None, seed=0):
    b, q, k, key, v, cu_q, cu_kv = expand_world(q_lens, kv_lens, heads, nope, rope, dt, seed)
    out = torch.full((q.shape[0], heads, nope), 7.0, dtype=dt, device="cuda")
    lse = torch.full((q.shape[0], heads), 7.0, device="cuda")
    b.attend(q, k, key, v, scale=scale, causal=causal, out=out, lse=lse)
    torch.cuda.synchronize()
    assert b.status() == 0
    for i in range(len(q_lens)):
        t, r = slice(cu_q[i], cu_q[i + 1]), slice(cu_kv[i], cu_kv[i + 1])
        o, z, ot, zt = lref.expanded(q[t].cpu(), k[r].cpu(), key[r].cpu(), v[r].cpu(), scale or (nope + rope) ** -0.5, causal)
        check_rows(i, out[t], o, ot, lse[t], z, zt)
    assert (out[cu_q[-1]:] == 7).all() and (lse[cu_q[-1]:] == 7).all()


@pytest.mark.parametrize("q_lens,kv_lens,heads,nope,rope,dt", EXPAND)
def test_expand(q_lens, kv_lens, heads, nope, rope, dt):
    check_expand(q_lens, kv_lens, heads, nope, rope, dt, seed=heads)


def test_expand_without_causality_and_far_scores():
    check_expand([40, 3, 2], [300, 1, 0], 3, 128, 64, BF, causal=False)
    check_expand([90, 70], [300, 64], 2, 64, 32, HF, scale=5.0)
    check_expand([300], [1000], 2, 128, 64, BF, scale=5.0)


def test_expand_bad_offsets_are_recorded():
    from expert_slot_cache_device_gb300 import ftmoe as F
    from expert_slot_cache_device_gb300.latent_cache import ExpandedBatch

    b, q, k, key, v, cu_q, cu_kv = expand_world([5, 4], [40, 30], 2, 64, 32, BF)
    good = b.attend(q, k, key, v).clone()
    assert b.status() == 0
    for cq, ck, mq, mk in (([0, 5, 900], cu_kv, 5, 40), ([0, 9, 5], cu_kv, 9, 40), (cu_q, [0, 40, 500], 5, 40), (cu_q, [-3, 40, 70], 5, 43),
                           (cu_q, cu_kv, 3, 40), (cu_q, cu_kv, 5, 20)):
        bad = ExpandedBatch(ints(cq), ints(ck), mq, mk)
        bad.attend(q, k, key, v)
        assert bad.status() == F.ERR_STATE
        bad.reset_status()
    assert torch.equal(b.attend(q, k, key, v)[:9], good[:9])


# ---------------------------------------------------------------- together
def test_a_layer_of_latent_attention():
    """Prompt chunks through append, read and the expanded form, single tokens through the absorbed form: both agree with
    plain attention over everything written, in 16 and 8 bits."""
    from expert_slot_cache_device_gb300.kv_cache import KVBatch, Rotary, rotary_frequencies
    from expert_slot_cache_device_gb300.latent_cache import ExpandedBatch, LatentCache

    heads, latent, rope, nope, page = 4, 256, 32, 64, 16
    g = torch.Generator().manual_seed(11)
    mk = lambda *s, std=1.0: (torch.randn(s, generator=g) * std).to(BF)  # noqa: E731
    w_k, w_v, weight = mk(heads, nope, latent, std=latent ** -0.5), mk(heads, nope, latent, std=latent ** -0.5), (torch.rand(latent, generator=g) + 0.5).to(BF)
    freq, factor = rotary_frequencies(rope)
    scale = (nope + rope) ** -0.5
    for bits in (16, 8):
        cache, rotary = LatentCache(16, page, latent, rope, BF, bits), Rotary(rope, layout="interleaved")
        lens, tables = [0, 0], ints([[3, 9, 1, 14, 7, 2], [0, 5, 8, 13, 12, 4]])
        c_all, k_all = [torch.zeros((0, latent)).double()] * 2, [torch.zeros((0, rope)).double()] * 2
        for new in ([40, 17], [30, 1], [1, 1], [1, 1]):
            cu = starts(new)
            pos = torch.cat([torch.arange(n, n + m) for n, m in zip(lens, new)]).to(torch.int32)
            lens = [n + m for n, m in zip(lens, new)]
            c, key, q = mk(cu[-1], latent, std=2.0), mk(cu[-1], rope), mk(cu[-1], heads, nope + rope)
            qd = q.cuda()
            batch = KVBatch(tables, ints(lens), ints(cu), max(new), max(lens))
            cache.append(batch, rotary, c.cuda(), key.cuda(), pos.cuda(), weight=weight.cuda(), q_rope=qd[..., nope:], q_out=qd[..., nope:])
            rows = cache.read(batch, ints(starts(lens)), rows=sum(lens))
            lat = rows[:, :latent].float()
            if max(new) > 1:
                k, v = (torch.einsum("rl,hnl->rhn", lat, x.cuda().float()).to(BF) for x in (w_k, w_v))
                got = ExpandedBatch(ints(cu), ints(starts(lens)), max(new), max(lens)).attend(qd, k, rows[:, latent:], v)
            else:
                ql = torch.einsum("thn,hnl->thl", qd[..., :nope].float(), w_k.cuda().float()).to(BF)
                o = cache.attend(batch, ql, qd[..., nope:], scale)
                got = torch.einsum("thl,hnl->thn", o.float(), w_v.cuda().float())
            torch.cuda.synchronize()
            assert cache.status() == 0
            y, _ = lref.norm(c, weight, 1e-6)
            kr, qr = ref.rotate(key[:, None], pos, freq, factor, rope, "interleaved")[:, 0], ref.rotate(q[..., nope:], pos, freq, factor, rope, "interleaved")
            for i in range(2):
                t = slice(cu[i], cu[i + 1])
                c_all[i], k_all[i] = torch.cat([c_all[i], y[t]]), torch.cat([k_all[i], kr[t]])
                kk, vv = (torch.einsum("rl,hnl->rhn", c_all[i], x.double()) for x in (w_k, w_v))
                s = (torch.einsum("thn,rhn->htr", q[t, :, :nope].double(), kk) + torch.einsum("thn,rn->htr", qr[t], k_all[i])) * scale
                at = torch.arange(lens[i] - new[i], lens[i])[:, None]
                p = s.masked_fill(torch.arange(lens[i])[None] > at, -math.inf).softmax(-1)
                want = torch.einsum("htr,rhn->thn", p, vv)
                # roundings of the latents (2^-8, or 2^-4 for codes), keys, values, queries and outputs, as random ones: a
                # value is a sum of `latent` products, so relative to the rms of the outputs they add up in squares; six such
                err = (got[t].double().cpu() - want).square().mean().sqrt() / want.square().mean().sqrt()
                assert err <= 6 * (2.0 ** -4 if bits == 8 else 2.0 ** -8), (bits, new, float(err))


def test_other_streams_and_replayed_graphs():
    """All four on a stream of their own, captured into a graph and replayed with other lengths, twice at a time."""
    w = World([1, 1, 1], [300, 64, 700], 512, 64, 16, BF, 16, seed=5)
    q, qr = w.queries(40)
    b, qx, k, key, v, *_ = expand_world([30, 200], [500, 200], 2, 128, 64, BF)
    rows_n = sum(w.kv_lens)
    cu_rows = ints(starts(w.kv_lens))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    def step(stream=None):
        return w.cache.attend(w.batch, q, qr, 0.07, stream=stream), w.cache.read(w.batch, cu_rows, rows=rows_n, stream=stream), b.attend(qx, k, key, v, stream=stream)

    want = [x.clone() for x in step()]
    got = step(side)
    side.synchronize()
    assert all(torch.equal(a, g) for a, g in zip(want[:2], got[:2])) and torch.equal(want[2][:230], got[2][:230])
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.stream(side):
            step()
            side.synchronize()
            with torch.cuda.graph(g, stream=side):
                graphs.append((g, step()))
    lens = [200, 64, 333]
    short = w.cache.attend(type(w.batch)(w.table.cuda(), ints(lens), ints(w.cu), 1, 700), q, qr, 0.07)
    w.batch.kv_lens.copy_(ints(lens))
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        graphs[0][0].replay()
    with torch.cuda.stream(other):
        graphs[1][0].replay()
    torch.cuda.synchronize()
    for _, got in graphs:
        assert torch.equal(got[0], short) and torch.equal(got[2][:230], want[2][:230])
