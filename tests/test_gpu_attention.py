"""The attention half of a decoder layer on the GPU against plain implementations in 64 bits:
rotary positions and the write to the paged cache, attention of single tokens and chunks with its
log-sum-exp and mass, and eviction. Tolerances are what the stated roundings may move a result
by (tests/attention_reference.py)."""
import math

import pytest
import torch

import attention_reference as ref

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]
BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _built():
    from expert_slot_cache_device_gb300 import build

    build.build()


class World:
    """A cache, a batch with random pages, and its plain copies."""

    def __init__(self, q_lens, kv_lens, heads, kv_heads, dim, page, dtype, seed=0, order="slot", window=0, slack=0):
        from expert_slot_cache_device_gb300.kv_cache import KVBatch, PagedKVCache

        g = torch.Generator().manual_seed(seed)
        self.q_lens, self.kv_lens, self.page = q_lens, kv_lens, page
        b = len(kv_lens)
        need = [-(-n // page) for n in kv_lens]
        pages = sum(need) + 2
        perm = torch.randperm(pages, generator=g)
        # entries that no call needs are junk
        width = max(need + [1]) + 1
        self.table = torch.full((b, width), -(1 << 30), dtype=torch.int32)
        at = 0
        for i, m in enumerate(need):
            self.table[i, :m] = perm[at:at + m].to(torch.int32)
            at += m
        shape = (pages, page, kv_heads, dim) if order == "slot" else (pages, kv_heads, page, dim)
        mk = lambda: torch.full(shape, math.nan, dtype=dtype)  # noqa: E731  # slots never written hold NaN
        k, v = mk(), mk()
        if order != "slot":
            k, v = k.permute(0, 2, 1, 3), v.permute(0, 2, 1, 3)
        self.k_seq, self.v_seq = [], []
        for i, n in enumerate(kv_lens):
            ks, vs = (torch.randn((n, kv_heads, dim), generator=g).to(dtype) for _ in range(2))
            lo = max(0, n - q_lens[i] - window + 1) if window else 0  # the first slot that a row sees
            ks[:lo], vs[:lo] = math.nan, math.nan
            p, r = ref.cells(self.table[i], page, n)
            k[p, r], v[p, r] = ks, vs
            if window:
                self.table[i, :lo // page] = 1 << 29  # pages a window has left behind may be gone
            self.k_seq.append(ks)
            self.v_seq.append(vs)
        dev = lambda t: torch.empty_strided(t.shape, t.stride(), dtype=t.dtype, device="cuda").copy_(t)  # noqa: E731
        self.cache = PagedKVCache(pages, page, kv_heads, dim, dtype, k_pages=dev(k), v_pages=dev(v))
        self.cu = [sum(q_lens[:i]) for i in range(b + 1)]
        self.tokens = self.cu[-1] + slack
        self.batch = KVBatch(self.table.cuda(), torch.tensor(kv_lens, dtype=torch.int32).cuda(),
                             torch.tensor(self.cu, dtype=torch.int32).cuda(), max_q=max(q_lens), max_kv=max(kv_lens))
        # queries as a slice of a fused projection's output: rows further apart than heads * dim
        wide = torch.randn((self.tokens, heads + 2, dim), generator=g) * 1.5
        self.q = wide.to(dtype).cuda()[:, 1:heads + 1]
        self.heads, self.kv_heads, self.dim, self.dtype, self.gen = heads, kv_heads, dim, dtype, g


ATTEND = [
    # q_lens, kv_lens, heads, kv_heads, dim, page, window, dtype
    ([1], [1], 1, 1, 64, 16, 0, BF),
    ([1, 1, 1], [0, 17, 16], 4, 2, 128, 16, 0, BF),
    ([1] * 5, [1, 63, 64, 65, 700], 8, 1, 128, 32, 0, HF),
    ([1] * 3, [5000, 1, 2049], 16, 1, 64, 16, 0, BF),
    ([1] * 2, [333, 4100], 15, 3, 128, 64, 0, HF),
    ([1] * 2, [900, 130], 40, 2, 128, 256, 0, BF),
    ([1] * 4, [300, 127, 128, 129], 12, 4, 64, 16, 128, HF),
    ([1] * 2, [2000, 999], 6, 2, 128, 16, 1000, BF),
    ([2, 1], [9, 3], 2, 2, 64, 16, 0, BF),
    ([7, 0, 1, 30], [40, 12, 600, 30], 10, 2, 128, 16, 0, BF),
    ([130, 64], [131, 64], 7, 1, 64, 32, 0, HF),
    ([257], [1500], 6, 2, 128, 16, 0, BF),
    ([33, 100], [1000, 400], 24, 8, 64, 128, 0, BF),
    ([200, 3], [777, 500], 16, 2, 128, 64, 128, HF),
    ([64, 300], [65, 300], 4, 4, 64, 16, 1, BF),
    ([90], [260], 17, 1, 128, 16, 60, BF),
    ([520], [520], 12, 3, 128, 256, 0, HF),
    ([20, 5], [11, 5], 8, 4, 64, 16, 0, BF),    # more new tokens than cached ones: rows that see nothing
    ([300, 3], [170, 0], 4, 2, 128, 16, 0, HF),
    ([40, 4], [9000, 6100], 4, 1, 128, 16, 0, BF),
    ([2, 2], [3000, 12000], 8, 8, 64, 16, 0, HF),
    ([20, 9], [20000, 700], 8, 8, 64, 16, 0, BF),   # more pieces of work than SMs, in both passes of a chunk
    ([33, 40], [9000, 4100], 24, 8, 128, 32, 0, HF),
    ([97, 40, 13, 88, 2, 61, 30], [1500, 900, 1100, 300, 640, 1290, 200], 40, 8, 64, 16, 0, HF),  # pieces of 1, 2, ... row tiles
    ([300, 120, 7], [900, 2500, 3100], 32, 8, 64, 16, 200, BF),
]


def check_attend(w, window, sinks, causal, scale=None, mass=True, want_lse=True):
    b, n = len(w.kv_lens), max(w.kv_lens + [1])
    out = torch.full((w.tokens, w.heads, w.dim), 7.0, dtype=w.dtype, device="cuda")
    lse = torch.full((w.tokens, w.heads), 7.0, device="cuda") if want_lse else None
    m0 = torch.rand((b, w.kv_heads, n + 3), generator=w.gen)
    m = m0.cuda() if mass else None
    w.cache.attend(w.batch, w.q, window=window, sinks=sinks, causal=causal, out=out, lse=lse, mass=m, scale=scale)
    torch.cuda.synchronize()
    assert w.cache.status() == 0
    for i in range(b):
        part = slice(w.cu[i], w.cu[i + 1])
        o, l, ma, ot, lt, mt = ref.attention(w.q[part].cpu(), w.k_seq[i], w.v_seq[i],
                                             w.dim ** -0.5 if scale is None else scale, window, causal, sinks)
        d = (out[part].double().cpu() - o).abs()
        assert (d <= ot).all(), (i, "out", float((d - ot).max()), float((d / ot).max()))
        if want_lse:
            got = lse[part].double().cpu()
            inf = l == -math.inf
            assert torch.equal(got == -math.inf, inf), (i, "empty rows")
            d = (got - l).abs()[~inf]
            assert (d <= lt[~inf]).all(), (i, "lse", float((d / lt[~inf]).max()))
        if mass:
            got = m[i].double().cpu()
            d = (got[:, :w.kv_lens[i]] - (m0[i].double()[:, :w.kv_lens[i]] + ma)).abs()
            tol = mt + 4 * ref.F32 * (m0[i].double()[:, :w.kv_lens[i]] + ma)
            assert (d <= tol).all(), (i, "mass", float((d / tol).max()))
            assert torch.equal(m[i][:, w.kv_lens[i]:].cpu(), m0[i][:, w.kv_lens[i]:]), "mass past the length changed"
    rest = slice(w.cu[-1], w.tokens)
    assert (out[rest] == 7.0).all() and (lse is None or (lse[rest] == 7.0).all()), "rows of no sequence changed"


@pytest.mark.parametrize("case", ATTEND, ids=[str(i) for i in range(len(ATTEND))])
@pytest.mark.parametrize("mass", [False, True])
def test_attention(case, mass):
    q_lens, kv_lens, heads, kv, dim, page, window, dt = case
    w = World(q_lens, kv_lens, heads, kv, dim, page, dt, seed=len(kv_lens) + dim, window=window, slack=2)
    check_attend(w, window, None, True, mass=mass)


@pytest.mark.parametrize("count,q,heads,kv,dim,page", [(400, 1, 17, 1, 64, 16), (300, 1, 2, 1, 128, 16), (390, 3, 8, 1, 64, 32),
                                                       (150, 2, 6, 2, 128, 16)])
def test_attention_many_sequences(count, q, heads, kv, dim, page):
    """More sequences than a CTA has threads, some without new tokens, some empty."""
    r = torch.Generator().manual_seed(count)
    q_lens = [int(torch.randint(0, q + 1, (1,), generator=r)) for _ in range(count)]
    kv_lens = [int(torch.randint(0, 70, (1,), generator=r)) + n for n in q_lens]
    kv_lens[3], kv_lens[count - 1], q_lens[count - 1] = 0, 300, q
    w = World(q_lens, kv_lens, heads, kv, dim, page, BF, seed=count)
    check_attend(w, 0, None, True)


@pytest.mark.parametrize("heads,kv,q_lens,kv_lens", [(128, 1, [3, 2], [200, 90]), (40, 1, [9, 1], [30, 400]), (33, 1, [1], [77]),
                                                     (100, 2, [5], [300])])
def test_attention_wide_groups(heads, kv, q_lens, kv_lens):
    """Query heads a key head up to the most there can be, and ones that leave rows of a tile unused."""
    for dim, dt in ((64, BF), (128, HF)):
        check_attend(World(q_lens, kv_lens, heads, kv, dim, 16, dt, seed=heads), 0, None, True)


@pytest.mark.parametrize("case", [ATTEND[i] for i in (1, 4, 6, 9, 13, 17, 19)], ids=str)
def test_attention_sinks_and_head_order(case):
    """A sink logit per head (one of them -inf: none), and caches with heads outside slots."""
    q_lens, kv_lens, heads, kv, dim, page, window, dt = case
    w = World(q_lens, kv_lens, heads, kv, dim, page, dt, seed=5, order="head", window=window)
    sinks = torch.linspace(-2, 3, heads)
    sinks[0] = -math.inf
    check_attend(w, window, sinks.cuda(), True, mass=True)


@pytest.mark.parametrize("case", [ATTEND[i] for i in (2, 9, 10, 16)], ids=str)
def test_attention_not_causal(case):
    q_lens, kv_lens, heads, kv, dim, page, _, dt = case
    w = World(q_lens, kv_lens, heads, kv, dim, page, dt, seed=6)
    check_attend(w, 0, None, False, mass=True, scale=0.3, want_lse=False)


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("q_lens,kv_lens", [([1, 1], [2500, 40]), ([70, 9], [600, 2000])])
def test_attention_large_scores(dt, q_lens, kv_lens):
    """Scores of about +-150, so that most probabilities vanish and the running maximum jumps."""
    w = World(q_lens, kv_lens, 8, 2, 64, 16, dt, seed=9)
    check_attend(w, 0, None, True, mass=True, scale=3.0)


def test_attention_repeats_bit_for_bit_and_on_another_stream():
    w = World([1, 90, 5], [4000, 800, 2600], 12, 2, 128, 16, BF, seed=3)
    got = []
    side = torch.cuda.Stream()
    for stream in (None, None, side, side.cuda_stream):
        m = torch.zeros((3, 2, 4000), device="cuda")
        torch.cuda.synchronize()
        o = w.cache.attend(w.batch, w.q, mass=m, stream=stream)
        torch.cuda.synchronize()
        got.append((o.clone(), m))
    for o, m in got[1:]:
        assert torch.equal(o, got[0][0]) and torch.equal(m, got[0][1])


def test_attention_of_one_batch_on_two_streams_at_once():
    """Calls of one batch that overlap on two streams, whose workspaces the batch keeps, growing in between."""
    w = World([1, 90, 5], [4000, 800, 2600], 12, 2, 128, 16, BF, seed=5)
    want = w.cache.attend(w.batch, w.q).clone()
    mass = torch.zeros((3, 2, 4000), device="cuda")
    w.cache.attend(w.batch, w.q, mass=mass)
    sides = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [[torch.empty_like(want) for _ in range(12)] for _ in sides]
    sums = [torch.zeros_like(mass) for _ in sides]
    torch.cuda.synchronize()
    for i in range(12):
        for s, o, m in zip(sides, outs, sums):
            with torch.cuda.stream(s):
                w.cache.attend(w.batch, w.q, out=o[i], mass=m if i == 7 else None)
    torch.cuda.synchronize()
    for o, m in zip(outs, sums):
        assert all(torch.equal(x, want) for x in o) and torch.equal(m, mass)


def test_attention_in_a_graph_follows_its_device_arrays():
    """A captured step reads lengths and tables when it is replayed."""
    w = World([1, 1, 1], [900, 17, 450], 8, 2, 64, 16, BF, seed=4)
    out = torch.empty((3, 8, 64), dtype=BF, device="cuda")
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        w.cache.attend(w.batch, w.q, out=out)
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            w.cache.attend(w.batch, w.q, out=out)
    short = [300, 1, 449]
    w.batch.kv_lens.copy_(torch.tensor(short, dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    for i, n in enumerate(short):
        o, _, _, ot, _, _ = ref.attention(w.q[i:i + 1].cpu(), w.k_seq[i][:n], w.v_seq[i][:n], 64 ** -0.5, 0, True, None)
        assert ((out[i:i + 1].double().cpu() - o).abs() <= ot).all()


def test_bad_pages_and_lengths_are_recorded():
    """A table entry outside the cache, lengths out of their bounds: recorded, nothing else touched."""
    from expert_slot_cache_device_gb300 import ftmoe as F

    for q in (1, 40):
        w = World([q, q], [100, 100], 4, 2, 64, 16, BF, seed=8)
        w.batch.block_table[0, 3] = w.cache.num_pages
        o = w.cache.attend(w.batch, w.q, mass=torch.zeros((2, 2, 100), device="cuda"))
        assert w.cache.status() == F.ERR_ID_RANGE
        r, _, _, t, _, _ = ref.attention(w.q[q:].cpu(), w.k_seq[1], w.v_seq[1], 64 ** -0.5, 0, True, None)
        assert ((o[q:].double().cpu() - r).abs() <= t).all()
        w.cache.reset_status()
        assert w.cache.status() == 0
        w.batch.block_table[0, 3] = 0
        w.batch.kv_lens[0] = 1000
        w.cache.attend(w.batch, w.q)
        assert w.cache.status() == F.ERR_STATE
        w.cache.reset_status()
        w.batch.kv_lens[0] = 100
        w.batch.cu_q[2] = 5 * q
        w.cache.attend(w.batch, w.q)
        assert w.cache.status() == F.ERR_STATE


# ---------------------------------------------------------------- append
@pytest.mark.parametrize("dim,rot,layout,scaling,dt,page,order", [
    (128, 128, "half", None, BF, 16, "slot"),
    (128, 64, "interleaved", dict(kind="yarn", factor=8.0, original=4096), HF, 32, "slot"),
    (64, 16, "half", dict(kind="linear", factor=4.0), BF, 16, "head"),
    (96, 48, "interleaved", dict(kind="base", factor=2.0), HF, 64, "slot"),
    (256, 256, "half", dict(kind="banded", factor=8.0, original=8192), BF, 256, "head"),
    (80, 32, "half", None, BF, 16, "slot"),
])
@pytest.mark.parametrize("q_lens,kv_lens", [([1], [1]), ([1, 1, 1, 1], [33, 1, 16, 500]), ([70, 0, 3], [90, 7, 3])])
def test_append(dim, rot, layout, scaling, dt, page, order, q_lens, kv_lens):
    from expert_slot_cache_device_gb300.kv_cache import Rotary, rotary_frequencies

    w = World(q_lens, kv_lens, 6, 3, dim, page, dt, seed=dim + rot, order=order, slack=1)
    rot_plan = Rotary(dim, rot, 10000.0, layout, scaling)
    freq, factor = rotary_frequencies(rot, 10000.0, scaling)
    k, v = (torch.randn((w.tokens, 3, dim), generator=w.gen).to(dt).cuda() for _ in range(2))
    pos = torch.randint(0, 1 << 24, (w.tokens,), generator=w.gen).to(torch.int32)
    pos[0] = (1 << 24) - 1
    before_k, before_v = w.cache.k_pages.clone(), w.cache.v_pages.clone()
    q_in = w.q.clone()
    q_out = torch.full_like(q_in, 7.0)
    w.cache.append(w.batch, rot_plan, w.q, k, v, pos.cuda(), q_out=q_out)
    assert w.cache.status() == 0

    def close(got, x, sel):
        want = ref.rotate(x[sel], pos[sel], freq, factor, rot, layout)
        size = x[sel].double().cpu().abs()
        pair = size.max(-1, keepdim=True).values * 2
        # the result's rounding; angles within 2^-23 turns (6.3 radians each) and the sine's last places
        tol = ref.U[dt] * want.abs() + factor * pair * 2.0 ** -19 + 2.0 ** -25
        assert ((got.double().cpu() - want).abs() <= tol).all()
        assert torch.equal(got[..., rot:].cpu(), x[sel][..., rot:].cpu())

    used = torch.zeros(before_k.shape[:2], dtype=torch.bool)
    for i, n in enumerate(kv_lens):
        sel = slice(w.cu[i], w.cu[i + 1])
        if q_lens[i] == 0:
            continue
        close(q_out[sel], q_in, sel)
        p, r = ref.cells(w.table[i], page, n)
        p, r = p[n - q_lens[i]:], r[n - q_lens[i]:]
        close(w.cache.k_pages[p, r], k, sel)
        assert torch.equal(w.cache.v_pages[p, r], v[sel])
        used[p, r] = True
    keep = ~used.cuda()
    for got, was in ((w.cache.k_pages, before_k), (w.cache.v_pages, before_v)):
        assert torch.equal(got[keep].nan_to_num(9.0), was[keep].nan_to_num(9.0)), "another slot changed"
    assert (q_out[w.cu[-1]:] == 7.0).all()
    # in place, and without queries
    w.cache.append(w.batch, rot_plan, w.q, k, v, pos.cuda(), q_out=w.q)
    assert torch.equal(w.q[:w.cu[-1]], q_out[:w.cu[-1]])
    w.cache.append(w.batch, rot_plan, None, k, v, pos.cuda())
    assert w.cache.status() == 0


def test_append_slots_without_a_page():
    """More new tokens than cached ones: the rows before slot 0 write nothing, their queries turn."""
    from expert_slot_cache_device_gb300 import ftmoe as F
    from expert_slot_cache_device_gb300.kv_cache import Rotary

    w = World([5], [3], 2, 1, 64, 16, BF, seed=1)
    k, v = (torch.randn((5, 1, 64), generator=w.gen).to(BF).cuda() for _ in range(2))
    pos = torch.zeros(5, dtype=torch.int32, device="cuda")
    out = w.cache.append(w.batch, Rotary(64), w.q, k, v, pos)
    p, r = ref.cells(w.table[0], 16, 3)
    assert torch.equal(w.cache.v_pages[p, r], v[2:]) and torch.equal(out, w.q) and w.cache.status() == 0
    w.batch.block_table[0, 0] = -5
    was = w.cache.k_pages.clone()
    w.cache.append(w.batch, Rotary(64), w.q, k, v, pos)
    assert w.cache.status() == F.ERR_ID_RANGE
    assert torch.equal(w.cache.k_pages.nan_to_num(9.0), was.nan_to_num(9.0))


# ---------------------------------------------------------------- evict
@pytest.mark.parametrize("lens,kv,dim,page,budget,recent,dt", [
    ([1], 1, 64, 16, 1, 0, BF),
    ([0, 5, 17, 16], 2, 64, 16, 16, 4, BF),
    ([100, 99, 3], 3, 128, 32, 50, 50, HF),
    ([1000, 2049, 2048], 2, 128, 16, 700, 0, BF),
    ([5000], 4, 64, 64, 4999, 100, HF),
    ([9000, 20], 1, 96, 16, 33, 1, BF),
    ([70001, 400], 1, 64, 256, 5000, 128, BF),
])
@pytest.mark.parametrize("kind", ["spread", "ties", "odd"])
def test_evict(lens, kv, dim, page, budget, recent, dt, kind):
    w = World([1] * len(lens), lens, kv, kv, dim, page, dt, seed=len(lens), order="head" if kv == 2 else "slot")
    g = w.gen
    n = max(lens)
    mass = torch.rand((len(lens), kv, n + 1), generator=g) * 4
    if kind == "ties":
        mass = mass.floor() * 0.5  # three values: most of the order is by slot
    if kind == "odd":  # negative numbers, both zeros, infinities, NaN, subnormals
        pick = torch.randint(0, 8, mass.shape, generator=g)
        special = torch.tensor([0.0, -0.0, math.inf, -math.inf, math.nan, 1e-40, -3.0, 2.0])
        mass = torch.where(torch.rand(mass.shape, generator=g) < 0.6, special[pick], mass - 2)
    most = min(budget, n)
    width = -(-most // page)
    pages = w.cache.num_pages
    from expert_slot_cache_device_gb300.kv_cache import PagedKVCache

    big_k = torch.full((pages + width * len(lens), page, kv, dim), 5.0, dtype=dt, device="cuda")
    big_v = big_k.clone()
    big_k[:pages], big_v[:pages] = w.cache.k_pages, w.cache.v_pages
    cache = PagedKVCache(big_k.shape[0], page, kv, dim, dt, k_pages=big_k, v_pages=big_v)
    new_table = (pages + torch.randperm(width * len(lens), generator=g)).view(len(lens), width).to(torch.int32)
    before = cache.k_pages.clone()
    kept, new_mass, new_lens = cache.evict(w.batch, mass.cuda(), new_table.cuda(), budget=budget, recent=recent)
    assert cache.status() == 0
    written = torch.zeros(big_k.shape[:3], dtype=torch.bool)
    for i, m in enumerate(lens):
        assert int(new_lens[i]) == min(m, budget)
        for h in range(kv):
            want = ref.evict(mass[i, h], m, budget, recent)
            assert kept[i, h].tolist() == want + [-1] * (budget - len(want)), (i, h)
            assert torch.equal(new_mass[i, h, :len(want)].cpu().nan_to_num(77.0), mass[i, h, want].nan_to_num(77.0))
            assert (new_mass[i, h, len(want):] == 0).all()
            p, r = ref.cells(new_table[i], page, len(want))
            written[p, r, h] = True
            assert torch.equal(cache.k_pages[p, r, h].cpu(), w.k_seq[i][want, h])
            assert torch.equal(cache.v_pages[p, r, h].cpu(), w.v_seq[i][want, h])
    rest = ~written.cuda()
    assert torch.equal(cache.k_pages[rest].nan_to_num(9.0), before[rest].nan_to_num(9.0)), "another row changed"


def test_evict_bad_pages():
    from expert_slot_cache_device_gb300 import ftmoe as F

    w = World([1], [64], 1, 1, 64, 16, BF, seed=2)
    mass = torch.rand((1, 1, 64), device="cuda")
    was = w.cache.v_pages.clone()
    w.cache.evict(w.batch, mass, torch.full((1, 2), 1 << 20, dtype=torch.int32, device="cuda"), budget=32, recent=4)
    assert w.cache.status() == F.ERR_ID_RANGE
    assert torch.equal(w.cache.v_pages.nan_to_num(9.0), was.nan_to_num(9.0))


# ---------------------------------------------------------------- together
def test_mass_of_a_chunk_equals_its_tokens_one_by_one():
    """The same rows as one chunk and as single tokens: outputs and mass agree within both bounds."""
    w = World([24], [400], 8, 2, 128, 16, BF, seed=12)
    from expert_slot_cache_device_gb300.kv_cache import KVBatch

    a, b = (torch.zeros((1, 2, 400), device="cuda") for _ in range(2))
    whole = w.cache.attend(w.batch, w.q, mass=a)
    cu = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    for i in range(24):
        n = 400 - 24 + i + 1
        one = KVBatch(w.batch.block_table, torch.tensor([n], dtype=torch.int32, device="cuda"), cu, 1, n)
        out = w.cache.attend(one, w.q[i:i + 1], mass=b)
        o, _, _, ot, _, _ = ref.attention(w.q[i:i + 1].cpu(), w.k_seq[0][:n], w.v_seq[0][:n], 128 ** -0.5, 0, True, None)
        assert ((out.double() - whole[i:i + 1].double()).abs().cpu() <= 2 * ot).all()
    assert torch.allclose(a, b, rtol=1e-4, atol=1e-6)
    assert abs(float(a.sum()) - 24 * 8) < 1e-2


def test_long_cache_offsets_past_32_bits():
    """Pages whose element offsets do not fit 32 bits are read, written and moved."""
    from expert_slot_cache_device_gb300.kv_cache import KVBatch, PagedKVCache, Rotary

    page, kv, dim = 256, 8, 128
    pages = (1 << 32) // (page * kv * dim) + 3  # 2^32 elements and some: 8.6 GB each
    cache = PagedKVCache(pages, page, kv, dim, BF)
    g = torch.Generator(device="cuda").manual_seed(0)
    use = [pages - 1, 0, pages - 2]
    for p in use:
        cache.k_pages[p].normal_(generator=g)
        cache.v_pages[p].normal_(generator=g)
    n = 300
    table = torch.tensor([use[:2]], dtype=torch.int32, device="cuda")
    for q_len in (1, 40):
        batch = KVBatch(table, torch.tensor([n], dtype=torch.int32, device="cuda"),
                        torch.tensor([0, q_len], dtype=torch.int32, device="cuda"), q_len, n)
        q, k, v = (torch.randn((q_len, h, dim), generator=g, device="cuda").to(BF) for h in (16, kv, kv))
        pos = torch.arange(n - q_len, n, dtype=torch.int32, device="cuda")
        q = cache.append(batch, Rotary(dim), q, k, v, pos)
        mass = torch.zeros((1, kv, n), device="cuda")
        out = cache.attend(batch, q, mass=mass)
        p, r = ref.cells(table[0].cpu(), page, n)
        o, _, m, ot, _, _ = ref.attention(q.cpu(), cache.k_pages[p, r].cpu(), cache.v_pages[p, r].cpu(), dim ** -0.5, 0, True, None)
        assert torch.equal(cache.v_pages[p, r][n - q_len:], v)
        assert ((out.double().cpu() - o).abs() <= ot).all()
        assert torch.allclose(mass[0].double().cpu(), m, rtol=1e-4, atol=1e-7)
    kept, _, lens = cache.evict(batch, mass, torch.tensor([[use[2]]], dtype=torch.int32, device="cuda"), budget=200, recent=16)
    assert int(lens) == 200 and cache.status() == 0
    for h in range(kv):
        j = kept[0, h].long()
        assert torch.equal(cache.k_pages[use[2], :200, h], cache.k_pages[p.cuda()[j], r.cuda()[j], h])
