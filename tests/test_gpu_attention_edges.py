"""The attention half at the ends of what its calls take, against its calls in plain use and plain
implementations in 64 bits."""
import math

import pytest
import torch

import attention_reference as ref
from test_gpu_attention import BF, HF, World, check_attend

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from expert_slot_cache_device_gb300 import build

    build.build()


def run(w, window=0, sinks=None, mass=True, q=None, out=None):
    """(out, lse, mass) of a call on the world's cache."""
    q = w.q if q is None else q
    out = torch.full((w.tokens, w.heads, w.dim), 7.0, dtype=w.dtype, device="cuda") if out is None else out
    lse = torch.full((w.tokens, w.heads), 7.0, device="cuda")
    m = torch.zeros((len(w.kv_lens), w.kv_heads, max(w.kv_lens + [1])), device="cuda") if mass else None
    w.cache.attend(w.batch, q, window=window, sinks=sinks, out=out, lse=lse, mass=m)
    torch.cuda.synchronize()
    assert w.cache.status() == 0
    return out, lse, m


@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 60, 1 << 30, 2 ** 32 + 5, 2 ** 63 - 1])
@pytest.mark.parametrize("q_lens,kv_lens,heads,kv,dim,dt", [
    ([300, 70], [300, 200], 8, 2, 64, BF),     # chunks: a whole prompt, and one late in its context
    ([90, 40], [70, 11], 4, 2, 128, HF),       # more new tokens than cached ones
    ([1, 1], [500, 33], 8, 2, 64, BF),         # single tokens
    ([4, 2], [1, 9], 4, 2, 128, BF),
])
def test_a_window_wider_than_any_cache_is_none(q_lens, kv_lens, heads, kv, dim, dt, window):
    w = World(q_lens, kv_lens, heads, kv, dim, 16, dt, seed=21)
    got, want = run(w, window), run(w, 0)
    for g, x in zip(got, want):
        assert torch.equal(g, x)
    check_attend(w, 0, None, True)


@pytest.mark.parametrize("q,kv_len", [(1, 130), (40, 130)])
def test_windows_about_the_length_of_the_cache(q, kv_len):
    for window in (kv_len - 1, kv_len, kv_len + 1):
        w = World([q], [kv_len], 4, 2, 64, 16, BF, seed=window, window=window)
        check_attend(w, window, None, True)


@pytest.mark.parametrize("q", [1, 40])
@pytest.mark.parametrize("with_sinks", [False, True])
def test_mass_of_caches_that_hold_nothing(q, with_sinks):
    """No sequence has a cached token, and the bound says so: out = 0, lse is the sink, mass stays."""
    w = World([q, q], [0, 0], 4, 2, 64, 16, BF, seed=3)
    assert w.batch.max_kv == 0
    sinks = torch.linspace(-1, 1, 4).cuda() if with_sinks else None
    out, lse, mass = run(w, 0, sinks)
    assert (out == 0).all() and (mass == 0).all()
    if with_sinks:
        assert torch.allclose(lse, sinks.expand_as(lse), rtol=1e-6, atol=1e-6)
    else:
        assert (lse == -math.inf).all()


@pytest.mark.parametrize("q_lens,kv_lens,heads,kv,dim,page,dt", [
    ([1, 1, 1], [700, 5, 64], 8, 2, 128, 16, BF),      # single tokens
    ([1, 2], [9000, 4000], 8, 2, 64, 16, HF),
    ([70, 3, 0, 20], [400, 500, 9, 20], 8, 2, 64, 16, HF),  # chunks: whole items
    ([600, 90], [4000, 300], 12, 4, 128, 32, BF),      # joined parts
    ([30], [33], 17, 1, 128, 16, BF),                  # rows of a tile unused
])
@pytest.mark.parametrize("mass", [False, True])
def test_output_over_the_queries(q_lens, kv_lens, heads, kv, dim, page, dt, mass):
    """`out` may be the queries themselves, as a view of a wider projection too."""
    w = World(q_lens, kv_lens, heads, kv, dim, page, dt, seed=heads, slack=1)
    want = run(w, mass=mass)
    q = w.q._base.clone()[:, 1:heads + 1]  # w.q is a slice of a wider array
    assert q.stride() == w.q.stride()
    got = run(w, mass=mass, q=q, out=q)
    assert torch.equal(got[0][:w.cu[-1]], want[0][:w.cu[-1]]) and torch.equal(got[1], want[1])
    assert torch.equal(got[0][w.cu[-1]:], w.q[w.cu[-1]:])  # a row of no sequence stays
    assert not mass or torch.equal(got[2], want[2])


def test_calls_of_one_batch_from_two_threads_do_not_share_a_workspace_at_once(monkeypatch):
    """Two host threads that use one batch on one stream: the launches of a call, which share its workspace, may not come between
    another's. The library's call is a stand-in that waits; nothing is launched."""
    import threading
    import time

    from expert_slot_cache_device_gb300 import ftmoe as F

    w = World([1, 90], [4000, 800], 12, 2, 128, 16, BF, seed=3)
    inside, clashes = {}, []

    def call(*args):
        ws = args[-3]
        assert ws
        if inside.get(ws):
            clashes.append(ws)
        inside[ws] = inside.get(ws, 0) + 1
        time.sleep(0.02)
        inside[ws] -= 1

    monkeypatch.setattr(F, "ftmoe_paged_attention", call)
    threads = [threading.Thread(target=lambda: [w.cache.attend(w.batch, w.q) for _ in range(5)]) for _ in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not clashes


def test_attention_of_one_batch_from_two_threads():
    """Calls of one batch from several threads on the default stream, with and without mass, give what each gives alone."""
    import threading

    w = World([1, 90, 5], [4000, 800, 2600], 12, 2, 128, 16, BF, seed=5)
    want, _, mass = run(w)
    outs = [[torch.empty_like(want) for _ in range(20)] for _ in range(4)]
    sums = [[torch.zeros_like(mass) for _ in range(20)] for _ in range(4)]
    torch.cuda.synchronize()

    def work(k):
        for i in range(20):
            w.cache.attend(w.batch, w.q, out=outs[k][i], mass=sums[k][i] if (i + k) % 2 else None)

    threads = [threading.Thread(target=work, args=(k,)) for k in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for k in range(4):
        for i in range(20):
            assert torch.equal(outs[k][i], want), (k, i)
            assert not (i + k) % 2 or torch.equal(sums[k][i], mass), (k, i)


def test_a_batch_keeps_no_large_workspace():
    """Kept scores of long caches go back to the allocator after the call (their call takes far longer than the allocation)."""
    n = 70000
    w = World([1] * 16, [n] + [40] * 14 + [3000], 64, 4, 64, 16, BF, seed=6)
    w.cache.attend(w.batch, w.q)
    small = sum(t.numel() for t in w.batch._spaces.values())
    before = torch.cuda.memory_allocated()
    mass = torch.zeros((16, 4, n), device="cuda")
    for _ in range(2):
        out, _, mass = run(w)
        torch.cuda.synchronize()
    assert sum(t.numel() for t in w.batch._spaces.values()) == small <= 256 << 20
    del out
    assert torch.cuda.memory_allocated() - before <= 4 * mass.numel() + (1 << 20)
    check_attend(w, 0, None, True)


def _calls(w):
    """Every call that a cache, and 4-bit weights, take, by name."""
    from expert_slot_cache_device_gb300.kv_cache import Rotary
    from expert_slot_cache_device_gb300.w4 import W4Weights

    k, v = (torch.zeros((w.tokens, w.kv_heads, w.dim), dtype=w.dtype, device="cuda") for _ in range(2))
    pos = torch.zeros(w.tokens, dtype=torch.int32, device="cuda")
    rotary, mass = Rotary(w.dim), torch.zeros((1, w.kv_heads, 64), device="cuda")
    table = torch.tensor([[0, 0, 0, 0]], dtype=torch.int32, device="cuda")
    codes, scales = torch.zeros((16, 64), dtype=torch.uint8, device="cuda"), torch.zeros((16, 1), dtype=BF, device="cuda")
    weights, x = W4Weights(codes, scales), torch.zeros((2, 128), dtype=BF, device="cuda")
    return {"append": lambda: w.cache.append(w.batch, rotary, w.q, k, v, pos), "attend": lambda: w.cache.attend(w.batch, w.q),
            "evict": lambda: w.cache.evict(w.batch, mass, table, 64, 1), "pack": lambda: W4Weights(codes, scales),
            "matvec": lambda: weights.matvec(x)}, weights


def test_calls_with_another_device_current_are_refused(monkeypatch):
    """Kernels go to the current device: a call on memory of another one is refused before anything is enqueued."""
    from expert_slot_cache_device_gb300 import kv_cache

    calls, _ = _calls(World([1], [20], 4, 2, 64, 16, BF))
    for call in calls.values():
        call()
    monkeypatch.setattr(kv_cache, "_current_device", lambda: 1, raising=False)
    for name, call in calls.items():
        with pytest.raises(ValueError, match="device"):
            call()
            pytest.fail(name)


def test_tensors_of_another_device_are_refused():
    """A cache and weights that say they are elsewhere than the arguments."""
    w = World([1], [20], 4, 2, 64, 16, BF)
    calls, weights = _calls(w)
    w.cache._dev = weights._dev = 1
    for name in ("append", "attend", "evict", "matvec"):
        with pytest.raises(ValueError):
            calls[name]()
            pytest.fail(name)


PROBE = r"""
#include "kv_tc05.cuh"
using namespace ftmoe::kv;
__global__ void probe(AttendParams p, Seq s, const long long *at, int n, long long *units, int4 *places) {
    const int n_qt = row_tiles(p, s);
    const long long per = seq_units(p, s, n_qt);
    if (threadIdx.x == 0) *units = per;
    for (int i = 0; i < n; i++) {
        const Place x = place_of(p, s, n_qt, per, at[i]);
        if (threadIdx.x == 0) places[i] = make_int4(x.hk, x.qt, x.at, 0);
    }
}
extern "C" int place(int group, int window, int causal, int q_len, int kv_len, const long long *at, int n, long long *units, int4 *places) {
    AttendParams p{};
    p.group = group, p.window = window, p.causal = causal, p.item_tokens = 2 * (128 / group);
    Seq s{0, q_len, kv_len};
    probe<<<1, 32>>>(p, s, at, n, units, places);
    return (int)cudaDeviceSynchronize();
}
"""


@pytest.fixture(scope="module")
def place(tmp_path_factory):
    import ctypes
    import subprocess

    from expert_slot_cache_device_gb300 import build as B

    d = tmp_path_factory.mktemp("line")
    src, lib = d / "probe.cu", d / "probe.so"
    src.write_text(PROBE)
    subprocess.run([B.nvcc(), *B.NVCC_FLAGS, "-shared", "-o", str(lib), str(src)], check=True)
    f = ctypes.CDLL(str(lib)).place
    f.argtypes = [ctypes.c_int] * 5 + [ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p]
    return f


@pytest.mark.parametrize("group,window,causal,q_len,kv_len,heads", [
    (4, 0, 1, 1000, 4000, 2),
    (17, 300, 1, 70, 5000, 3),
    (1, 0, 0, 600, 129, 1),
    (128, 0, 1, 1 << 20, 1 << 20, 1),          # 2^31 steps and some in one sequence and head
    (8, 0, 1, 1 << 21, 1 << 21, 8),            # 2^32 and some in its eight heads
    (128, 1 << 20, 1, 700001, (1 << 30) - 5, 2),
    (128, 0, 0, 513, 1 << 30, 4),              # few items of 2^23 steps
])
def test_places_on_a_line_longer_than_32_bits(place, group, window, causal, q_len, kv_len, heads):
    """The arithmetic that cuts the chunk kernel's work, at its places in long prompts (no attention is computed)."""
    import numpy as np

    t = 2 * (128 // group)
    n = -(-q_len // t)
    i0 = np.arange(n, dtype=np.int64) * t
    i1 = np.minimum(i0 + t, q_len)
    first = kv_len - q_len
    hi = np.maximum(first + i1, 0) if causal else np.where(first + i1 > 0, kv_len, 0)
    lo = np.maximum(first + i0 - window + 1, 0) if window else np.zeros_like(i0)
    lo = np.minimum(lo, hi) // 128 * 128
    units = np.maximum(-(-(hi - lo) // 128), 1) + 2  # an item's start and end count as two steps
    ends = np.cumsum(units)
    per = int(ends[-1])
    rng = np.random.default_rng(q_len)
    at = np.concatenate([rng.integers(0, per * heads, 40), [0, per - 1, per, per * heads - 1] if heads > 1 else [0, per - 1]])
    d_at = torch.from_numpy(at).cuda()
    d_units, d_places = torch.zeros(1, dtype=torch.int64, device="cuda"), torch.zeros((len(at), 4), dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    assert place(group, window, causal, q_len, kv_len, d_at.data_ptr(), len(at), d_units.data_ptr(), d_places.data_ptr()) == 0
    assert int(d_units) == per
    qt = np.searchsorted(ends, at % per, side="right")
    want = np.stack([at // per, qt, at % per - (ends - units)[qt]], 1)
    assert (d_places[:, :3].cpu().numpy() == want).all()


def test_append_of_no_tokens_returns_its_output():
    from expert_slot_cache_device_gb300.kv_cache import Rotary

    w = World([0], [5], 4, 2, 64, 16, BF)
    q, k = (torch.empty((0, h, 64), dtype=BF, device="cuda") for h in (4, 2))
    pos, out = torch.empty(0, dtype=torch.int32, device="cuda"), torch.empty_like(q)
    assert w.cache.append(w.batch, Rotary(64), q, k, k, pos, q_out=out) is out
    assert w.cache.append(w.batch, Rotary(64), q, k, k, pos).shape == q.shape
    assert w.cache.append(w.batch, Rotary(64), None, k, k, pos) is None


def test_bounds_past_32_bits_are_refused():
    """Host integers that the C views' 32 bits would cut: a bound of 2^32 would have become no token at all."""
    from expert_slot_cache_device_gb300.kv_cache import KVBatch

    w = World([1], [40], 4, 2, 64, 16, BF)
    for q, n in ((2 ** 32, 40), (2 ** 31, 40), (1, 2 ** 32 + 40), (1, 2 ** 31)):
        with pytest.raises(ValueError):
            KVBatch(w.batch.block_table, w.batch.kv_lens, w.batch.cu_q, q, n)
    mass, table = torch.zeros((1, 2, 40), device="cuda"), torch.zeros((1, 4), dtype=torch.int32, device="cuda")
    for budget, recent in ((2 ** 32 + 8, 4), (8, 2 ** 32 + 4)):
        with pytest.raises(ValueError):
            w.cache.evict(w.batch, mass, table, budget, recent, kept=torch.zeros((1, 2, 8), dtype=torch.int32, device="cuda"),
                          new_mass=torch.zeros((1, 2, 8), device="cuda"))


@pytest.mark.parametrize("layout", ["pages", "slots", "heads"])
@pytest.mark.parametrize("q_lens,kv_lens", [([1, 1], [300, 17]), ([60, 2], [300, 17])])
def test_keys_and_values_in_one_allocation(layout, q_lens, kv_lens):
    """K and V as two halves of a page, of a slot or of a head: written, read and moved through their strides."""
    from expert_slot_cache_device_gb300.kv_cache import PagedKVCache, Rotary

    w = World(q_lens, kv_lens, 8, 2, 64, 16, BF, seed=14)
    pages = w.cache.num_pages + 2
    shape, at = {"pages": ((pages, 2, 16, 2, 64), 1), "slots": ((pages, 16, 2, 2, 64), 2), "heads": ((pages, 16, 2, 2, 64), 3)}[layout]
    both = torch.zeros(shape, dtype=BF, device="cuda")
    k, v = both.select(at, 0), both.select(at, 1)
    k[:w.cache.num_pages], v[:w.cache.num_pages] = w.cache.k_pages, w.cache.v_pages
    cache = PagedKVCache(pages, 16, 2, 64, BF, k_pages=k, v_pages=v)
    apart, w.cache = w.cache, cache
    check_attend(w, 0, None, True)
    new_k, new_v = (torch.randn((w.tokens, 2, 64), generator=w.gen).to(BF).cuda() for _ in range(2))
    pos = torch.arange(w.tokens, dtype=torch.int32, device="cuda")
    got = [c.append(w.batch, Rotary(64), w.q, new_k, new_v, pos) for c in (cache, apart)]
    assert torch.equal(*got)
    for a, b in ((k, apart.k_pages), (v, apart.v_pages)):
        assert torch.equal(a[:-2].nan_to_num(9.0), b.nan_to_num(9.0))
    mass = torch.rand((2, 2, 300), device="cuda")
    table = torch.tensor([[pages - 2], [pages - 1]], dtype=torch.int32, device="cuda")
    kept, _, _ = cache.evict(w.batch, mass, table, 16, 3)
    for i in range(2):
        p, r = ref.cells(w.table[i], 16, kv_lens[i])
        for h in range(2):
            j = kept[i, h].cpu().long()
            assert torch.equal(k[pages - 2 + i, :, h], k[p[j], r[j], h]) and torch.equal(v[pages - 2 + i, :, h], v[p[j], r[j], h])
    assert cache.status() == 0


@pytest.mark.parametrize("q_lens,kv_lens,short", [([1, 1, 1], [5000, 17, 450], [300, 1, 449]), ([90, 1, 30], [2000, 17, 450], [700, 1, 449])])
def test_captured_calls_with_mass(q_lens, kv_lens, short):
    """Single tokens and chunks with mass in a graph, with another call of the batch after its capture: replays follow the
    lengths and have workspaces of their own."""
    w = World(q_lens, kv_lens, 8, 2, 64, 16, BF, seed=15)
    n = max(kv_lens)
    out, mass = torch.empty_like(w.q, memory_format=torch.contiguous_format), torch.zeros((3, 2, n), device="cuda")
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        w.cache.attend(w.batch, w.q, out=out, mass=mass)
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            w.cache.attend(w.batch, w.q, out=out, mass=mass)
    w.batch.kv_lens.copy_(torch.tensor(short, dtype=torch.int32))
    want, _, want_mass = run(w)
    for _ in range(2):
        out.zero_(), mass.zero_()
        graph.replay()
        w.cache.attend(w.batch, w.q, mass=torch.zeros_like(mass))
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(mass, want_mass)
    for i, m in enumerate(short):
        part = slice(w.cu[i], w.cu[i + 1])
        o, _, _, ot, _, _ = ref.attention(w.q[part].cpu(), w.k_seq[i][:m], w.v_seq[i][:m], 64 ** -0.5, 0, True, None)
        assert ((out[part].double().cpu() - o).abs() <= ot).all()


@pytest.mark.parametrize("q,n,heads,kv,dim", [(1, 1, 4, 2, 64), (1, 200, 8, 2, 128), (1, 9000, 16, 1, 64), (4, 300, 4, 2, 64),
                                              (40, 300, 4, 2, 64), (300, 2000, 8, 2, 128)])
def test_a_nan_that_a_row_sees_reaches_its_results(q, n, heads, kv, dim):
    """Sixteen keys of one head are NaN: output and log-sum-exp of the rows that see them are too, the other head's and the other
    sequence's rows are not."""
    w = World([q, q], [n, n], heads, kv, dim, 16, BF, seed=q + n)
    at = min(16, n - 1) if q == 1 else n - 2 * q if n > 2 * q else 0
    p, r = ref.cells(w.table[0], 16, n)
    bad = slice(at, min(at + 16, n - q + 1))  # every row sees these
    w.cache.k_pages[p[bad], r[bad], 0] = math.nan
    out, lse, mass = run(w)
    per = heads // kv
    assert torch.isnan(out[:q, :per]).all() and torch.isnan(lse[:q, :per]).all()
    assert torch.isnan(mass[0, 0, :n]).all()
    assert torch.isfinite(out[q:]).all() and torch.isfinite(lse[q:]).all() and torch.isfinite(mass[1]).all()
    assert torch.isfinite(out[:q, per:]).all() and torch.isfinite(lse[:q, per:]).all() and torch.isfinite(mass[0, 1:]).all()
