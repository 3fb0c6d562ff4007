"""Latent attention where it can go wrong without a plain shape showing it: many sequences, many blocks of heads, powers of two at
the ends of their range, NaN that rows see, offsets past 32 bits, calls at the same time, other devices. Tolerances as in
tests/latent_reference.py."""
import math
import threading
import time

import pytest
import torch

import attention_reference as ref
import latent_reference as lref
from test_gpu_latent import BF, HF, World, check_attend, check_expand, check_rows, expand_world, ints, starts

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from expert_slot_cache_device_gb300 import build

    build.build()


@pytest.mark.parametrize("q_lens,kv_lens,heads,latent,page,dt,bits", [
    ([1] * 700, [(29 * i) % 200 for i in range(700)], 2, 128, 16, BF, 16),          # more sequences than threads
    ([1] * 1100, [(17 * i) % 140 for i in range(1100)], 1, 128, 16, HF, 8),
    ([1 + 3 * (i % 2) for i in range(280)], [5 + (41 * i) % 250 for i in range(280)], 40, 128, 32, BF, 16),  # several items each
    ([i % 23 for i in range(520)], [(19 * i) % 160 for i in range(520)], 33, 128, 16, BF, 8),
    ([90, 0, 41, 3], [300, 77, 41, 500], 48, 256, 64, BF, 16),                      # an item a token, more than a lane counts
    ([1, 1], [6000, 200], 96, 384, 64, HF, 8),                                      # three blocks of heads
    ([1, 3], [2500, 700], 130, 384, 128, BF, 8),                                    # five
    ([1, 2], [900, 40], 200, 512, 16, BF, 16),                                      # four: pairs of blocks
    ([2, 1], [90, 1500], 600, 128, 256, HF, 16),
    ([1], [40000], 128, 512, 64, BF, 8),                                            # one sequence over all SMs
    ([1] * 100, [(67 * i) % 640 for i in range(100)], 16, 256, 64, BF, 16),         # whole items of several steps
    ([1] * 60, [300 + (89 * i) % 400 for i in range(60)], 128, 256, 32, HF, 16),    # pairs of them
    ([1] * 250, [(31 * i) % 513 for i in range(250)], 32, 128, 16, BF, 8),          # two waves
    ([2] * 70, [2 + (57 * i) % 500 for i in range(70)], 130, 128, 16, BF, 16),
])
def test_attend_plans(q_lens, kv_lens, heads, latent, page, dt, bits):
    check_attend(World(q_lens, kv_lens, latent, 32, page, dt, bits, seed=heads), heads)


def test_loose_bounds():
    """Bounds far above the lengths (2^31 - 1 new tokens, 2^30 slots where the table allows them) only cost time."""
    from expert_slot_cache_device_gb300.kv_cache import KVBatch
    from expert_slot_cache_device_gb300.latent_cache import ExpandedBatch

    w = World([3, 1], [300, 64], 256, 32, 16, BF, 16, seed=7)
    w.batch = KVBatch(w.table.cuda(), ints(w.kv_lens), ints(w.cu), max_q=2 ** 31 - 1, max_kv=w.table.shape[1] * 16)
    check_attend(w, 20)
    b, q, k, key, v, cu_q, cu_kv = expand_world([30, 200], [500, 200], 2, 64, 32, BF)
    b = ExpandedBatch(ints(cu_q), ints(cu_kv), 2 ** 31 - 1, 2 ** 30)
    out = b.attend(q, k, key, v)
    assert b.status() == 0
    for i in range(2):
        t, r = slice(cu_q[i], cu_q[i + 1]), slice(cu_kv[i], cu_kv[i + 1])
        o, _, ot, _ = lref.expanded(q[t].cpu(), k[r].cpu(), key[r].cpu(), v[r].cpu(), 96 ** -0.5, True)
        check_rows(i, out[t], o, ot, None, None, None)


@pytest.mark.parametrize("bits", [16, 8])
def test_nothing_cached(bits):
    w = World([1, 2, 0], [0, 0, 0], 256, 32, 16, BF, bits)
    out, lse = check_attend(w, 70)
    assert (out == 0).all() and (lse == -math.inf).all()
    rows = torch.full((4, 288), 7.0, dtype=BF, device="cuda")
    w.cache.read(w.batch, ints([0, 0, 0, 0]), out=rows)
    assert w.cache.status() == 0 and (rows == 7).all()


@pytest.mark.parametrize("q_lens,kv_lens,heads", [([5] * 450, [3 + (23 * i) % 120 for i in range(450)], 1),
                                                  ([i % 7 for i in range(900)], [(11 * i) % 90 for i in range(900)], 2),
                                                  ([5000], [5000], 1), ([4200, 300], [4300, 400], 2),
                                                  ([100, 256, 7], [700, 1000, 500], 40), ([200] * 9, [1100, 200, 900, 201, 345, 600, 777, 1024, 1023], 16)])
def test_expand_plans(q_lens, kv_lens, heads):
    check_expand(q_lens, kv_lens, heads, 64, 16, BF, seed=heads)


def test_expand_without_rows():
    from expert_slot_cache_device_gb300.latent_cache import ExpandedBatch

    b = ExpandedBatch(ints([0, 3]), ints([0, 0]), 3, 0)
    q, none = torch.randn((3, 2, 96), device="cuda").to(BF), torch.empty((0, 2, 64), dtype=BF, device="cuda")
    lse = torch.full((3, 2), 7.0, device="cuda")
    out = b.attend(q, none, torch.empty((0, 32), dtype=BF, device="cuda"), none, out=torch.full((3, 2, 64), math.nan, dtype=BF, device="cuda"), lse=lse)
    assert b.status() == 0 and (out == 0).all() and (lse == -math.inf).all()


def refill(w, i, c):
    """Sequence i's latents, as its cache holds them."""
    n = len(c)
    if w.bits == 16:
        rows = torch.cat([c, w.key[i]], 1).view(torch.uint8)
    else:
        codes, powers, _ = lref.encode(c)
        c, rows = lref.decode(codes, powers, w.dtype).to(w.dtype), lref.pack(codes, powers, w.key[i])
    p, r = ref.cells(w.table[i], w.page, n)
    w.raw[p.cuda(), r.cuda(), :rows.shape[1]] = rows.cuda()
    w.c[i] = c


@pytest.mark.parametrize("dt,sizes", [(BF, (-120, -100, -30, 20, 60)), (HF, (-24, -16, -9, 3, 14))])
def test_powers_of_two_of_every_size(dt, sizes):
    """Groups of one slot have powers far apart, at both ends of what the type holds: products by bits and by floats, in one tile."""
    w = World([1, 2], [300, 70], 256, 32, 16, dt, 8, seed=2)
    for i, n in enumerate(w.kv_lens):
        e = torch.tensor(sizes, dtype=torch.float64)[torch.randint(0, len(sizes), (n, 8), generator=w.gen)]
        if i:
            e[:] = torch.tensor(sizes[:1], dtype=torch.float64)
        size = torch.exp2(e).repeat_interleave(32, 1)
        refill(w, i, (torch.randn((n, 256), generator=w.gen).double() * size).clamp(-60000 if dt == HF else -1e38, 60000 if dt == HF else 1e38).to(dt))
    # scores of about 1: the largest size decides
    check_attend(w, 20, scale=2.0 ** -(sizes[-1] + 5))
    rows = w.cache.read(w.batch, ints(starts(w.kv_lens)), rows=370)
    assert torch.equal(rows[:, :256].cpu(), torch.cat(w.c))


@pytest.mark.parametrize("q,n,heads,bits", [(1, 1, 4, 16), (1, 200, 20, 8), (1, 9000, 128, 16), (1, 700, 32, 8), (4, 300, 40, 16), (40, 300, 5, 8)])
@pytest.mark.parametrize("part", ["latent", "rope"])
def test_a_nan_that_a_row_sees_reaches_its_results(q, n, heads, bits, part):
    w = World([q, q], [n, n], 256, 32, 16, BF, bits, seed=q + n)
    at = min(16, n - 1) if q == 1 else n - 2 * q if n > 2 * q else 0
    p, r = ref.cells(w.table[0], 16, n)
    bad = slice(at, min(at + 16, n - q + 1))  # every row sees these
    row = lref.row_bytes(256, 32, bits)
    where = slice(row - 64, row) if part == "rope" else slice(0, row - 64)
    w.raw[p[bad].cuda(), r[bad].cuda(), where] = 255  # NaN in 16 bits; of codes, power 255 is
    qv, qr = w.queries(heads)
    lse = torch.zeros((2 * q, heads), device="cuda")
    out = w.cache.attend(w.batch, qv, qr, 0.06, lse=lse)
    assert torch.isnan(out[:q]).all() and torch.isnan(lse[:q]).all()
    assert torch.isfinite(out[q:]).all() and torch.isfinite(lse[q:]).all()


@pytest.mark.parametrize("q,n,heads", [(1, 1, 1), (30, 400, 2), (300, 2000, 3), (2, 9000, 1)])
@pytest.mark.parametrize("part", ["k", "key", "v"])
def test_a_nan_row_reaches_expanded_results(q, n, heads, part):
    b, qx, k, key, v, cu_q, cu_kv = expand_world([q, q], [n, n], heads, 64, 32, BF, seed=n)
    at = max(n - 2 * q, 0)
    {"k": k, "key": key, "v": v}[part][at] = math.nan
    lse = torch.zeros((2 * q + 1, heads), device="cuda")
    out = b.attend(qx, k, key, v, lse=lse)
    assert torch.isnan(out[:q]).all() and torch.isfinite(out[q:2 * q]).all() and torch.isfinite(lse[q:2 * q]).all()
    assert torch.isnan(lse[:q]).all() if part != "v" else torch.isfinite(lse[:q]).all()


@pytest.mark.parametrize("bits", [16, 8])
def test_long_cache_offsets_past_32_bits(bits):
    """Pages whose offsets do not fit 32 bits are written, read back and read by attention."""
    from expert_slot_cache_device_gb300.kv_cache import KVBatch, Rotary
    from expert_slot_cache_device_gb300.latent_cache import LatentCache

    page, latent, rope, n = 256, 512, 64, 300
    row = lref.row_bytes(latent, rope, bits)
    pages = (1 << 32) // (page * row // (2 if bits == 16 else 1)) + 3  # 2^32 elements, or bytes, and some
    cache = LatentCache(pages, page, latent, rope, BF, bits)
    g = torch.Generator().manual_seed(0)
    use = [pages - 1, 0]
    cache.pages[use[0]] = cache.pages[use[1]] = 0
    table, c = ints([use]), torch.randn((n, latent), generator=g).to(BF)
    key, pos = torch.randn((n, rope), generator=g).to(BF), torch.arange(n, dtype=torch.int32)
    batch = KVBatch(table, ints([n]), ints([0, n]), n, n)
    cache.append(batch, Rotary(rope), c.cuda(), key.cuda(), pos.cuda())
    rows = cache.read(batch, ints([0, n]), rows=n).cpu()
    want = c if bits == 16 else lref.decode(*lref.encode(c)[:2], BF).to(BF)
    assert torch.equal(rows[:, :latent], want)
    for q_len in (1, 40):
        b = KVBatch(table, ints([n]), ints([0, q_len]), q_len, n)
        q, qr = torch.randn((q_len, 16, latent), generator=g).to(BF), torch.randn((q_len, 16, rope), generator=g).to(BF)
        out = cache.attend(b, q.cuda(), qr.cuda(), 0.07)
        o, _, ot, _ = lref.absorbed(q, qr, rows[:, :latent], rows[:, latent:], 0.07, True)
        assert cache.status() == 0 and ((out.double().cpu() - o).abs() <= ot).all()


def test_expanded_rows_past_32_bits():
    """Keys, values, queries and outputs whose row strides put them past 2^32 elements."""
    from expert_slot_cache_device_gb300.latent_cache import ExpandedBatch

    n, heads, step = 300, 2, 1 << 24
    g = torch.Generator().manual_seed(1)
    big = torch.empty(n * step, dtype=BF, device="cuda")  # 10 GB: all four in one row's length
    take = lambda at, *s: big.as_strided((n, *s), (step, s[-1], 1) if len(s) == 2 else (step, 1), at)  # noqa: E731
    q, k, v, key, out = take(0, heads, 96), take(1024, heads, 64), take(2048, heads, 64), take(4096, 32), take(8192, heads, 64)
    for t in (q, k, v, key):
        t.copy_(torch.randn(t.shape, generator=g).to(BF))
    b = ExpandedBatch(ints([0, n]), ints([0, n]), n, n)
    lse = torch.zeros((n, heads), device="cuda")
    b.attend(q, k, key, v, out=out, lse=lse)
    o, z, ot, zt = lref.expanded(q.cpu(), k.cpu(), key.cpu(), v.cpu(), 96 ** -0.5, True)
    check_rows(0, out, o, ot, lse, z, zt)


def test_calls_repeat_bit_for_bit_and_on_two_streams_at_once():
    for bits, heads in ((16, 16), (16, 128), (8, 32)):
        w = World([1] * 6, [5000, 4000, 70, 1, 2600, 300], 512, 64, 64, BF, bits, seed=heads)
        q, qr = w.queries(heads)
        want = w.cache.attend(w.batch, q, qr, 0.07).clone()
        b, qx, k, key, v, cu, _ = expand_world([30, 300], [3000, 900], 2, 128, 64, BF)
        wide = b.attend(qx, k, key, v)[:cu[-1]].clone()
        torch.cuda.synchronize()
        sides, got = [torch.cuda.Stream(), torch.cuda.Stream()], []
        for _ in range(12):
            for s in sides:
                with torch.cuda.stream(s):
                    got.append((w.cache.attend(w.batch, q, qr, 0.07), b.attend(qx, k, key, v)))
        torch.cuda.synchronize()
        assert all(torch.equal(x, want) and torch.equal(y[:cu[-1]], wide) for x, y in got)


def test_one_batch_from_several_threads():
    w = World([1, 9, 5], [4000, 800, 2600], 256, 64, 16, BF, 16, seed=5)
    q, qr = w.queries(12)
    want = w.cache.attend(w.batch, q, qr, 0.07).clone()
    b, qx, k, key, v, cu, _ = expand_world([30, 300], [3000, 900], 2, 64, 64, BF)
    wide = b.attend(qx, k, key, v)[:cu[-1]].clone()
    outs = [[(torch.empty_like(want), torch.empty((qx.shape[0], 2, 64), dtype=BF, device="cuda")) for _ in range(15)] for _ in range(4)]
    torch.cuda.synchronize()

    def work(i):
        for o, x in outs[i]:
            w.cache.attend(w.batch, q, qr, 0.07, out=o)
            b.attend(qx, k, key, v, out=x)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) and torch.equal(x[:cu[-1]], wide) for part in outs for o, x in part)


def test_calls_of_one_batch_from_two_threads_do_not_share_a_workspace_at_once(monkeypatch):
    """The library's calls are a stand-in that waits; nothing is launched."""
    from expert_slot_cache_device_gb300 import ftmoe as F

    w = World([1, 1], [4000, 800], 256, 32, 16, BF, 16, seed=3)
    q, qr = w.queries(12)
    b, qx, k, key, v, *_ = expand_world([30, 300], [3000, 900], 2, 64, 64, BF)
    inside, clashes = {}, []

    def call(*args):
        ws = args[-3]
        assert ws
        if inside.get(ws):
            clashes.append(ws)
        inside[ws] = inside.get(ws, 0) + 1
        time.sleep(0.02)
        inside[ws] -= 1

    monkeypatch.setattr(F, "ftmoe_latent_attention", call)
    monkeypatch.setattr(F, "ftmoe_expanded_attention", call)
    for one in (lambda: w.cache.attend(w.batch, q, qr, 0.1), lambda: b.attend(qx, k, key, v)):
        threads = [threading.Thread(target=lambda: [one() for _ in range(4)]) for _ in range(3)]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
    assert not clashes


def _calls(w):
    from expert_slot_cache_device_gb300.kv_cache import Rotary

    c, key = (torch.zeros((w.tokens, d), dtype=w.dtype, device="cuda") for d in (w.latent, w.rope))
    pos, rotary = torch.zeros(w.tokens, dtype=torch.int32, device="cuda"), Rotary(w.rope)
    q, qr = w.queries(4)
    b, qx, k, kr, v, *_ = expand_world([3], [20], 2, 64, 32, BF)
    n = sum(w.kv_lens)
    return {"append": lambda: w.cache.append(w.batch, rotary, c, key, pos), "attend": lambda: w.cache.attend(w.batch, q, qr, 0.1),
            "read": lambda: w.cache.read(w.batch, ints(starts(w.kv_lens)), rows=n), "expand": lambda: b.attend(qx, k, kr, v)}, b


def test_calls_with_another_device_current_are_refused(monkeypatch):
    from expert_slot_cache_device_gb300 import kv_cache

    calls, _ = _calls(World([1], [20], 256, 32))
    for call in calls.values():
        call()
    monkeypatch.setattr(kv_cache, "_current_device", lambda: 1, raising=False)
    for name, call in calls.items():
        with pytest.raises(ValueError, match="device"):
            call()
            pytest.fail(name)


def test_tensors_of_another_device_are_refused():
    w = World([1], [20], 256, 32)
    calls, b = _calls(w)
    w.cache._dev = b._dev = 1
    for name, call in calls.items():
        with pytest.raises(ValueError):
            call()
            pytest.fail(name)


def test_captured_writes_follow_their_device_arrays():
    """A captured append and read, replayed with other lengths, tables and positions."""
    from expert_slot_cache_device_gb300.kv_cache import Rotary

    for bits in (16, 8):
        w = World([1, 1], [20, 33], 256, 32, 16, BF, bits, seed=8)
        rotary, g = Rotary(32), w.gen
        c, key = torch.randn((2, 256), generator=g).to(BF).cuda(), torch.randn((2, 32), generator=g).to(BF).cuda()
        pos, cu = ints([19, 32]), ints([0, 20, 53])
        rows = torch.zeros((80, 288), dtype=BF, device="cuda")
        w.cache.append(w.batch, rotary, c, key, pos)
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            side.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                w.cache.append(w.batch, rotary, c, key, pos)
                w.cache.read(w.batch, cu, out=rows)
        for lens in ([20, 33], [7, 16], [12, 1]):
            c.normal_(generator=torch.Generator("cuda").manual_seed(lens[0]))
            w.batch.kv_lens.copy_(ints(lens))
            pos.copy_(ints([n - 1 for n in lens]))
            cu.copy_(ints(starts(lens)))
            graph.replay()
            torch.cuda.synchronize()
            got = rows[[lens[0] - 1, sum(lens) - 1], :256].cpu()
            want = c.cpu() if bits == 16 else lref.decode(*lref.encode(c.cpu())[:2], BF).to(BF)
            assert w.cache.status() == 0 and torch.equal(got, want)
            assert torch.equal(rows[:lens[0] - 1, :256].cpu(), w.c[0][:lens[0] - 1])
            for i in range(2):
                w.c[i][lens[i] - 1] = want[i]  # stays for the next


def test_positions_and_slots_of_one_page_twice():
    """Two sequences may share the pages of a common start; each writes its own last page."""
    w = World([0, 0], [48, 48], 256, 32, 16, BF, 16, seed=1)
    w.table[1, :2] = w.table[0, :2]
    from expert_slot_cache_device_gb300.kv_cache import KVBatch

    b = KVBatch(w.table.cuda(), ints([48, 48]), ints([0, 1, 2]), 1, 48)
    for i in range(2):
        w.c[i], w.key[i] = (torch.cat([x[0][:32], x[i][32:]]) for x in (w.c, w.key))
    q, qr = torch.randn((2, 8, 256), generator=w.gen).to(BF), torch.randn((2, 8, 32), generator=w.gen).to(BF)
    out = w.cache.attend(b, q.cuda(), qr.cuda(), 0.08)
    for i in range(2):
        o, _, ot, _ = lref.absorbed(q[i:i + 1], qr[i:i + 1], w.c[i], w.key[i], 0.08, True)
        assert ((out[i:i + 1].double().cpu() - o).abs() <= ot).all()
