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


# ---------------------------------------------------------------- what lies beside a sequence's rows and slots
@pytest.mark.parametrize("nope,rope", [(128, 64), (64, 32)])
@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("lens,cut", [([70, 40, 33, 130], False), ([1, 250, 129, 90], False), ([1500, 700, 260, 1900], True), ([127, 1, 2, 1250], True)])
def test_expanded_rows_beside_a_sequence_hold_nan(nope, rope, dt, lens, cut):
    """A step reads 128 rows, past the sequence's last one into the next one's: there are NaN in keys, rotary parts and
    values, in a sequence without new tokens and in one whose own results are NaN for it."""
    from expert_slot_cache_device_gb300 import ftmoe as F

    q_lens, heads = [min(lens[0], 9), 0, 2, min(lens[3], 140)], 2
    b, q, k, key, v, cu_q, cu_kv = expand_world(q_lens, lens, heads, nope, rope, dt, seed=sum(lens))
    for t in (k, key, v):
        t[cu_kv[1]:cu_kv[2]] = math.nan  # no token sees these
        t[cu_kv[2]] = math.nan           # the first row of the third sequence, which its tokens see
    need = F.ftmoe_expanded_attention_workspace_bytes(b._ref(q.shape[0], k.shape[0]), F.DT_BF16, heads, nope, rope, nope, True)
    assert (need > 0) == cut  # parts that are joined, or none
    for causal in (True, False):
        out = torch.full((q.shape[0], heads, nope), 7.0, dtype=dt, device="cuda")
        lse = torch.full((q.shape[0], heads), 7.0, device="cuda")
        b.attend(q, k, key, v, causal=causal, out=out, lse=lse)
        assert b.status() == 0
        for i in (0, 3):
            t, r = slice(cu_q[i], cu_q[i + 1]), slice(cu_kv[i], cu_kv[i + 1])
            o, z, ot, zt = lref.expanded(q[t].cpu(), k[r].cpu(), key[r].cpu(), v[r].cpu(), (nope + rope) ** -0.5, causal)
            check_rows(i, out[t], o, ot, lse[t], z, zt)
        third = slice(cu_q[2], cu_q[3])
        assert torch.isnan(out[third]).all() and torch.isnan(lse[third]).all()
        assert (out[cu_q[-1]:] == 7).all() and (lse[cu_q[-1]:] == 7).all()


def test_four_operators_captured_and_replayed_with_other_lengths():
    """append, read, both attentions in one graph, replayed twice on two streams with lengths, offsets and inputs of their own."""
    from expert_slot_cache_device_gb300.kv_cache import KVBatch, Rotary, rotary_frequencies
    from expert_slot_cache_device_gb300.latent_cache import ExpandedBatch, LatentCache

    latent, rope, heads, page, most, bits = 256, 32, 12, 16, 700, 16
    table, g = torch.arange(2 * 44, dtype=torch.int32).view(2, 44).cuda(), torch.Generator().manual_seed(21)
    mk = lambda *s: torch.randn(s, generator=g).to(BF)  # noqa: E731
    rotary, (freq, factor) = Rotary(rope), rotary_frequencies(rope)
    side = [torch.cuda.Stream(), torch.cuda.Stream()]

    class Step:
        """A layer's calls over buffers that stay where they are."""

        def __init__(self):
            self.cache = LatentCache(2 * 44, page, latent, rope, BF, bits)
            self.cache.pages.copy_(mk(*self.cache.pages.shape))
            self.lens, self.cu_q, self.cu_rows = ints([most, most]), ints([0, 1, 4]), ints([0, most, 2 * most])
            self.batch = KVBatch(table, self.lens, self.cu_q, 3, most)
            self.wide = ExpandedBatch(self.cu_q, self.cu_rows, 3, most)
            self.c, self.key, self.pos = mk(4, latent).cuda(), mk(4, rope).cuda(), ints([0, 0, 0, 0])
            self.q, self.qr, self.qx = mk(4, heads, latent).cuda(), mk(4, heads, rope).cuda(), mk(4, heads, 64 + rope).cuda()
            self.k, self.v = mk(2 * most, heads, 64).cuda(), mk(2 * most, heads, 64).cuda()
            self.rows = torch.full((2 * most, latent + rope), 7.0, dtype=BF, device="cuda")

        def run(self):
            qr = self.cache.append(self.batch, rotary, self.c, self.key, self.pos, q_rope=self.qr)
            rows = self.cache.read(self.batch, self.cu_rows, out=self.rows)
            lse = torch.empty((4, heads), device="cuda")
            return qr, self.cache.attend(self.batch, self.q, qr, 0.07, lse=lse), lse, self.wide.attend(self.qx, self.k, rows[:, latent:], self.v)

        def check(self, got, lens, cu):
            qr, o, lse, x = got
            assert self.cache.status() == 0 and self.wide.status() == 0
            pages, at = self.cache.pages.cpu(), 0
            turned = ref.rotate(self.key[:, None].cpu(), self.pos.cpu(), freq, factor, rope, "half")[:, 0]
            for i, n in enumerate(lens):
                p, r = ref.cells(table[i].cpu(), page, n)
                have, t, rows = pages[p, r], slice(cu[i], cu[i + 1]), slice(at, at + n)
                new = cu[i + 1] - cu[i]
                assert torch.equal(have[n - new:, :latent], self.c[t].cpu())
                pair = self.key[t].cpu().double().abs().amax(-1, keepdim=True)  # as check_turned of the other tests
                assert ((have[n - new:, latent:].double() - turned[t]).abs() <= ref.U[BF] * turned[t].abs() + pair * 2.0 ** -19 + 2.0 ** -25).all()
                assert torch.equal(self.rows[rows].cpu(), have)
                want = lref.absorbed(self.q[t].cpu(), qr[t].cpu(), have[:, :latent], have[:, latent:], 0.07, True)
                check_rows(i, o[t], want[0], want[2], lse[t], want[1], want[3])
                want = lref.expanded(self.qx[t].cpu(), self.k[rows].cpu(), have[:, latent:], self.v[rows].cpu(), 96 ** -0.5, True)
                check_rows(i, x[t], want[0], want[2], None, None, None)
                at += n

    steps, graphs = [Step(), Step()], []
    for s, st in zip(steps, side):
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            s.run()
            st.synchronize()
            g_ = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g_, stream=st):
                out = s.run()
            graphs.append((g_, out))
    for turn, (lens, cu) in enumerate((([700, 700], [0, 1, 4]), ([300, 33], [0, 3, 4]), ([1, 129], [0, 1, 4]), ([640, 5], [0, 2, 4]))):
        for s in steps:
            s.lens.copy_(ints(lens)), s.cu_q.copy_(ints(cu)), s.cu_rows.copy_(ints(starts(lens)))
            s.c.copy_(mk(4, latent)), s.q.copy_(mk(4, heads, latent)), s.pos.copy_(torch.randint(0, 5000, (4,), generator=g))
        torch.cuda.synchronize()
        for (g_, _), st in zip(graphs, side):
            with torch.cuda.stream(st):
                g_.replay()
        torch.cuda.synchronize()
        for s, (_, out) in zip(steps, graphs):
            s.check(out, lens, cu)


def test_sequences_that_share_their_first_pages_write_their_own():
    """Two sequences have the pages of a common start; each writes a token to its last page, and the common ones stay."""
    from expert_slot_cache_device_gb300.kv_cache import KVBatch, Rotary

    for bits in (16, 8):
        w = World([0, 0], [47, 40], 256, 32, 16, BF, bits, seed=1)
        w.table[1, :2] = w.table[0, :2]
        lens, g = [48, 41], w.gen
        batch = KVBatch(w.table.cuda(), ints(lens), ints([0, 1, 2]), 1, 48)
        before = w.raw.clone()
        c, key = torch.randn((2, 256), generator=g).to(BF), torch.randn((2, 32), generator=g).to(BF)
        w.cache.append(batch, Rotary(32), c.cuda(), key.cuda(), ints([0, 0]))  # position 0: the rotary part as it is
        assert w.cache.status() == 0
        codes, powers, _ = lref.encode(c)
        new = lref.pack(codes, powers, key) if bits == 8 else torch.cat([c, key], 1).view(torch.uint8)
        after = before.cpu()
        for i, n in enumerate(lens):
            p, r = ref.cells(w.table[i], 16, n)
            row = new[i].clone()
            after[p[-1], r[-1], :256 + 8 if bits == 8 else row.numel()] = row[:256 + 8 if bits == 8 else row.numel()]
            after[p[-1], r[-1], row.numel() - 64:row.numel()] = row[-64:]
        assert torch.equal(w.raw.cpu(), after)
        w.kv_lens = lens
        values = []
        for i, n in enumerate(lens):
            rows = w.cells(i)[:, :lref.row_bytes(256, 32, bits)].contiguous()
            lat = lref.decode(rows[:, :256], rows[:, 256:264], BF).to(BF) if bits == 8 else rows[:, :512].contiguous().view(BF)
            values.append((lat, rows[:, -64:].contiguous().view(BF)))
        q, qr = torch.randn((2, 8, 256), generator=g).to(BF), torch.randn((2, 8, 32), generator=g).to(BF)
        out = w.cache.attend(batch, q.cuda(), qr.cuda(), 0.08)
        for i in range(2):
            o, _, ot, _ = lref.absorbed(q[i:i + 1], qr[i:i + 1], *values[i], 0.08, True)
            check_rows(i, out[i:i + 1], o, ot, None, None, None)


@pytest.mark.parametrize("bits,page", [(16, 16), (16, 256), (8, 64)])
def test_pages_whose_slots_are_apart(bits, page):
    """Slot r of every page before slot r + 1 of the first: the strides of pages and slots the other way round."""
    from expert_slot_cache_device_gb300.kv_cache import Rotary
    from expert_slot_cache_device_gb300.latent_cache import LatentCache

    w = World([3, 1, 70], [300, 64, 500], 256, 48, page, BF, bits, seed=5)
    turned = w.cache.pages.transpose(0, 1).contiguous().transpose(0, 1)
    w.cache = LatentCache(turned.shape[0], page, 256, 48, BF, bits, pages=turned)
    check_attend(w, 20)
    rows = w.cache.read(w.batch, ints(starts(w.kv_lens)), rows=864).cpu()
    assert torch.equal(rows, torch.cat([torch.cat([c, k], 1) for c, k in zip(w.c, w.key)]))
    c, key = torch.randn((74, 256), generator=w.gen).to(BF), torch.randn((74, 48), generator=w.gen).to(BF)
    w.cache.append(w.batch, Rotary(48), c.cuda(), key.cuda(), torch.zeros(74, dtype=torch.int32, device="cuda"))
    new = torch.cat([c if bits == 16 else lref.decode(*lref.encode(c)[:2], BF).to(BF), key], 1)  # position 0: nothing turns
    for at, t in ((297, slice(0, 3)), (363, slice(3, 4)), (794, slice(4, 74))):
        rows[at:at + t.stop - t.start] = new[t]
    assert torch.equal(w.cache.read(w.batch, ints(starts(w.kv_lens)), rows=864).cpu(), rows) and w.cache.status() == 0


@pytest.mark.parametrize("bits", [16, 8])
def test_read_under_a_loose_bound(bits):
    """A bound of cached tokens far above the rows of `out`: the same rows; a sequence with more tokens than rows is recorded and cut."""
    from expert_slot_cache_device_gb300 import ftmoe as F
    from expert_slot_cache_device_gb300.kv_cache import KVBatch

    w = World([1, 1, 1], [33, 1, 200], 128, 32, 16, HF, bits, seed=4)
    table = torch.full((3, 1 << 13), -1, dtype=torch.int32)
    table[:, :w.table.shape[1]] = w.table
    batch = KVBatch(table.cuda(), ints(w.kv_lens), ints(w.cu), 1, 1 << 17)
    want = torch.cat([torch.cat([c, k], 1) for c, k in zip(w.c, w.key)])
    for rows in (234, 300):
        out = torch.full((rows, 160), 7.0, dtype=HF, device="cuda")
        w.cache.read(batch, ints([0, 33, 34, 234]), out=out)
        assert w.cache.status() == 0 and torch.equal(out[:234].cpu(), want) and (out[234:] == 7).all()
    out = torch.full((40, 160), 7.0, dtype=HF, device="cuda")
    w.cache.read(batch, ints([0, 33, 34, 234]), out=out)  # six rows for the last sequence
    assert w.cache.status() == F.ERR_STATE and torch.equal(out.cpu(), want[:40])
