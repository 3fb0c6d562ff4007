"""The attention half and the routed experts together, as examples/decoder_layer.py runs them: prompts in
ragged chunks, single-token steps and an eviction, against the same layer in plain 64-bit torch."""
import importlib.util
import os

import pytest
import torch

import attention_reference as ref

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    from expert_slot_cache_device_gb300 import build

    build.build()
    spec = importlib.util.spec_from_file_location("decoder_layer", os.path.join(ROOT, "examples", "decoder_layer.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


class Plain:
    """The layer in 64 bits; activations are rounded to bf16 where the framework hands them on."""

    def __init__(self, layer, plain):
        from expert_slot_cache_device_gb300.kv_cache import rotary_frequencies

        self.l, self.p = layer, plain
        self.freq, _ = rotary_frequencies(layer.dim)
        self.k, self.v = {}, {}

    @staticmethod
    def bf(x):
        return x.to(torch.bfloat16)

    def forward(self, norm, x, new, pos, mass):
        l, p = self.l, self.p
        n = x.shape[0]
        y, _ = ref.w4(norm(x), *p["qkv"], None, 64)
        q, k, v = self.bf(y).view(n, -1, l.dim).split([l.heads, l.kv_heads, l.kv_heads], 1)
        q, k = (self.bf(ref.rotate(t, pos, self.freq, 1.0, l.dim, "half")) for t in (q, k))
        out, at = [], 0
        for i, m in enumerate(new):
            for store, t in ((self.k, k), (self.v, v)):
                store[i] = torch.cat([store[i], t[at:at + m]]) if i in store else t[at:at + m]
            o, _, w, _, _, _ = ref.attention(q[at:at + m], self.k[i], self.v[i], l.dim ** -0.5, 0, True, None)
            mass[i][:, :w.shape[1]] += w
            out.append(self.bf(o))
            at += m
        y, _ = ref.w4(torch.cat(out).reshape(n, -1), *p["o"], None, 64)
        x = x + self.bf(y)
        h = norm(x)
        s = torch.softmax(h.double() @ p["router"].double().T, -1)
        weights, ids = s.topk(l.topk)
        gap = s.sort(-1, descending=True).values
        weights = weights / weights.sum(-1, keepdim=True)
        y = torch.zeros(x.shape, dtype=torch.float64)
        for t in range(n):
            for j in range(l.topk):
                e = int(ids[t, j])
                gu = p["gate_up"][e].double() @ h[t].double()
                a, b = gu.chunk(2)
                y[t] += weights[t, j] * (p["down"][e].double() @ (torch.nn.functional.silu(a) * b))
        # rows whose routing does not hang on a rounding
        return x + self.bf(y), (gap[:, l.topk - 1] - gap[:, l.topk]) > 2e-2


def close(a, b, what):
    a, b = a.double().cpu(), b.double().cpu()
    err = float((a - b).norm() / b.norm())
    # four roundings to bf16 (2^-9 relative on average) on the way, each carried through a layer of O(1) gain
    assert err < 1e-2, (what, err)


def test_layer_against_plain(example):
    layer, plain = example.synthetic_layer()
    want = Plain(layer, plain)
    seqs = example.Sequences(layer, 3, 256)
    mass = [torch.zeros((layer.kv_heads, 256), dtype=torch.float64) for _ in range(3)]
    g = torch.Generator().manual_seed(2)
    seen = 0
    for step, new in enumerate([[33, 1, 20], [17, 40, 2], [1, 1, 1], [1, 1, 1]]):
        batch, pos = seqs.grow(new)
        x = torch.randn((sum(new), 256), generator=g).to(torch.bfloat16)
        got = layer.forward(x.cuda(), batch, pos, seqs.mass)
        ref_out, sure = want.forward(example.norm, x, new, pos.cpu(), mass)
        assert sure.any()
        close(got[sure.cuda()], ref_out[sure], step)
        seen += int(sure.sum())
        for i in range(3):
            close(seqs.mass[i, :, :seqs.lens[i]], mass[i][:, :seqs.lens[i]], "mass")
    assert seen > 60
    # eviction: the kept rows are the cache's, and the next step attends to them alone
    lens = list(seqs.lens)
    rows = []
    for i, n in enumerate(lens):
        p, r = ref.cells(torch.tensor(seqs.tables[i]), 16, n)
        rows.append((layer.cache.k_pages[p, r].cpu(), layer.cache.v_pages[p, r].cpu()))
    m = seqs.mass.cpu().clone()
    kept = seqs.evict(layer, batch, budget=24, recent=6)
    assert seqs.lens == [24, 24, 24 if lens[2] > 24 else lens[2]]
    for i, n in enumerate(lens):
        ks, vs = [], []
        for h in range(layer.kv_heads):
            sel = ref.evict(m[i, h], n, 24, 6)
            assert kept[i, h, :len(sel)].tolist() == sel
            ks.append(rows[i][0][sel, h])
            vs.append(rows[i][1][sel, h])
        want.k[i], want.v[i] = torch.stack(ks, 1), torch.stack(vs, 1)
    batch, pos = seqs.grow([1, 1, 1])
    assert pos.tolist() == lens  # positions run on, slots do not
    x = torch.randn((3, 256), generator=g).to(torch.bfloat16)
    got = layer.forward(x.cuda(), batch, pos, seqs.mass)
    ref_out, sure = want.forward(example.norm, x, [1, 1, 1], pos.cpu(), [torch.zeros((layer.kv_heads, 256), dtype=torch.float64)] * 3)
    if sure.any():
        close(got[sure.cuda()], ref_out[sure], "after eviction")
    assert layer.cache.status() == 0 and layer.experts.status() == 0
    layer.experts.close()


def test_example_runs(example, capsys):
    example.main()
    assert "cached tokens" in capsys.readouterr().out
