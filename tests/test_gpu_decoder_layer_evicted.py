"""The decoder layer of examples/decoder_layer.py on caches that were evicted: outputs and mass against the same layer in plain
64-bit torch over the kept rows alone."""
import pytest
import torch

import attention_reference as ref
from test_gpu_decoder_layer import Plain, close, example  # noqa: F401

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]


@pytest.mark.parametrize("after", [[[1, 1, 1]] * 16, [[20, 3, 9], [1, 1, 1], [2, 0, 17]]], ids=["single tokens", "chunks"])
def test_layer_after_an_eviction(example, after):  # noqa: F811
    layer, plain = example.synthetic_layer()
    want = Plain(layer, plain)
    seqs = example.Sequences(layer, 3, 256)
    g = torch.Generator().manual_seed(4)
    prompt = [33, 21, 40]
    batch, pos = seqs.grow(prompt)
    layer.forward(torch.randn((sum(prompt), 256), generator=g).to(torch.bfloat16).cuda(), batch, pos, seqs.mass)
    rows = []
    for i, n in enumerate(prompt):
        p, r = ref.cells(torch.tensor(seqs.tables[i]), 16, n)
        rows.append((layer.cache.k_pages[p, r].cpu(), layer.cache.v_pages[p, r].cpu()))
    kept = seqs.evict(layer, batch, budget=24, recent=6).cpu().long()
    assert seqs.lens == [24, 21, 24]
    for i, n in enumerate(seqs.lens):
        k, v = (torch.stack([t[kept[i, h, :n], h] for h in range(layer.kv_heads)], 1) for t in rows[i])
        want.k[i], want.v[i] = k, v
    mass = [seqs.mass[i].double().cpu() for i in range(3)]
    assert all((m[:, n:] == 0).all() for m, n in zip(mass, seqs.lens))
    seen = 0
    for step, new in enumerate(after):
        batch, pos = seqs.grow(new)
        x = torch.randn((sum(new), 256), generator=g).to(torch.bfloat16)
        got = layer.forward(x.cuda(), batch, pos, seqs.mass)
        ref_out, sure = want.forward(example.norm, x, new, pos.cpu(), mass)  # rows whose routing hangs on no rounding
        if sure.any():
            close(got[sure.cuda()], ref_out[sure], step)
        seen += int(sure.sum())
        for i, n in enumerate(seqs.lens):
            close(seqs.mass[i, :, :n], mass[i][:, :n], ("mass", step))
            assert (seqs.mass[i, :, n:] == 0).all()
    assert seen >= 12  # of 48 and 52
    assert pos[-1] == prompt[2] + sum(a[2] for a in after) - 1  # positions run on, slots do not
    assert layer.cache.status() == 0 and layer.experts.status() == 0
    layer.experts.close()
