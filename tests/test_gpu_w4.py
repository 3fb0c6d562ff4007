"""Products with 4-bit weights on the GPU against a plain implementation in 64 bits."""
import pytest
import torch

import attention_reference as ref

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]
BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _built():
    from expert_slot_cache_device_gb300 import build

    build.build()


def _weights(n, k, group, zeros, dt, g):
    codes = torch.randint(0, 256, (n, k // 2), generator=g, dtype=torch.uint8)
    scales = (torch.rand((n, k // group), generator=g) * 0.05 - 0.02).to(dt)
    z = torch.randint(0, 16, (n, k // group), generator=g, dtype=torch.uint8) if zeros else None
    return codes, scales, z


@pytest.mark.parametrize("n,k,group", [(1, 32, 32), (16, 64, 64), (17, 96, 32), (100, 128, 128), (33, 320, 64),
                                       (250, 2880, 32), (384, 7168, 128), (1000, 1344, 64), (4113, 640, 128)])
@pytest.mark.parametrize("tokens", [1, 2, 7, 8, 9, 16, 17, 24, 32, 33, 65, 70, 131])
@pytest.mark.parametrize("zeros", [False, True])
def test_matvec(n, k, group, tokens, zeros):
    from expert_slot_cache_device_gb300.w4 import W4Weights

    for dt in (BF, HF):
        g = torch.Generator().manual_seed(n + k + tokens)
        codes, scales, z = _weights(n, k, group, zeros, dt, g)
        w = W4Weights(codes.cuda(), scales.cuda(), z.cuda() if zeros else None, group)
        wide = torch.randn((tokens, k + 24), generator=g).to(dt)
        x = wide.cuda()[:, 8:8 + k]  # rows further apart than K
        out = torch.full((tokens, n + 3), 7.0, dtype=dt, device="cuda")
        y = w.matvec(x, out=out[:, :n])
        want, size = ref.w4(x, codes, scales, z, group)
        # one rounding of y, and fp32 sums: k / 16 tensor-core steps and a scale a group, each at
        # most 2^-22 of the terms' magnitudes
        tol = ref.U[dt] * want.abs() + (k / 16 + k / group + 16) * 2.0 ** -22 * size + 2.0 ** -25
        d = (y.double().cpu() - want).abs()
        assert (d <= tol).all(), float((d / tol).max())
        assert (out[:, n:] == 7.0).all()


def test_matvec_repeats_bit_for_bit_and_keeps_values():
    """The same call twice, on another stream and in a graph; a weight of one non-zero code
    gives x times that weight alone; infinities stay in their own rows and tokens."""
    from expert_slot_cache_device_gb300.w4 import W4Weights

    g = torch.Generator().manual_seed(0)
    n, k, group = 48, 256, 64
    codes = torch.full((n, k // 2), 0x88, dtype=torch.uint8)  # every weight 0
    col = torch.randint(0, k, (n,), generator=g)
    for i in range(n):
        c = int(col[i])
        codes[i, c // 2] = 0x8F if c % 2 == 0 else 0xF8  # code 15: w = 7 s
    scales = torch.full((n, k // group), 0.5, dtype=BF)
    w = W4Weights(codes.cuda(), scales.cuda(), None, group)
    x = torch.randn((5, k), generator=g).to(BF)
    y = w.matvec(x.cuda())
    assert torch.equal(y.cpu(), (x[:, col].float() * 3.5).to(BF))
    side = torch.cuda.Stream()
    xc, z = x.cuda(), torch.empty_like(y)
    torch.cuda.synchronize()
    again = w.matvec(xc, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(again, y)
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            w.matvec(xc, out=z)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(z, y)
    x[2, int(col[4])] = float("inf")
    y = w.matvec(x.cuda()).cpu()
    assert torch.isfinite(y[[0, 1, 3, 4]]).all() and y[2, 4] == float("inf")
    assert w.matvec(x.cuda()[:0]).shape == (0, n)


@pytest.mark.parametrize("tokens,n,group", [(24, 300, 64), (70, 144, 128), (17, 2000, 32)])
def test_matvec_many_tokens_repeats_and_keeps_values(tokens, n, group):
    """The same for more tokens: bit for bit again, from a graph too; a token's infinity or NaN and a row's
    infinite scale stay their own."""
    from expert_slot_cache_device_gb300.w4 import W4Weights

    k = 1024
    g = torch.Generator().manual_seed(tokens)
    codes, scales, z = _weights(n, k, group, True, BF, g)
    w = W4Weights(codes.cuda(), scales.cuda(), z.cuda(), group)
    x = torch.randn((tokens, k), generator=g).to(BF).cuda()
    y = w.matvec(x)
    out = torch.empty_like(y)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            w.matvec(x, out=out)
    for _ in range(2):
        out.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, y)
    x[3, 5], x[tokens - 1, k - 1] = float("inf"), float("nan")
    scales[n - 1, 0] = float("inf")
    w = W4Weights(codes.cuda(), scales.cuda(), z.cuda(), group)
    got = w.matvec(x)
    keep = [t for t in range(tokens) if t not in (3, tokens - 1)]
    assert torch.equal(got[keep, :n - 1], y[keep, :n - 1])
    assert not torch.isfinite(got[3]).any() and torch.isnan(got[tokens - 1]).all() and not torch.isfinite(got[:, n - 1]).any()
