"""Products with 4-bit weights of prompts: many tokens, against a plain implementation in 64 bits and against the same rows in
smaller calls."""
import pytest
import torch

import attention_reference as ref
from test_gpu_w4 import BF, HF, _weights

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from expert_slot_cache_device_gb300 import build

    build.build()


def test_more_tokens_than_a_grid_has_tiles():
    from expert_slot_cache_device_gb300.w4 import W4Weights

    g = torch.Generator().manual_seed(1)
    n, k, tokens = 16, 32, (1 << 22) + 70
    codes, scales, z = _weights(n, k, 32, True, BF, g)
    w = W4Weights(codes.cuda(), scales.cuda(), z.cuda(), 32)
    x = torch.randn((tokens, k), generator=torch.Generator("cuda").manual_seed(2), device="cuda").to(BF)
    y = w.matvec(x)
    for at in (0, 65535 * 32, (1 << 21) - 64, 1 << 21, (1 << 22) - 64, tokens - 134):
        assert torch.equal(y[at:at + 134], w.matvec(x[at:at + 134])), at
    at = torch.randint(0, tokens, (2000,), generator=g)
    want, size = ref.w4(x[at.cuda()], codes, scales, z, 32)
    # one rounding of y, and fp32 sums as in test_gpu_w4
    tol = ref.U[BF] * want.abs() + (k / 16 + k / 32 + 16) * 2.0 ** -22 * size + 2.0 ** -25
    assert ((y[at.cuda()].double().cpu() - want).abs() <= tol).all()


@pytest.mark.parametrize("n,k,group", [(300, 1344, 64), (144, 2880, 32), (1000, 7168, 128)])
@pytest.mark.parametrize("tokens", [129, 200, 513, 1000])
@pytest.mark.parametrize("zeros", [False, True])
def test_matvec_of_prompts(n, k, group, tokens, zeros):
    from expert_slot_cache_device_gb300.w4 import W4Weights

    for dt in (BF, HF):
        g = torch.Generator().manual_seed(n + tokens)
        codes, scales, z = _weights(n, k, group, zeros, dt, g)
        w = W4Weights(codes.cuda(), scales.cuda(), z.cuda() if zeros else None, group)
        x = torch.randn((tokens, k + 8), generator=g).to(dt)[:, :k]
        out = torch.full((tokens, n + 1), 7.0, dtype=dt, device="cuda")
        wide = torch.zeros((tokens, k + 8), dtype=dt, device="cuda")
        wide[:, :k] = x.cuda()
        y = w.matvec(wide[:, :k], out=out[:, :n])
        want, size = ref.w4(x, codes, scales, z, group)
        tol = ref.U[dt] * want.abs() + (k / 16 + k / group + 16) * 2.0 ** -22 * size + 2.0 ** -25  # as in test_gpu_w4
        d = (y.double().cpu() - want).abs()
        assert (d <= tol).all(), float((d / tol).max())
        assert (out[:, n:] == 7.0).all()
