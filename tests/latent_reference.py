"""Plain implementations in 64 bits of the latent-attention operators, on the CPU, and what
rounding may move their results by. Shared by the tests."""
import torch

import attention_reference as ref

U, F32 = ref.U, ref.F32


def row_bytes(latent, rope, bits):
    return 2 * (latent + rope) if bits == 16 else latent + -(-latent // 512) * 16 + 2 * rope


def encode(y):
    """Latents of a 16-bit type [rows, latent] -> (codes uint8, powers uint8), value by value in 64 bits:
    the least e in [-127, 127] with max |y| <= 448 * 2^e, codes to nearest even."""
    x = y.double().cpu().view(len(y), -1, 32)
    bad = ~torch.isfinite(x).all(2)
    x = torch.where(bad[..., None], 0.0, x)
    most = 61440.0 if y.dtype == torch.float16 else 1.875 * 2.0 ** 127  # the next code's value would be infinite
    x = x.clamp(-most, most)
    top = x.abs().amax(2)
    e = torch.full(top.shape, -127, dtype=torch.int64)
    for _ in range(255):
        e = torch.where(top > 448 * torch.exp2(e.double()), e + 1, e)
    z = x / torch.exp2(e.double())[..., None]
    mag = z.abs()
    exp = torch.floor(torch.log2(mag.clamp(min=2.0 ** -6))).clamp(max=8)
    n = torch.round(mag / torch.exp2(exp - 3)).long()       # eighths of 2^exp, ties to even
    up = n == 16
    exp, n = torch.where(up, exp + 1, exp), torch.where(up, 8, n)
    code = torch.where(n < 8, n, (exp.long() + 7) * 8 + n - 8)  # n < 8 at 2^-6: steps of 2^-9
    code = torch.where(torch.signbit(z), code + 128, code)
    power = torch.where(bad, 255, e + 127)
    return code.view(len(y), -1).to(torch.uint8), power.to(torch.uint8), bad


def decode(codes, powers, dtype):
    """Values of stored codes, rounded to dtype, as fp64."""
    c = codes.long()
    exp, frac = c // 8 % 16, (c % 8).double()
    mag = torch.where(exp == 0, frac * 2.0 ** -9, (1 + frac / 8) * torch.exp2((exp - 7).double()))
    mag = torch.where(c % 128 == 127, torch.nan, mag)
    p = torch.exp2(powers.double() - 127)
    p = torch.where(powers == 255, torch.nan, p)
    return (torch.where(c >= 128, -mag, mag) * p.repeat_interleave(32, -1)).to(dtype).double()


def pack(codes, powers, key):
    """Stored rows of 8 bits."""
    pad = torch.zeros((len(codes), -powers.shape[1] % 16), dtype=torch.uint8)
    return torch.cat([codes, powers, pad, key.contiguous().view(torch.uint8)], 1)


def norm(c, weight, eps):
    """(y in fp64, bound of what fp32 and one rounding to c's type may move it by)."""
    x = c.double().cpu()
    y = x / torch.sqrt((x * x).mean(1, keepdim=True) + eps) * weight.double().cpu()
    # a sum of n squares in fp32 is off by n units at most, its root by half of that; rsqrt by 2 units, three products
    return y, (U[c.dtype] + (c.shape[1] / 2 + 8) * F32) * y.abs() + 2.0 ** -25


def absorbed(q, q_rope, c, key, scale, causal):
    """One sequence: q [rows, heads, latent], q_rope [rows, heads, rope], c [slots, latent], key [slots, rope]
    (values of q's type). (out, lse, out_tol, lse_tol) as attention_reference.attention gives them."""
    dt, latent = q.dtype, q.shape[2]
    k = torch.cat([c, key], 1)[:, None].to(dt)
    v = torch.cat([c, torch.zeros_like(key)], 1)[:, None].to(dt)
    out, lse, _, ot, lt, _ = ref.attention(torch.cat([q, q_rope], 2), k, v, scale, 0, causal, None)
    return out[..., :latent], lse, ot[..., :latent], lt


def expanded(q, k, key, v, scale, causal):
    """One sequence: q [rows, heads, nope + rope], k [slots, heads, nope], key [slots, rope], v [slots, heads, vd]."""
    n, heads, vd = v.shape
    kk = torch.cat([k, key[:, None].expand(-1, heads, -1)], 2)
    vv = torch.cat([v, torch.zeros((n, heads, kk.shape[2] - vd), dtype=v.dtype)], 2)
    out, lse, _, ot, lt, _ = ref.attention(q, kk, vv, scale, 0, causal, None)
    return out[..., :vd], lse, ot[..., :vd], lt
