"""Plain implementations in 64 bits of the attention half's operators, and what rounding may
move their results by. CPU only; shared by the tests."""
import math

import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}  # unit roundoff: 8 and 11 significant bits
F32 = 2.0 ** -24


def rotate(x, pos, freq, factor, rot, layout):
    """x [tokens, heads, dim] (any float type) -> fp64."""
    x = x.double().cpu().clone()
    a = pos.double().cpu()[:, None] * freq
    c, s = (a.cos() * factor)[:, None], (a.sin() * factor)[:, None]
    h = rot // 2
    i, j = (slice(0, h), slice(h, rot)) if layout == "half" else (slice(0, rot, 2), slice(1, rot, 2))
    p, q = x[..., i].clone(), x[..., j].clone()
    x[..., i], x[..., j] = p * c - q * s, q * c + p * s
    return x


def cells(table, page, n):
    j = torch.arange(n)
    return table[j // page].long(), j % page


def attention(q, k, v, scale, window, causal, sinks):
    """One sequence: q [rows, heads, dim], k and v [slots, kv_heads, dim]. Returns fp64 out, lse,
    mass [kv_heads, slots], and bounds on what the arithmetic that the operator states may move
    them by: scores in fp32 (eps), probabilities rounded to the cache's type for out alone."""
    dt = q.dtype
    q, k, v = q.double().cpu(), k.double().cpu(), v.double().cpu()
    rows, heads, dim = q.shape
    n, kv = k.shape[:2]
    rep = heads // kv
    at = torch.arange(rows)[:, None] + n - rows
    j = torch.arange(n)[None]
    sees = (j <= at) if causal else (at >= 0).expand(rows, n).clone()
    if window:
        sees &= j > at - window
    out, lse = torch.zeros_like(q), torch.full((rows, heads), -math.inf, dtype=torch.float64)
    mass, out_tol = torch.zeros(kv, n, dtype=torch.float64), torch.zeros_like(q)
    lse_tol, mass_tol = torch.zeros(rows, heads, dtype=torch.float64), torch.zeros(kv, n, dtype=torch.float64)
    live = sees.any(0)  # slots no row sees may hold anything
    k, v = torch.where(live[:, None, None], k, 0.0), torch.where(live[:, None, None], v, 0.0)
    for h in range(heads):
        g = h // rep
        s = (q[:, h] @ k[:, g].T * scale).masked_fill(~sees, -math.inf)
        # |error| of an fp32 dot product of dim terms, of its product with scale and log2 e, and of
        # the exponential (2 units in the last place): relative error of a probability
        mag = (q[:, h].abs() @ k[:, g].abs().T * scale).masked_fill(~sees, 0.0)
        eps = ((dim + 8) * F32 * mag.max(1).values if n else torch.zeros(rows)) + 16 * F32
        full = torch.cat([s, sinks[h].double().cpu().expand(rows, 1)], 1) if sinks is not None else s
        z = torch.logsumexp(full, 1) if full.shape[1] else torch.full((rows,), -math.inf, dtype=torch.float64)
        p = torch.where(z[:, None] == -math.inf, 0.0, torch.exp(s - z[:, None]))
        lse[:, h], out[:, h] = z, p @ v[:, g]
        weight = p @ v[:, g].abs()
        small = n * 2.0 ** -25 * v[:, g].abs().max() if n and dt == torch.float16 else 0.0  # subnormal probabilities
        out_tol[:, h] = U[dt] * out[:, h].abs() + (U[dt] + 2 * eps[:, None] + n * F32) * weight + small + 2.0 ** -25
        lse_tol[:, h] = torch.where(z == -math.inf, 0.0, 2 * eps + n * F32 / 16 + 4 * F32 * z.abs().nan_to_num(0, 0, 0))
        mass[g] += p.sum(0)
        mass_tol[g] += ((2 * eps + n * F32 / 16 + 4 * F32 * z.abs().nan_to_num(0, 0, 0) + 16 * F32)[:, None] * p).sum(0)
    mass_tol += rows * rep * F32 * mass
    return out, lse, mass, out_tol, lse_tol, mass_tol


def evict(mass, n, budget, recent):
    """Slots kept of one (sequence, key head): python sort, ties to the lowest slot."""
    if n <= budget:
        return list(range(n))
    m = mass[:n].double().cpu().tolist()
    old = n - recent
    order = sorted(range(old), key=lambda j: (-(m[j] if m[j] == m[j] else -math.inf), m[j] != m[j], j))
    return sorted(order[:budget - recent]) + list(range(old, n))


def w4(x, codes, scales, zeros, group):
    """y in fp64 and the sum of its terms' magnitudes."""
    codes = codes.cpu()
    n, half = codes.shape
    q = torch.empty((n, 2 * half), dtype=torch.float64)
    q[:, 0::2], q[:, 1::2] = (codes & 15).double(), (codes >> 4).double()
    z = zeros.cpu().double().repeat_interleave(group, 1) if zeros is not None else 8.0
    w = (q - z) * scales.cpu().double().repeat_interleave(group, 1)
    x = x.cpu().double()
    return x @ w.T, x.abs() @ w.abs().T
