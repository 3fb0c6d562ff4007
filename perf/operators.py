"""Operators of the attention half of a decoder layer, next to the expert cache: what is timed.

Four operators, each as a program that serves a mixture-of-experts model from the slot cache
calls it:

* ``append``  rotary positions on the new tokens' queries and keys; keys and values go to the
              pages of a paged key/value cache;
* ``attend``  attention of the new tokens (one a sequence, or a chunk) over that cache, with
              the log-sum-exp and, where asked for, the attention weight each cached token drew
              added to its running mass;
* ``evict``   the cached tokens of largest mass, and the most recent ones, move to new pages;
* ``matvec``  products with 4-bit weights and group scales (the layer's dense projections).

``run`` computes them with elementary torch operations in 32 bits where ``own`` is false, and
with the framework's calls where it is true. ``exact`` gives the same in 64 bits.
"""
import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16}
MAX_POS = 1 << 17


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one new token for each of 16 running sequences: latency of a decode step
        dict(name="append step", op="append", batch=16, q=1, ctx=9000, heads=32, kv_heads=4, dim=128, rot=128,
             layout="half", scaling="none", page=16, dtype="bf16"),
        # a ragged batch of prompt chunks; half of each head rotated in interleaved pairs, positions
        # stretched for a long context
        dict(name="append prompt", op="append", batch=3, q=4001, ctx=12000, heads=64, kv_heads=8, dim=128, rot=64,
             layout="interleaved", scaling="yarn", page=32, dtype="f16"),
        # a single user's decode step on a short context: the smallest call
        dict(name="step short", op="attend", batch=1, q=1, ctx=777, heads=32, kv_heads=4, dim=128, page=16,
             window=0, sinks=False, mass=False, dtype="bf16"),
        # a batch of decode steps over long caches, accumulating the mass that eviction goes by
        dict(name="step long mass", op="attend", batch=24, q=1, ctx=16300, heads=64, kv_heads=4, dim=128, page=16,
             window=0, sinks=False, mass=True, dtype="bf16"),
        # decode steps of a layer with a sliding window and a sink logit per head
        dict(name="step window", op="attend", batch=64, q=1, ctx=5000, heads=64, kv_heads=8, dim=64, page=32,
             window=128, sinks=True, mass=False, dtype="f16"),
        # short ragged chunks, one to about a hundred tokens, in one call with decode steps
        dict(name="chunk ragged", op="attend", batch=7, q=97, ctx=1500, heads=40, kv_heads=8, dim=64, page=16,
             window=0, sinks=False, mass=False, dtype="f16"),
        # a whole prompt at once
        dict(name="chunk prompt", op="attend", batch=1, q=4096, ctx=4096, heads=32, kv_heads=4, dim=128, page=64,
             window=0, sinks=False, mass=False, dtype="bf16"),
        # a chunk of a long prompt late in its context, with mass: the call with the most arithmetic
        dict(name="chunk long mass", op="attend", batch=1, q=2048, ctx=31000, heads=32, kv_heads=8, dim=128, page=16,
             window=0, sinks=False, mass=True, dtype="bf16"),
        # two short sequences cut to half their length
        dict(name="evict small", op="evict", batch=2, ctx=1013, kv_heads=4, dim=128, page=16, budget=500, recent=64,
             dtype="bf16"),
        # a batch of long sequences cut to a quarter
        dict(name="evict large", op="evict", batch=16, ctx=16384, kv_heads=8, dim=128, page=16, budget=4096,
             recent=512, dtype="bf16"),
        # one token through a projection with zero points
        dict(name="matvec one", op="matvec", tokens=1, n=2048, k=7168, group=128, zeros=True, dtype="bf16"),
        # a decode batch through a large projection
        dict(name="matvec batch", op="matvec", tokens=24, n=16384, k=7168, group=64, zeros=False, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    """Spread over the logarithm, and off the large powers of two."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return v + (v % 512 == 0)


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "attend", "evict", "matvec"])
    dtype = rng.choice(["bf16", "f16"])
    if op == "matvec":
        group = rng.choice([32, 64, 128])
        return dict(op=op, tokens=_log(rng, 1, 32), n=_log(rng, 120, 16000),
                    k=group * (2 * _log(rng, 1, 3500 // group) + 1), group=group,
                    zeros=rng.random() < 0.5, dtype=dtype)
    page = rng.choice([16, 32, 64, 128])
    kv = rng.choice([1, 2, 4, 8])
    if op == "evict":
        ctx = _log(rng, 40, 16384)
        budget = max(2, int(ctx * rng.uniform(0.1, 1.1)))
        return dict(op=op, batch=_log(rng, 1, 16), ctx=ctx, kv_heads=kv, dim=rng.choice([64, 128]), page=page,
                    budget=budget, recent=int(budget * rng.uniform(0, 0.5)), dtype=dtype)
    heads = kv * rng.choice([1, 2, 3, 4, 5, 7, 8])
    dim = rng.choice([64, 128])
    if op == "append":
        q = 1 if rng.random() < 0.5 else _log(rng, 2, 4000)
        batch = _log(rng, 1, 64) if q == 1 else _log(rng, 1, 3)
        return dict(op=op, batch=batch, q=q, ctx=q + _log(rng, 1, 8000), heads=heads, kv_heads=kv, dim=dim,
                    rot=rng.choice([dim, dim // 2, dim // 4]), layout=rng.choice(["half", "interleaved"]),
                    scaling=rng.choice(["none", "linear", "yarn"]), page=page, dtype=dtype)
    if rng.random() < 0.5:
        q, batch = 1, _log(rng, 1, 48)
        ctx = _log(rng, 1, 12000)
    else:
        q = _log(rng, 2, 2048)
        batch = _log(rng, 1, max(1.01, min(8.0, 2048 / q)))
        ctx = q + _log(rng, 1, 16000)
    return dict(op=op, batch=batch, q=q, ctx=ctx, heads=heads, kv_heads=kv, dim=dim, page=page,
                window=rng.choice([0, 0, 0, 128, 1000]), sinks=rng.random() < 0.25, mass=rng.random() < 0.35,
                dtype=dtype)


def _lens(case):
    """(new tokens, cached tokens with them) of each sequence: the first as long as the case
    says, the others shorter, at random but the same for the same case."""
    r = random.Random("%d %d %d" % (case["batch"], case.get("q", 0), case["ctx"]))
    q, n = [], []
    for i in range(case["batch"]):
        qi = case.get("q", 1) if i == 0 else r.randint(1, case.get("q", 1))
        ni = case["ctx"] if i == 0 else r.randint(qi, case["ctx"])
        q.append(qi)
        n.append(max(ni, qi))
    return q, n


def _visible(case):
    """Query-key pairs (of one head) and cached tokens that at least one query sees."""
    w, pairs, seen = case["window"], 0, 0
    for q, n in zip(*_lens(case)):
        for lo, hi in ((n - q + 1, n),):  # query i sees its own position and those before it
            if w:
                full = max(0, hi - max(lo, w) + 1)
                low = min(hi, w - 1)
                pairs += full * w + (max(0, low * (low + 1) - (lo - 1) * lo) // 2 if low >= lo else 0)
            else:
                pairs += (lo + hi) * q // 2
        seen += min(n, q + w - 1) if w else n
    return pairs, seen


def work(case):
    if case["op"] == "matvec":
        t, n, k = case["tokens"], case["n"], case["k"]
        groups = n * k // case["group"]
        return {"bytes": n * k // 2 + groups * (3 if case["zeros"] else 2) + 2 * t * (n + k), "flops": 2 * t * n * k}
    row = 2 * case["dim"]
    q, n = _lens(case)
    if case["op"] == "evict":
        kept = sum(min(x, case["budget"]) for x in n) * case["kv_heads"]
        return {"bytes": kept * (4 * row + 8) + sum(n) * case["kv_heads"] * 4, "flops": 0}
    tokens = sum(q)
    if case["op"] == "append":
        return {"bytes": 2 * tokens * (case["heads"] + 2 * case["kv_heads"]) * row + 4 * tokens,
                "flops": 3 * tokens * (case["heads"] + case["kv_heads"]) * case["rot"]}
    pairs, seen = _visible(case)
    return {"bytes": tokens * case["heads"] * (2 * row + 4) + seen * case["kv_heads"] * (2 * row + (8 if case["mass"] else 0)),
            "flops": 4 * pairs * case["heads"] * case["dim"]}


# ---------------------------------------------------------------- inputs
def _freq(case):
    """Rotary frequencies (radians a position, 64 bits) and the factor on the rotated part, as
    the framework's own plan defines them: base 10000; "linear" divides positions by 4; "yarn"
    divides by 8 the frequencies that turn less than once in 4096 positions, keeps those that
    turn more than 32 times, and blends between them, with the factor 0.1 ln 8 + 1."""
    half = case["rot"] // 2
    f = torch.arange(half, dtype=torch.float64).mul_(-2.0 / case["rot"] * math.log(10000.0)).exp_()
    if case["scaling"] == "linear":
        return f / 4.0, 1.0
    if case["scaling"] == "yarn":
        at = lambda turns: case["rot"] * math.log(4096 / (turns * 2 * math.pi)) / (2 * math.log(10000.0))  # noqa: E731
        lo, hi = max(math.floor(at(32.0)), 0), min(math.ceil(at(1.0)), case["rot"] - 1)
        ramp = ((torch.arange(half, dtype=torch.float64) - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
        return f * (1 - ramp) + f / 8.0 * ramp, 0.1 * math.log(8.0) + 1.0
    return f, 1.0


def _scaling(case):
    return {"none": None, "linear": dict(kind="linear", factor=4.0),
            "yarn": dict(kind="yarn", factor=8.0, original=4096, beta_fast=32.0, beta_slow=1.0)}[case["scaling"]]


def _randn(g, shape, dtype, std=1.0):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).mul_(std).to(dtype)


def _cells(g, pages, page, heads, dim, dtype):
    out = torch.empty((pages, page, heads, dim), dtype=dtype, device="cuda")
    return out.normal_(generator=g)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed * 7919 + 13)
    dt = DT[case["dtype"]]
    s = {"case": case}
    if case["op"] == "matvec":
        n, k, gr = case["n"], case["k"], case["group"]
        s["codes"] = torch.randint(0, 256, (n, k // 2), generator=g, device="cuda", dtype=torch.uint8)
        s["scales"] = (torch.rand((n, k // gr), generator=g, device="cuda") * 0.02 + 0.002).to(dt)
        s["zeros"] = torch.randint(4, 12, (n, k // gr), generator=g, device="cuda", dtype=torch.uint8) if case["zeros"] else None
        s["x"] = _randn(g, (case["tokens"], k), dt)
        s["y"] = torch.empty((case["tokens"], n), dtype=dt, device="cuda")
        if own:  # a serving program lays its weights out once, when it loads them
            from expert_slot_cache_device_gb300.w4 import W4Weights

            s["weights"] = W4Weights(s["codes"], s["scales"], s["zeros"], group=gr)
        return s
    page, kv, dim = case["page"], case["kv_heads"], case["dim"]
    q, n = _lens(case)
    b, need = case["batch"], [-(-x // page) for x in n]
    extra = -(-case["budget"] // page) if case["op"] == "evict" else 0
    pages = sum(need) + b * extra + 3
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed))
    table = torch.zeros((b, max(need)), dtype=torch.int32)
    at = 0
    for i, m in enumerate(need):
        table[i, :m] = order[at:at + m]
        at += m
    s["k"], s["v"] = _cells(g, pages, page, kv, dim, dt), _cells(g, pages, page, kv, dim, dt)
    s["table"], s["lens"] = table.cuda(), torch.tensor(n, dtype=torch.int32, device="cuda")
    s["max_kv"], s["max_q"] = max(n), max(q)
    s["cu_q"] = torch.tensor([sum(q[:i]) for i in range(b + 1)], dtype=torch.int32, device="cuda")
    tokens = sum(q)
    if case["op"] == "append":
        freq, s["factor"] = _freq(case)
        if own:
            from expert_slot_cache_device_gb300.kv_cache import Rotary

            s["rotary"] = Rotary(dim, rot_dim=case["rot"], base=10000.0, layout=case["layout"], scaling=_scaling(case))
        else:  # the table that a program without the framework's plan keeps
            angle = torch.outer(torch.arange(MAX_POS, dtype=torch.float64, device="cuda"), freq.cuda())
            s["cos"], s["sin"] = (angle.cos() * s["factor"]).float(), (angle.sin() * s["factor"]).float()
        s["q"] = _randn(g, (tokens, case["heads"], dim), dt)
        s["new_k"], s["new_v"] = _randn(g, (tokens, kv, dim), dt), _randn(g, (tokens, kv, dim), dt)
        # positions run on from a start of their own: slots were evicted before
        start = torch.randint(0, MAX_POS - case["ctx"] - 1, (b,), generator=g, device="cuda")
        ends = torch.repeat_interleave(torch.tensor(n, device="cuda") - s["cu_q"][1:] + start, torch.tensor(q, device="cuda"))
        s["pos"] = (torch.arange(tokens, device="cuda") + ends).to(torch.int32)
        s["out"] = torch.empty_like(s["q"])
    elif case["op"] == "attend":
        s["q"] = _randn(g, (tokens, case["heads"], dim), dt, 1.5)
        s["sinks"] = torch.randn(case["heads"], generator=g, device="cuda") if case["sinks"] else None
        s["mass"] = torch.rand((b, kv, max(n)), generator=g, device="cuda") if case["mass"] else None
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty((tokens, case["heads"]), dtype=torch.float32, device="cuda")
    else:
        # a few tokens drew most of the weight, many drew none at all
        u = torch.rand((b, kv, max(n)), generator=g, device="cuda")
        s["mass"] = torch.where(u < 0.3, torch.zeros_like(u), u.pow(6).mul_(20.0))
        s["new_table"] = torch.zeros((b, extra), dtype=torch.int32)
        for i in range(b):
            s["new_table"][i] = order[at + i * extra:at + (i + 1) * extra]
        s["new_table"] = s["new_table"].cuda()
        s["kept"] = torch.empty((b, kv, case["budget"]), dtype=torch.int32, device="cuda")
        s["new_mass"] = torch.empty((b, kv, case["budget"]), dtype=torch.float32, device="cuda")
        s["new_lens"] = torch.empty(b, dtype=torch.int32, device="cuda")
    if own:
        from expert_slot_cache_device_gb300.kv_cache import KVBatch, PagedKVCache

        s["cache"] = PagedKVCache(pages, page, kv, dim, dtype=dt, k_pages=s["k"], v_pages=s["v"])
        s["batch"] = KVBatch(s["table"], s["lens"], s["cu_q"], max_q=s["max_q"], max_kv=s["max_kv"])
    return s


# ---------------------------------------------------------------- plain forms (32 bits)
def _owner(s, tokens):
    t = torch.arange(tokens, device="cuda")
    return t, torch.searchsorted(s["cu_q"][1:].contiguous(), t.to(torch.int32), right=True)


def _append(s):
    case = s["case"]
    rot, half = case["rot"], case["rot"] // 2
    c, w = (s[x][s["pos"].long()].unsqueeze(1) for x in ("cos", "sin"))

    def turned(x):
        x = x.float()
        r = x[..., :rot]
        a, b = (r[..., :half], r[..., half:]) if case["layout"] == "half" else (r[..., 0::2], r[..., 1::2])
        p, q = a * c - b * w, b * c + a * w
        r = torch.cat([p, q], -1) if case["layout"] == "half" else torch.stack([p, q], -1).flatten(-2)
        return torch.cat([r, x[..., rot:]], -1)

    t, seq = _owner(s, s["q"].shape[0])
    slot = (s["lens"] - s["cu_q"][1:])[seq].long() + t
    page = s["table"][seq, slot // case["page"]].long()
    s["k"][page, slot % case["page"]] = turned(s["new_k"]).to(s["k"].dtype)
    s["v"][page, slot % case["page"]] = s["new_v"]
    return {"q": turned(s["q"]).to(s["q"].dtype), "k": s["k"], "v": s["v"]}


def _attend(s):
    case = s["case"]
    b, kv, dim, page = case["batch"], case["kv_heads"], case["dim"], case["page"]
    rep, m, n = case["heads"] // case["kv_heads"], s["max_q"], s["max_kv"]
    t, seq = _owner(s, s["q"].shape[0])
    row = t - s["cu_q"][seq]
    q = torch.zeros((b, m, kv, rep, dim), device="cuda")
    q[seq, row] = s["q"].float().view(-1, kv, rep, dim)
    j = torch.arange(n, device="cuda")
    cell = s["table"][:, j // page].long() * page + j % page
    held = (j < s["lens"][:, None])[:, :, None, None]
    k, v = (torch.where(held, x.view(-1, kv, dim)[cell].float(), 0.0).permute(0, 2, 1, 3) for x in (s["k"], s["v"]))
    at = (s["lens"] - s["cu_q"][1:] + s["cu_q"][:-1])[:, None] + torch.arange(m, device="cuda")  # the queries' own slots
    sees = (j <= at[:, :, None]) & (at < s["lens"][:, None])[:, :, None]
    if case["window"]:
        sees = sees & (j > at[:, :, None] - case["window"])
    score = torch.matmul(q.permute(0, 2, 1, 3, 4).reshape(b, kv, m * rep, dim), k.transpose(2, 3))
    score = score.mul_(dim ** -0.5).view(b, kv, m, rep, n).masked_fill_(~sees[:, None, :, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    if case["sinks"]:
        top = torch.maximum(top, s["sinks"].view(1, kv, 1, rep, 1))
    top = torch.where(top == -math.inf, 0.0, top)
    p = score.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    if case["sinks"]:
        total = total + (s["sinks"].view(1, kv, 1, rep, 1) - top).exp()
    p = p.div_(torch.where(total == 0, 1.0, total))
    out = torch.matmul(p.view(b, kv, m * rep, n), v).view(b, kv, m, rep, dim).permute(0, 2, 1, 3, 4)[seq, row]
    lse = (total.log() + top).squeeze(-1).permute(0, 2, 1, 3)[seq, row]
    if case["mass"]:
        s["mass"] += p.sum((2, 3))
    return {"out": out.reshape(s["q"].shape).to(s["q"].dtype), "lse": lse.reshape(-1, case["heads"]), "mass": s["mass"]}


def _evict(s):
    case = s["case"]
    page, budget = case["page"], case["budget"]
    n = s["mass"].shape[2]
    j = torch.arange(n, device="cuda")
    lens = s["lens"][:, None, None]
    rank = torch.where(j >= lens - case["recent"], math.inf, s["mass"])
    rank = torch.where(j >= lens, -1.0, rank)
    take = min(budget, n)
    best = rank.sort(dim=-1, descending=True, stable=True).indices[..., :take]
    best = torch.where(best < lens, best, n).sort(dim=-1).values
    valid = best < n
    src = best.clamp(max=n - 1)
    b = torch.arange(case["batch"], device="cuda")[:, None, None]
    h = torch.arange(case["kv_heads"], device="cuda")[None, :, None]
    i = torch.arange(take, device="cuda")
    from_page, to_page = s["table"][b, src // page].long(), s["new_table"][b, i // page].long()
    at = [x[valid] for x in torch.broadcast_tensors(to_page, i % page, h)]
    got = [x[valid] for x in torch.broadcast_tensors(from_page, src % page, h)]
    s["k"][at[0], at[1], at[2]] = s["k"][got[0], got[1], got[2]]
    s["v"][at[0], at[1], at[2]] = s["v"][got[0], got[1], got[2]]
    s["kept"].fill_(-1)[..., :take] = torch.where(valid, best, -1).to(torch.int32)
    s["new_mass"].fill_(0.0)[..., :take] = torch.where(valid, s["mass"].gather(-1, src), 0.0)
    s["new_lens"].copy_(s["lens"].clamp(max=budget))
    return {"kept": s["kept"], "mass": s["new_mass"], "lens": s["new_lens"], "k": s["k"], "v": s["v"]}


def _matvec(s):
    case = s["case"]
    q = torch.stack([s["codes"] & 15, s["codes"] >> 4], -1).view(case["n"], -1, case["group"]).float()
    q = q - (s["zeros"].float().unsqueeze(-1) if case["zeros"] else 8.0)
    w = (q * s["scales"].float().unsqueeze(-1)).view(case["n"], case["k"])
    return {"y": torch.matmul(s["x"].float(), w.t()).to(s["x"].dtype)}


def run(s):
    op = s["case"]["op"]
    if not own:
        return {"append": _append, "attend": _attend, "evict": _evict, "matvec": _matvec}[op](s)
    if op == "append":
        s["cache"].append(s["batch"], s["rotary"], s["q"], s["new_k"], s["new_v"], s["pos"], q_out=s["out"])
        return {"q": s["out"], "k": s["k"], "v": s["v"]}
    if op == "attend":
        s["cache"].attend(s["batch"], s["q"], window=s["case"]["window"], sinks=s["sinks"], out=s["out"], lse=s["lse"],
                          mass=s["mass"])
        return {"out": s["out"], "lse": s["lse"], "mass": s["mass"]}
    if op == "evict":
        s["cache"].evict(s["batch"], s["mass"], s["new_table"], budget=s["case"]["budget"], recent=s["case"]["recent"],
                         kept=s["kept"], new_mass=s["new_mass"], new_lens=s["new_lens"])
        return {"kept": s["kept"], "mass": s["new_mass"], "lens": s["new_lens"], "k": s["k"], "v": s["v"]}
    s["weights"].matvec(s["x"], out=s["y"])
    return {"y": s["y"]}


# ---------------------------------------------------------------- the definitions, in 64 bits
def exact(case, seed):
    """Each operator from its definition, a sequence and a head at a time."""
    s = prepare(case, seed)
    if case["op"] == "matvec":
        code = torch.empty((case["n"], case["k"]), dtype=torch.float64, device="cuda")
        code[:, 0::2], code[:, 1::2] = s["codes"].remainder(16).double(), s["codes"].div(16, rounding_mode="floor").double()
        zero = s["zeros"].double() if case["zeros"] else torch.full_like(s["scales"], 8.0, dtype=torch.float64)
        y = torch.zeros((case["tokens"], case["n"]), dtype=torch.float64, device="cuda")
        for j in range(case["k"] // case["group"]):
            part = slice(j * case["group"], (j + 1) * case["group"])
            y += (s["x"][:, part].double() @ (code[:, part] - zero[:, j:j + 1]).T) * s["scales"][:, j].double()
        return {"y": y}
    q, n = _lens(case)
    page, kv = case["page"], case["kv_heads"]
    table = s["table"].cpu()
    cells = lambda i, m, tab: (tab[i, torch.arange(m) // page].long() * page + torch.arange(m) % page).cuda()  # noqa: E731
    flat_k, flat_v = s["k"].view(-1, kv, case["dim"]), s["v"].view(-1, kv, case["dim"])
    if case["op"] == "append":
        freq, factor = _freq(case)
        angle = s["pos"].double()[:, None] * freq.cuda()
        turn = torch.polar(torch.full_like(angle, factor), angle)[:, None, :]

        def rotate(x):
            x = x.double().clone()
            h = case["rot"] // 2
            first, second = (slice(0, h), slice(h, 2 * h)) if case["layout"] == "half" else (slice(0, 2 * h, 2), slice(1, 2 * h, 2))
            z = torch.complex(x[..., first].contiguous(), x[..., second].contiguous()) * turn
            x[..., first], x[..., second] = z.real, z.imag
            return x

        k, v, new_k, at = flat_k.double(), flat_v.double(), rotate(s["new_k"]), 0
        for i in range(case["batch"]):
            where = cells(i, n[i], table)[n[i] - q[i]:]
            k[where], v[where] = new_k[at:at + q[i]], s["new_v"][at:at + q[i]].double()
            at += q[i]
        return {"q": rotate(s["q"]), "k": k.view(s["k"].shape), "v": v.view(s["v"].shape)}
    if case["op"] == "evict":
        mass, new_mass = s["mass"].double(), torch.zeros(s["new_mass"].shape, dtype=torch.float64, device="cuda")
        k, v, new_table = flat_k.double(), flat_v.double(), s["new_table"].cpu()
        for i in range(case["batch"]):
            m = min(n[i], case["budget"])
            src, dst = cells(i, n[i], table), cells(i, m, new_table)
            for h in range(kv):
                old = n[i] - min(case["recent"], m)
                top = torch.argsort(-mass[i, h, :old], stable=True)[:m - (n[i] - old)]
                keep = torch.cat([top.sort().values, torch.arange(old, n[i], device="cuda")])
                k[dst, h], v[dst, h], new_mass[i, h, :m] = k[src[keep], h], v[src[keep], h], mass[i, h, keep]
        return {"kept": None, "mass": new_mass, "lens": None, "k": k.view(s["k"].shape), "v": v.view(s["v"].shape)}
    if 4 * _visible(case)[0] * case["heads"] * case["dim"] > 4e12:
        return None  # minutes in 64 bits
    rep, out, lse = case["heads"] // kv, s["q"].double(), torch.zeros(s["lse"].shape, dtype=torch.float64, device="cuda")
    mass, at = s["mass"].double() if case["mass"] else None, 0
    for i in range(case["batch"]):
        where = cells(i, n[i], table)
        own_slot = torch.arange(n[i] - q[i], n[i], device="cuda")[:, None]
        j = torch.arange(n[i], device="cuda")[None]
        hidden = (j > own_slot) | (j <= own_slot - (case["window"] or 1 << 40))
        for h in range(case["heads"]):
            k, v = flat_k[where, h // rep].double(), flat_v[where, h // rep].double()
            x = (s["q"][at:at + q[i], h].double() @ k.T / math.sqrt(case["dim"])).masked_fill(hidden, -math.inf)
            full = torch.cat([x, s["sinks"][h].double().expand(q[i], 1)], 1) if case["sinks"] else x
            lse[at:at + q[i], h] = torch.logsumexp(full, 1)
            p = torch.exp(x - lse[at:at + q[i], h, None])
            out[at:at + q[i], h] = p @ v
            if case["mass"]:
                mass[i, h // rep, :n[i]] += p.sum(0)
        at += q[i]
    return {"out": out, "lse": lse, "mass": mass}
