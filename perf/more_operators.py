"""Operators of latent attention, next to the paged key/value cache: what is timed.

A model with latent attention caches one shared vector a token: a normalised latent, from which
every head's key and value are products, and one rotary part of the key that all heads share. Four
operators, as a program that serves such a model calls them:

* ``append``  norm of the new tokens' latents, rotary positions on the shared key part and on the
              queries' rotary parts; latent and key part go to the pages, in 16 bits or with the
              latent in 8 (e4m3 codes, a power of two for every 32). With 8 bits the pass goes on to
              read the sequences back, which is what the chunk that wrote them does next;
* ``read``    the cached tokens of every sequence as consecutive rows in 16 bits, the input of the
              product that expands latents to keys and values;
* ``attend``  the absorbed form: queries that went through the key product meet the latents
              themselves, which are keys and values of all heads at once;
* ``expand``  the expanded form, for chunks of a prompt: keys and values of each head as rows, with
              the rotary key part shared by the heads.

``run`` computes them with elementary torch operations in 32 bits where ``own`` is false, and
with the framework's calls where it is true. ``exact`` gives the same in 64 bits.
"""
import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16}
MAX_POS = 1 << 17
EPS = 1e-6
GROUP = 32  # latents that share a power of two in 8 bits


# ---------------------------------------------------------------- cases
def listed():
    lat = dict(latent=512, rope=64)
    return [
        # one new token for each of 64 running sequences: latency of a decode step
        dict(name="append step", op="append", batch=64, q=1, ctx=2000, heads=16, bits=16, layout="interleaved", scaling="yarn",
             page=64, dtype="bf16", **lat),
        # a ragged batch of prompt chunks, many query heads
        dict(name="append prompt", op="append", batch=3, q=4001, ctx=9000, heads=128, bits=16, layout="interleaved",
             scaling="yarn", page=64, dtype="bf16", **lat),
        # a chunk written to an 8-bit cache and read back with what came before it
        dict(name="append chunk 8 bits", op="append", batch=1, q=1777, ctx=6300, heads=32, bits=8, layout="half", scaling="none",
             page=16, dtype="bf16", **lat),
        # short ragged sequences read back for expansion
        dict(name="read ragged", op="read", batch=7, q=1, ctx=1500, bits=16, page=16, dtype="f16", latent=256, rope=32),
        # long sequences of an 8-bit cache read back
        dict(name="read long 8 bits", op="read", batch=8, q=1, ctx=30000, bits=8, page=64, dtype="bf16", **lat),
        # a single user's decode step on a short context: the smallest call
        dict(name="step short", op="attend", batch=1, q=1, ctx=777, heads=16, bits=16, page=16, dtype="bf16", **lat),
        # a decode batch over long caches, with as many heads as a large model has: as much arithmetic as memory
        dict(name="step batch", op="attend", batch=48, q=1, ctx=9000, heads=128, bits=16, page=64, dtype="bf16", **lat),
        # a decode batch over 8-bit caches
        dict(name="step batch 8 bits", op="attend", batch=96, q=1, ctx=7000, heads=32, bits=8, page=64, dtype="bf16", **lat),
        # four drafted tokens a sequence, checked at once
        dict(name="step draft", op="attend", batch=12, q=4, ctx=3300, heads=20, bits=16, page=32, dtype="f16", latent=256, rope=64),
        # short ragged chunks in one call
        dict(name="chunk ragged", op="expand", batch=5, q=301, ctx=1900, heads=20, nope=64, rope=32, vdim=64, dtype="f16"),
        # a whole prompt at once
        dict(name="chunk prompt", op="expand", batch=1, q=4096, ctx=4096, heads=32, nope=128, rope=64, vdim=128, dtype="bf16"),
        # a chunk of a long prompt late in its context: the call with the most arithmetic
        dict(name="chunk long", op="expand", batch=1, q=2048, ctx=25000, heads=16, nope=128, rope=64, vdim=128, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    """Spread over the logarithm, and off the large powers of two."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return v + (v % 512 == 0)


def draw(rng):
    op = rng.choice(["append", "read", "attend", "attend", "attend", "expand", "expand"])
    dtype = rng.choice(["bf16", "f16"])
    if op == "expand":
        q = _log(rng, 2, 2048)
        batch = _log(rng, 1, max(1.01, min(8.0, 2048 / q)))
        dims = rng.choice([dict(nope=128, rope=64, vdim=128), dict(nope=64, rope=32, vdim=64), dict(nope=64, rope=64, vdim=64)])
        case = dict(op=op, batch=batch, q=q, ctx=q + _log(rng, 1, 16000), heads=_log(rng, 1, 40), dtype=dtype, **dims)
        while work(case)["flops"] > 4e11:
            case["heads"] = max(1, case["heads"] // 2)
        return case
    case = dict(op=op, bits=rng.choice([16, 8]), page=rng.choice([16, 32, 64, 128]), dtype=dtype,
                latent=rng.choice([256, 512, 512]), rope=rng.choice([32, 64, 64]))
    if op == "read":
        return dict(case, batch=_log(rng, 1, 16), q=1, ctx=_log(rng, 1, 16000))
    if op == "append":
        q = 1 if rng.random() < 0.5 else _log(rng, 2, 4000)
        batch = _log(rng, 1, 64) if q == 1 else _log(rng, 1, 3)
        return dict(case, batch=batch, q=q, ctx=q + _log(rng, 1, 4000), heads=_log(rng, 1, 128),
                    layout=rng.choice(["half", "interleaved"]), scaling=rng.choice(["none", "yarn"]))
    kind, heads = rng.random(), _log(rng, 1, 128)
    if kind < 0.6:  # decode steps
        return dict(case, batch=_log(rng, 1, 64), q=1, ctx=_log(rng, 1, 10000), heads=heads)
    if kind < 0.85:  # drafted tokens
        q = rng.randint(2, 8)
        return dict(case, batch=_log(rng, 1, 16), q=q, ctx=q + _log(rng, 1, 6000), heads=heads)
    q = _log(rng, 9, 300)  # a short chunk that is not worth expanding
    return dict(case, batch=1, q=q, ctx=q + _log(rng, 1, 4000), heads=heads)


def _lens(case):
    """(new tokens, cached tokens with them) of each sequence: the first as long as the case
    says, the others shorter, at random but the same for the same case."""
    r = random.Random("%d %d %d" % (case["batch"], case["q"], case["ctx"]))
    q, n = [], []
    for i in range(case["batch"]):
        qi = case["q"] if i == 0 else r.randint(1, case["q"])
        ni = case["ctx"] if i == 0 else r.randint(qi, case["ctx"])
        q.append(qi)
        n.append(max(ni, qi))
    return q, n


def _stored(case):
    """Bytes of a cached token."""
    if case["bits"] == 16:
        return 2 * (case["latent"] + case["rope"])
    return case["latent"] + 16 * -(-case["latent"] // (16 * GROUP)) + 2 * case["rope"]


def work(case):
    q, n = _lens(case)
    tokens, cached = sum(q), sum(n)
    pairs = sum((2 * b - a + 1) * a // 2 for a, b in zip(q, n))
    if case["op"] == "expand":
        kd, vd = case["nope"] + case["rope"], case["vdim"]
        return {"bytes": tokens * case["heads"] * (2 * (kd + vd) + 4) + cached * 2 * (case["heads"] * (case["nope"] + vd) + case["rope"]),
                "flops": 2 * pairs * case["heads"] * (kd + vd)}
    row = 2 * (case["latent"] + case["rope"])
    if case["op"] == "read":
        return {"bytes": cached * (_stored(case) + row), "flops": 0}
    if case["op"] == "append":
        back = cached * (_stored(case) + row) if case["bits"] == 8 else 0
        return {"bytes": tokens * (row + _stored(case) + 4 * case["heads"] * case["rope"] + 4) + 2 * case["latent"] + back,
                "flops": tokens * (4 * case["latent"] + 3 * (case["heads"] + 1) * case["rope"])}
    return {"bytes": tokens * case["heads"] * (row + 2 * case["latent"] + 4) + cached * _stored(case),
            "flops": 2 * pairs * case["heads"] * (2 * case["latent"] + case["rope"])}


# ---------------------------------------------------------------- inputs
def _freq(case):
    """Rotary frequencies (radians a position, 64 bits) and the factor on the rotated part, as
    the framework's own plan defines them: base 10000; "yarn" divides by 8 the frequencies that
    turn less than once in 4096 positions, keeps those that turn more than 32 times, and blends
    between them, with the factor 0.1 ln 8 + 1."""
    rot = case["rope"]
    f = torch.arange(rot // 2, dtype=torch.float64).mul_(-2.0 / rot * math.log(10000.0)).exp_()
    if case["scaling"] == "none":
        return f, 1.0
    at = lambda turns: rot * math.log(4096 / (turns * 2 * math.pi)) / (2 * math.log(10000.0))  # noqa: E731
    lo, hi = max(math.floor(at(32.0)), 0), min(math.ceil(at(1.0)), rot - 1)
    ramp = ((torch.arange(rot // 2, dtype=torch.float64) - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
    return f * (1 - ramp) + f / 8.0 * ramp, 0.1 * math.log(8.0) + 1.0


def _randn(g, shape, dtype, std=1.0):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).mul_(std).to(dtype)


def _pages(case, g, pages):
    """Pages full of tokens: latents near N(0, 1), as a norm leaves them."""
    dt, latent, rope = DT[case["dtype"]], case["latent"], case["rope"]
    if case["bits"] == 16:
        return torch.empty((pages, case["page"], latent + rope), dtype=dt, device="cuda").normal_(generator=g)
    out = torch.zeros((pages, case["page"], _stored(case)), dtype=torch.uint8, device="cuda")
    for part in out.split(1 + (1 << 27) // (case["page"] * latent)):
        codes = torch.randn((*part.shape[:2], latent), generator=g, device="cuda").mul_(120.0).clamp_(-448, 448)
        part[..., :latent] = codes.to(torch.float8_e4m3fn).view(torch.uint8)
        part[..., latent:latent + latent // GROUP] = torch.randint(119, 122, (*part.shape[:2], latent // GROUP), generator=g,
                                                                   device="cuda", dtype=torch.uint8)
        part[..., -2 * rope:] = _randn(g, (*part.shape[:2], rope), dt).view(torch.uint8)
    return out


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed * 7919 + 13)
    dt = DT[case["dtype"]]
    s = {"case": case}
    q, n = _lens(case)
    b, tokens, cached = case["batch"], sum(q), sum(n)
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    s["lens"], s["max_kv"], s["max_q"] = ints(n), max(n), max(q)
    s["cu_q"], s["cu_rows"] = (ints([sum(x[:i]) for i in range(b + 1)]) for x in (q, n))
    if case["op"] == "expand":
        heads, nope, rope, vd = (case[x] for x in ("heads", "nope", "rope", "vdim"))
        s["q"] = _randn(g, (tokens, heads, nope + rope), dt, 1.5)
        kv = _randn(g, (cached, heads, nope + vd), dt)  # the expanding product's output: keys and values of a head side by side
        s["k"], s["v"] = kv[..., :nope], kv[..., nope:]
        s["k_rope"] = _randn(g, (cached, 4 * nope + rope), dt)[:, 4 * nope:]  # the rows that were read, latents before it
        s["out"] = torch.empty((tokens, heads, vd), dtype=dt, device="cuda")
        s["lse"] = torch.empty((tokens, heads), dtype=torch.float32, device="cuda")
        if own:
            from expert_slot_cache_device_gb300.latent_cache import ExpandedBatch

            s["batch"] = ExpandedBatch(s["cu_q"], s["cu_rows"], max_q=s["max_q"], max_kv=s["max_kv"])
        return s
    page, latent, rope = case["page"], case["latent"], case["rope"]
    need = [-(-x // page) for x in n]
    pages = sum(need) + 3
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed))
    table = torch.zeros((b, max(need)), dtype=torch.int32)
    for i, m in enumerate(need):
        table[i, :m] = order[sum(need[:i]):sum(need[:i + 1])]
    s["table"], s["pages"] = table.cuda(), _pages(case, g, pages)
    if case["op"] == "append":
        freq, s["factor"] = _freq(case)
        if own:
            from expert_slot_cache_device_gb300.kv_cache import Rotary

            s["rotary"] = Rotary(rope, base=10000.0, layout=case["layout"], scaling=None if case["scaling"] == "none" else
                                 dict(kind="yarn", factor=8.0, original=4096, beta_fast=32.0, beta_slow=1.0))
        else:  # the table that a program without the framework's plan keeps
            angle = torch.outer(torch.arange(MAX_POS, dtype=torch.float64, device="cuda"), freq.cuda())
            s["cos"], s["sin"] = (angle.cos() * s["factor"]).float(), (angle.sin() * s["factor"]).float()
        down = _randn(g, (tokens, latent + rope), dt, 2.0)  # the down product's output: latent and rotary part side by side
        s["c"], s["k_rope"] = down[:, :latent], down[:, latent:]
        s["weight"] = (torch.rand(latent, generator=g, device="cuda") + 0.5).to(dt)
        s["q"] = _randn(g, (tokens, case["heads"], 2 * rope), dt)[..., rope:]  # the rotary part of wider heads
        # positions run on from a start of their own
        start = torch.randint(0, MAX_POS - case["ctx"] - 1, (b,), generator=g, device="cuda")
        s["pos"] = (torch.arange(tokens, device="cuda") + torch.repeat_interleave(start - s["cu_q"][:-1], ints(q).long())).to(torch.int32)
        s["out"] = torch.empty((tokens, case["heads"], rope), dtype=dt, device="cuda")
    if case["op"] == "attend":
        s["q"], s["q_rope"] = _randn(g, (tokens, case["heads"], latent), dt), _randn(g, (tokens, case["heads"], 2 * rope), dt)[..., rope:]
        s["scale"] = (latent // 4 + rope) ** -0.5
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty((tokens, case["heads"]), dtype=torch.float32, device="cuda")
    else:
        s["rows"] = torch.empty((cached, latent + rope), dtype=dt, device="cuda")
    if own:
        from expert_slot_cache_device_gb300.kv_cache import KVBatch
        from expert_slot_cache_device_gb300.latent_cache import LatentCache

        s["cache"] = LatentCache(pages, page, latent, rope, dtype=dt, bits=case["bits"], pages=s["pages"])
        s["batch"] = KVBatch(s["table"], s["lens"], s["cu_q"], max_q=s["max_q"], max_kv=s["max_kv"])
    return s


# ---------------------------------------------------------------- plain forms (32 bits)
def _decode(s, cells):
    """Cached tokens as they are stored -> (latents in the cache's 16-bit type, rotary parts)."""
    case = s["case"]
    latent, dt = case["latent"], DT[case["dtype"]]
    if case["bits"] == 16:
        return cells[..., :latent], cells[..., latent:]
    code = cells[..., :latent].contiguous().view(torch.float8_e4m3fn).float()
    e = cells[..., latent:latent + latent // GROUP].to(torch.int32)
    power = torch.where(e == 0, 2.0 ** -127, (e << 23).view(torch.float32))
    c = (code.unflatten(-1, (-1, GROUP)) * power.unsqueeze(-1)).flatten(-2).to(dt)
    return c, cells[..., -2 * case["rope"]:].contiguous().view(dt)


def _encode(case, y):
    """Latents in 16 bits -> codes and the powers of two: the least with amax <= 448 times it."""
    x = y.float().unflatten(-1, (-1, GROUP))
    if case["dtype"] == "f16":
        x = x.clamp(-61440, 61440)  # the largest codes times powers of two that binary16 holds
    m, k = torch.frexp(x.abs().amax(-1))
    e = torch.where(m == 0, 0, k - 9 + (m > 0.875).int() + 127).clamp(0, 254).to(torch.int32)
    up = torch.where(e == 254, 2.0 ** -127, ((254 - e) << 23).view(torch.float32))
    return (x * up.unsqueeze(-1)).flatten(-2).to(torch.float8_e4m3fn).view(torch.uint8), e.to(torch.uint8)


def _owner(s, starts, rows):
    """Sequence of each of `rows` rows, and the row's number in it."""
    t = torch.arange(rows, device="cuda")
    seq = torch.searchsorted(starts[1:].contiguous(), t.to(torch.int32), right=True)
    return seq, t - starts[seq]


def _cell(s, seq, slot):
    page = s["case"]["page"]
    return s["table"][seq, slot // page].long(), slot % page


def _read(s):
    seq, slot = _owner(s, s["cu_rows"], s["rows"].shape[0])
    return {"rows": torch.cat(_decode(s, s["pages"][_cell(s, seq, slot)]), -1)}


def _append(s):
    case = s["case"]
    half, dt = case["rope"] // 2, DT[case["dtype"]]
    c, w = (s[x][s["pos"].long()] for x in ("cos", "sin"))

    def turned(x, c, w):
        x = x.float()
        a, b = (x[..., :half], x[..., half:]) if case["layout"] == "half" else (x[..., 0::2], x[..., 1::2])
        p, q = a * c - b * w, b * c + a * w
        return (torch.cat([p, q], -1) if case["layout"] == "half" else torch.stack([p, q], -1).flatten(-2)).to(dt)

    x = s["c"].float()
    y = (x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * s["weight"].float()).to(dt)
    key = turned(s["k_rope"], c, w)
    if case["bits"] == 16:
        rows = torch.cat([y, key], -1)
    else:
        codes, e = _encode(case, y)
        pad = torch.zeros((len(e), _stored(case) - case["latent"] - e.shape[1] - 2 * case["rope"]), dtype=torch.uint8, device="cuda")
        rows = torch.cat([codes, e, pad, key.view(torch.uint8)], -1)
    seq, i = _owner(s, s["cu_q"], len(y))
    new = s["cu_q"][1:] - s["cu_q"][:-1]
    s["pages"][_cell(s, seq, i + (s["lens"] - new)[seq])] = rows
    out = {"q": turned(s["q"], c.unsqueeze(1), w.unsqueeze(1))}
    return dict(out, **(_read(s) if case["bits"] == 8 else {"pages": s["pages"]}))


def _softmax(s, score):
    """Scores [batch, heads, new tokens, slots]; (their softmax over what each token sees, its log-sum-exp)."""
    m, n = score.shape[2:]
    new = (s["cu_q"][1:] - s["cu_q"][:-1])[:, None]
    at = s["lens"][:, None] - new + torch.arange(m, device="cuda")
    sees = (torch.arange(n, device="cuda") <= at[:, :, None]) & (at < s["lens"][:, None])[:, :, None]
    score.masked_fill_(~sees[:, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = score.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    return p.div_(torch.where(total == 0, 1.0, total)), (total.log() + top).squeeze(-1)


def _queries(s, *parts):
    """Queries in 32 bits, a sequence's new tokens padded to the longest: [batch, heads, new tokens, elements]."""
    seq, i = _owner(s, s["cu_q"], parts[0].shape[0])
    dim = sum(x.shape[2] for x in parts)
    q = torch.zeros((s["case"]["batch"], s["max_q"], s["case"]["heads"], dim), device="cuda")
    q[seq, i] = torch.cat([x.float() for x in parts], -1)
    return q.transpose(1, 2), seq, i


def _attend(s):
    case = s["case"]
    q, seq, i = _queries(s, s["q"], s["q_rope"])
    b, h, m, n = case["batch"], case["heads"], s["max_q"], s["max_kv"]
    slot = torch.arange(n, device="cuda")
    held = (slot < s["lens"][:, None])[..., None]
    c, key = _decode(s, s["pages"][_cell(s, torch.arange(b, device="cuda")[:, None], slot)])
    k = torch.where(held, torch.cat([c.float(), key.float()], -1), 0.0)
    score = torch.matmul(q.reshape(b, h * m, -1), k.transpose(1, 2)).mul_(s["scale"])
    p, lse = _softmax(s, score.view(b, h, m, n))
    out = torch.matmul(p.view(b, h * m, n), k[..., :case["latent"]]).view(b, h, m, -1)
    return {"out": out.transpose(1, 2)[seq, i].to(s["q"].dtype), "lse": lse.transpose(1, 2)[seq, i]}


def _expand(s):
    q, seq, i = _queries(s, s["q"])
    slot = torch.arange(s["max_kv"], device="cuda")
    held = slot < s["lens"][:, None]
    row = torch.where(held, s["cu_rows"][:-1, None] + slot, 0).long()
    heads = s["case"]["heads"]
    k = torch.cat([s["k"][row].float(), s["k_rope"][row].float().unsqueeze(2).expand(-1, -1, heads, -1)], -1)
    k, v = (torch.where(held[:, :, None, None], x, 0.0).transpose(1, 2) for x in (k, s["v"][row].float()))
    p, lse = _softmax(s, torch.matmul(q, k.transpose(2, 3)).mul_(q.shape[-1] ** -0.5))
    out = torch.matmul(p, v)
    return {"out": out.transpose(1, 2)[seq, i].to(s["q"].dtype), "lse": lse.transpose(1, 2)[seq, i]}


def run(s):
    case = s["case"]
    op = case["op"]
    if not own:
        return {"append": _append, "read": _read, "attend": _attend, "expand": _expand}[op](s)
    if op == "append":
        s["cache"].append(s["batch"], s["rotary"], s["c"], s["k_rope"], s["pos"], weight=s["weight"], eps=EPS, q_rope=s["q"],
                          q_out=s["out"])
        if case["bits"] == 16:
            return {"q": s["out"], "pages": s["pages"]}
        return {"q": s["out"], "rows": s["cache"].read(s["batch"], s["cu_rows"], out=s["rows"])}
    if op == "read":
        return {"rows": s["cache"].read(s["batch"], s["cu_rows"], out=s["rows"])}
    if op == "attend":
        s["cache"].attend(s["batch"], s["q"], s["q_rope"], s["scale"], out=s["out"], lse=s["lse"])
    else:
        s["batch"].attend(s["q"], s["k"], s["k_rope"], s["v"], out=s["out"], lse=s["lse"])
    return {"out": s["out"], "lse": s["lse"]}


# ---------------------------------------------------------------- the definitions, in 64 bits
def exact(case, seed):
    """Each operator from its definition, a sequence (and a head) at a time."""
    s = prepare(case, seed)
    q, n = _lens(case)
    if case["op"] in ("attend", "expand") and work(case)["flops"] > 4e12:
        return None  # too long in 64 bits
    if case["op"] != "expand":
        table, page, latent, rope, dt = s["table"].cpu(), case["page"], case["latent"], case["rope"], DT[case["dtype"]]
        flat = s["pages"].view(-1, s["pages"].shape[-1])
        where = [(table[i, torch.arange(m) // page].long() * page + torch.arange(m) % page).cuda() for i, m in enumerate(n)]

        def value(rows):
            """(latents, rotary parts) of stored rows: sign, exponent and fraction of each code."""
            if case["bits"] == 16:
                return rows[:, :latent].double(), rows[:, latent:].double()
            code = rows[:, :latent].long()
            exp, frac = code // 8 % 16, code % 8
            mag = torch.where(exp == 0, frac * 2.0 ** -9, torch.ldexp(1 + frac.double() / 8, exp - 7))
            power = torch.exp2(rows[:, latent:latent + latent // GROUP].double() - 127)
            c = torch.where(code >= 128, -mag, mag) * power.repeat_interleave(GROUP, 1)
            return c.to(dt).double(), rows[:, -2 * rope:].contiguous().view(dt).double()

    if case["op"] == "read":
        return {"rows": torch.cat([torch.cat(value(flat[w]), 1) for w in where])}
    if case["op"] == "append":
        freq, factor = _freq(case)
        angle = s["pos"].double()[:, None] * freq.cuda()
        turn = torch.polar(torch.full_like(angle, factor), angle)

        def rotate(x, turn):
            x = x.double().clone()
            h = rope // 2
            first, second = (slice(0, h), slice(h, None)) if case["layout"] == "half" else (slice(0, None, 2), slice(1, None, 2))
            z = torch.complex(x[..., first].contiguous(), x[..., second].contiguous()) * turn
            x[..., first], x[..., second] = z.real, z.imag
            return x

        x = s["c"].double()
        y = s["weight"].double() * x / torch.sqrt((x * x).sum(1, keepdim=True) / latent + EPS)
        if case["bits"] == 8:  # the definition rounds to 16 bits first
            y = y.to(dt).double().view(len(x), -1, GROUP)
            power = torch.exp2(torch.ceil(torch.log2(y.abs().amax(2, keepdim=True) / 448)).clamp(-127, 127))
            z = (y / power).abs()  # three fraction bits from 2^-6 up, steps of 2^-9 below
            step = torch.exp2(torch.floor(torch.log2(z.clamp(min=2.0 ** -6))) - 3)
            y = (torch.sign(y) * torch.round(z / step) * step * power).view(len(x), -1).to(dt).double()
        new, at, out = torch.cat([y, rotate(s["k_rope"], turn)], 1), 0, {"q": rotate(s["q"], turn[:, None])}
        stored = [torch.cat(value(flat[w]), 1) for w in where] if case["bits"] == 8 else flat.double()
        for i in range(case["batch"]):
            if case["bits"] == 8:
                stored[i][n[i] - q[i]:] = new[at:at + q[i]]
            else:
                stored[where[i][n[i] - q[i]:]] = new[at:at + q[i]]
            at += q[i]
        return dict(out, rows=torch.cat(stored)) if case["bits"] == 8 else dict(out, pages=stored.view(s["pages"].shape))
    out, lse = s["out"].double(), torch.zeros(s["lse"].shape, dtype=torch.float64, device="cuda")
    scale = s["scale"] if case["op"] == "attend" else (case["nope"] + case["rope"]) ** -0.5
    at = row = 0
    for i in range(case["batch"]):
        slot = torch.arange(n[i], device="cuda")
        hidden = slot[None] > torch.arange(n[i] - q[i], n[i], device="cuda")[:, None]
        if case["op"] == "attend":
            c, key = value(flat[where[i]])
        for h in range(case["heads"]):
            a = slice(at, at + q[i])
            if case["op"] == "attend":
                x, v = s["q"][a, h].double() @ c.T + s["q_rope"][a, h].double() @ key.T, c
            else:
                r = slice(row, row + n[i])
                k = torch.cat([s["k"][r, h], s["k_rope"][r]], 1).double()
                x, v = s["q"][a, h].double() @ k.T, s["v"][r, h].double()
            x = (x * scale).masked_fill(hidden, -math.inf)
            lse[a, h] = torch.logsumexp(x, 1)
            out[a, h] = torch.exp(x - lse[a, h, None]) @ v
        at, row = at + q[i], row + n[i]
    return {"out": out, "lse": lse}
