"""One decoder layer of a mixture-of-experts model, served from the expert slot cache: 4-bit
projections, rotary positions and the write to the paged key/value cache, attention of the new
tokens, eviction by attention mass, and the routed experts from their slots.

    python examples/decoder_layer.py

runs a prompt in two chunks, single-token steps and an eviction on synthetic weights. The norms, the
router and the residual sums are plain torch; everything else is the framework's.
"""
from __future__ import annotations

import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

from expert_slot_cache_device_gb300.cache import Bank, ExpertSlotCache  # noqa: E402
from expert_slot_cache_device_gb300.kv_cache import KVBatch, PagedKVCache, Rotary  # noqa: E402
from expert_slot_cache_device_gb300.w4 import W4Weights  # noqa: E402

BF16 = torch.bfloat16


def norm(x: torch.Tensor) -> torch.Tensor:
    f = x.float()
    return (f * torch.rsqrt(f.square().mean(-1, keepdim=True) + 1e-6)).to(x.dtype)


class DecoderLayer:
    """Weights and caches of one layer. ``experts`` is an ExpertSlotCache whose layer 0 this is."""

    def __init__(self, experts: ExpertSlotCache, topk: int, heads: int, kv_heads: int, head_dim: int, pages: int,
                 page_size: int, wqkv: W4Weights, wo: W4Weights, router: torch.Tensor, rotary: Rotary):
        self.experts, self.topk, self.heads, self.kv_heads, self.dim = experts, topk, heads, kv_heads, head_dim
        self.wqkv, self.wo, self.router, self.rotary = wqkv, wo, router, rotary
        self.cache = PagedKVCache(pages, page_size, kv_heads, head_dim)

    def forward(self, x: torch.Tensor, batch: KVBatch, positions: torch.Tensor, mass: torch.Tensor) -> torch.Tensor:
        """New tokens x [tokens, hidden] of the batch's sequences; adds to ``mass`` the attention
        weight that each cached token draws."""
        n = x.shape[0]
        qkv = self.wqkv.matvec(norm(x)).view(n, self.heads + 2 * self.kv_heads, self.dim)
        q, k, v = qkv.split([self.heads, self.kv_heads, self.kv_heads], 1)
        q = self.cache.append(batch, self.rotary, q, k, v, positions)
        y = self.cache.attend(batch, q, mass=mass)
        x = x + self.wo.matvec(y.view(n, -1))
        h = norm(x)
        weights, ids = torch.softmax(h.float() @ self.router.T, -1).topk(self.topk)
        weights = weights / weights.sum(-1, keepdim=True)
        ids, slots, out = ids.to(torch.int32), torch.empty((n, self.topk), dtype=torch.int32, device=x.device), torch.empty_like(x)
        self.experts.ensure(0, ids, slots)
        self.experts.copy_missing()
        self.experts.ffn(h, slots, weights.contiguous(), out)
        return x + out


def synthetic_layer(hidden=256, inter=128, experts=8, topk=2, heads=8, kv_heads=2, head_dim=64, pages=64, page_size=16,
                    max_tokens=96, seed=0):
    """A layer with random weights, and the plain weights by name."""
    g = torch.Generator().manual_seed(seed)

    def w4(n, k, group=64):
        codes = torch.randint(0, 256, (n, k // 2), generator=g, dtype=torch.uint8)
        scales = ((torch.rand((n, k // group), generator=g) + 0.5) * 0.25 * k ** -0.5).to(BF16)
        return codes, scales

    plain = {"qkv": w4((heads + 2 * kv_heads) * head_dim, hidden), "o": w4(hidden, heads * head_dim),
             "router": torch.randn((experts, hidden), generator=g) * hidden ** -0.5,
             "gate_up": (torch.randn((experts, 2 * inter, hidden), generator=g) * hidden ** -0.5).to(BF16),
             "down": (torch.randn((experts, hidden, inter), generator=g) * inter ** -0.5).to(BF16)}
    banks = [Bank("gate_up", "bf16", 2 * inter, 2 * hidden), Bank("down", "bf16", hidden, 2 * inter)]
    host = [[plain[b.name].reshape(-1).view(torch.uint8).pin_memory()] for b in banks]
    cache = ExpertSlotCache("bf16", experts, 1, experts, hidden, inter, banks, host, max_pairs=max_tokens * topk)
    packed = {k: W4Weights(plain[k][0].cuda(), plain[k][1].cuda(), group=64) for k in ("qkv", "o")}
    layer = DecoderLayer(cache, topk, heads, kv_heads, head_dim, pages, page_size, packed["qkv"], packed["o"],
                         plain["router"].cuda(), Rotary(head_dim))
    return layer, plain


class Sequences:
    """Block tables, lengths and positions of a few sequences: what a scheduler would keep."""

    def __init__(self, layer: DecoderLayer, count: int, max_tokens: int):
        self.page, self.free = layer.cache.page_size, list(range(layer.cache.num_pages))
        self.width = -(-max_tokens // self.page)
        self.tables, self.lens, self.seen = [[] for _ in range(count)], [0] * count, [0] * count
        self.mass = torch.zeros((count, layer.kv_heads, max_tokens), device="cuda")

    def table(self, rows):
        t = torch.zeros((len(rows), self.width), dtype=torch.int32)
        for i, r in enumerate(rows):
            t[i, :len(r)] = torch.tensor(r, dtype=torch.int32)
        return t.cuda()

    def grow(self, new):
        """Room for new[i] more tokens of each sequence; the batch and their positions."""
        pos = []
        for i, n in enumerate(new):
            pos += range(self.seen[i], self.seen[i] + n)
            self.lens[i] += n
            self.seen[i] += n
            while len(self.tables[i]) * self.page < self.lens[i]:
                self.tables[i].append(self.free.pop())
        cu = torch.tensor([0] + new, dtype=torch.int32).cumsum(0).to(torch.int32)
        batch = KVBatch(self.table(self.tables), torch.tensor(self.lens, dtype=torch.int32).cuda(), cu.cuda(), max(new), max(self.lens))
        return batch, torch.tensor(pos, dtype=torch.int32).cuda()

    def evict(self, layer: DecoderLayer, batch: KVBatch, budget: int, recent: int):
        """Cut every cache to at most `budget` tokens, in pages of its own; the old pages are free
        again for later work on the stream."""
        new = [[self.free.pop() for _ in range(-(-min(n, budget) // self.page))] for n in self.lens]
        kept, mass, _ = layer.cache.evict(batch, self.mass, self.table(new), budget, recent)
        for row in self.tables:
            self.free += row
        self.tables, self.lens = new, [min(n, budget) for n in self.lens]
        self.mass.zero_()[:, :, :budget] = mass
        return kept


def main():
    layer, _ = synthetic_layer()
    seqs = Sequences(layer, 3, 256)
    g = torch.Generator().manual_seed(1)
    tokens = lambda n: torch.randn((n, 256), generator=g).to(BF16).cuda()  # noqa: E731
    for new in ([40, 17, 5], [30, 1, 25]):  # prompts, in two chunks
        batch, pos = seqs.grow(new)
        x = layer.forward(tokens(sum(new)), batch, pos, seqs.mass)
    x = x[[sum(new[:i + 1]) - 1 for i in range(3)]]
    for step in range(24):
        batch, pos = seqs.grow([1, 1, 1])
        x = layer.forward(norm(x), batch, pos, seqs.mass)
        if step == 11:
            kept = seqs.evict(layer, batch, budget=32, recent=8)
            print("evicted to", seqs.lens, "first slots kept by sequence 0, head 0:", kept[0, 0, :8].tolist())
    torch.cuda.synchronize()
    assert layer.cache.status() == 0 and layer.experts.status() == 0 and torch.isfinite(x).all()
    print("cached tokens", seqs.lens, "of", seqs.seen, "seen; output norm", [round(float(v), 3) for v in x.float().norm(dim=-1)])
    layer.experts.close()


if __name__ == "__main__":
    main()
