"""Latent attention next to the expert slot cache: a paged cache of one shared vector a token (a
normalised latent and one rotary key part that all heads share), and attention in both its forms.

``LatentCache`` owns (or wraps) the pages of one layer; ``KVBatch`` and ``Rotary`` are those of
``kv_cache``. A decode step of a layer works on the latents themselves (q went through the key
product):

    q_rope = cache.append(batch, rotary, c, k_rope, positions, weight=norm, q_rope=q_rope)
    o = cache.attend(batch, q, q_rope, scale)               # [tokens, heads, latent], then the value product

a chunk of a prompt on each head's keys and values, expanded from what was read back:

    rows = cache.read(batch, cu_rows)                       # [cached tokens, latent + rope]
    k, v = ...                                              # products of rows[:, :latent]
    o = expanded.attend(q, k, rows[:, latent:], v)          # expanded = ExpandedBatch(cu_q, cu_rows, ...)

Everything is computed by libftmoe through the C-ABI binding (``ftmoe``); PyTorch provides device
memory. Arguments are checked here and in the library before anything is enqueued; what only the
device can see (a page outside the cache, lengths out of range) is recorded in a status word
(``status()``). Calls go to ``stream`` (the current stream by default) and do not wait.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import ftmoe as F
from .kv_cache import _DTYPES, _F32, _INT_MAX, KVBatch, Rotary, Status, Workspaces, _handle, _ints, _new


def row_bytes(latent: int, rope: int, bits: int = 16) -> int:
    """Bytes of a cached token: 16-bit elements, or a byte a latent and one for each 32 of them (padded
    to 16 bytes), then the rotary part in 16 bits."""
    return 2 * (latent + rope) if bits == 16 else latent + (latent // 32 + 15) // 16 * 16 + 2 * rope


def _rows(t: torch.Tensor, name: str, dtype, dev: int, dim: int, heads: Optional[int] = None, tokens: Optional[int] = None):
    """(reference to the C view of t [tokens, heads, dim], tokens, heads)."""
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.get_device() != dev or len(shape := t.shape) != 3:
        raise ValueError(f"{name}: needs a {dtype} tensor [tokens, heads, {dim}] on device {dev}")
    n, h, d = shape
    st, sh, sd = t.stride()
    if d != dim or sd != 1 or (heads is not None and h != heads) or (tokens is not None and n != tokens):
        raise ValueError(f"{name}: shape {list(shape)}, needs [{tokens if tokens is not None else 'tokens'}, "
                         f"{heads if heads is not None else 'heads'}, {dim}] with a contiguous last axis")
    # a stride over one element is never taken
    return ctypes.byref(F.RowsView(t.data_ptr(), st if n > 1 else 8, sh if h > 1 else dim)), n, h


def _flat(t: torch.Tensor, name: str, dtype, dev: int, dim: int, rows: Optional[int] = None):
    """(address, row stride, rows) of t [rows, dim]."""
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.get_device() != dev or len(shape := t.shape) != 2:
        raise ValueError(f"{name}: needs a {dtype} tensor [rows, {dim}] on device {dev}")
    n, d = shape
    row, one = t.stride()
    if d != dim or one != 1 or (rows is not None and n != rows):
        raise ValueError(f"{name}: shape {list(shape)}, needs [{rows if rows is not None else 'rows'}, {dim}] with contiguous rows")
    return t.data_ptr(), row if n > 1 else dim, n


def _lse(t: Optional[torch.Tensor], n: int, heads: int, dev: int):
    if t is None:
        return None
    if t.dtype is not _F32 or t.get_device() != dev or t.shape != (n, heads) or not t.is_contiguous():
        raise ValueError(f"lse: needs a contiguous fp32 tensor [{n}, {heads}] on device {dev}")
    return t.data_ptr()


class LatentCache(Status):
    """Latents and shared rotary key parts of one layer in pages.

    num_pages, page_size (a power of two, 16..256)
    latent  a multiple of 128, at most 512; rope: a multiple of 16, at most 64
    bits    16: elements of ``dtype`` (bfloat16 or float16); 8: the latent as e4m3 codes with a power of
            two for each 32 of them, the rotary part in ``dtype`` (``row_bytes`` bytes a token)
    pages   optional device tensor, [num_pages, page_size, latent + rope] of ``dtype``, or uint8
            [num_pages, page_size, row_bytes(...)] for 8 bits, any strides with the last axis contiguous;
            allocated here when omitted"""

    def __init__(self, num_pages: int, page_size: int, latent: int, rope: int, dtype=torch.bfloat16, bits: int = 16,
                 pages: Optional[torch.Tensor] = None, device="cuda"):
        F.lib()
        if dtype not in _DTYPES:
            raise ValueError(f"dtype {dtype}: bfloat16 or float16")
        if bits not in (16, 8):
            raise ValueError(f"bits={bits}: 16 or 8")
        if latent % 128 or not 128 <= latent <= 512 or rope % 16 or not 16 <= rope <= 64:
            raise ValueError(f"latent={latent}: a multiple of 128, at most 512; rope={rope}: a multiple of 16, at most 64")
        shape = (num_pages, page_size, latent + rope if bits == 16 else row_bytes(latent, rope, bits))
        kind = dtype if bits == 16 else torch.uint8
        if pages is None:
            pages = torch.empty(shape, dtype=kind, device=device)
        if tuple(pages.shape) != shape or pages.dtype != kind or not pages.is_cuda or pages.stride(2) != 1:
            raise ValueError(f"pages: needs a {kind} device tensor {list(shape)} with a contiguous last axis")
        self.pages, self.device, self._dev = pages, pages.device, pages.get_device()
        self.num_pages, self.page_size, self.latent, self.rope, self.bits, self.dtype = num_pages, page_size, latent, rope, bits, dtype
        super().__init__(self.device)
        size = pages.element_size()
        self._view = F.LatentCacheView(pages.data_ptr(), pages.stride(0) * size, pages.stride(1) * size, _DTYPES[dtype], bits,
                                       num_pages, page_size, latent, rope, self._status.data_ptr())
        self._ref = ctypes.byref(self._view)

    def _on(self, batch: KVBatch):
        if batch._dev != self._dev:
            raise ValueError(f"batch on device {batch._dev}, cache on {self._dev}")

    def append(self, batch: KVBatch, rotary: Rotary, c: torch.Tensor, k_rope: torch.Tensor, positions: torch.Tensor,
               weight: Optional[torch.Tensor] = None, eps: float = 1e-6, q_rope: Optional[torch.Tensor] = None,
               q_out: Optional[torch.Tensor] = None, stream=None) -> Optional[torch.Tensor]:
        """Write the new tokens to their slots: ``c`` [tokens, latent], normalised by its root mean square and
        ``weight`` [latent] unless that is None, and ``k_rope`` [tokens, rope] turned by ``positions`` (int32
        [tokens]). Turns ``q_rope`` [tokens, heads, rope] too and returns it (``q_out``, which may be q_rope itself)."""
        self._on(batch)
        if rotary._dev != self._dev:
            raise ValueError(f"rotary plan on device {rotary._dev}, cache on {self._dev}")
        if rotary.rot_dim != self.rope:
            raise ValueError(f"rotary plan of rot_dim {rotary.rot_dim}, cache of rope {self.rope}")
        ca, cs, n = _flat(c, "c", self.dtype, self._dev, self.latent)
        ka, ks, _ = _flat(k_rope, "k_rope", self.dtype, self._dev, self.rope, n)
        if _ints(positions, "positions", 1, self._dev).numel() != n:
            raise ValueError(f"positions has {positions.numel()} entries for {n} tokens")
        if weight is not None and (weight.dtype is not self.dtype or weight.get_device() != self._dev or weight.shape != (self.latent,)
                                   or not weight.is_contiguous()):
            raise ValueError(f"weight: needs a contiguous {self.dtype} tensor [{self.latent}] on device {self._dev}")
        qr = qo = None
        heads = 0
        if q_rope is not None:
            qr, _, heads = _rows(q_rope, "q_rope", self.dtype, self._dev, self.rope, None, n)
            if q_out is None:
                q_out = _new(q_rope.shape, q_rope.dtype, q_rope.device, stream)
            qo, _, _ = _rows(q_out, "q_out", self.dtype, self._dev, self.rope, heads, n)
        if n == 0:
            return q_out
        F.ftmoe_latent_append(self._ref, batch._ref(n), rotary.ref, ca, cs, ka, ks, weight.data_ptr() if weight is not None else None,
                              eps, qr, qo, heads, positions.data_ptr(), _handle(stream, self._dev))
        return q_out

    def read(self, batch: KVBatch, cu_rows: torch.Tensor, rows: Optional[int] = None, out: Optional[torch.Tensor] = None,
             stream=None) -> torch.Tensor:
        """The cached tokens of every sequence as rows [latent + rope] of ``dtype``: slot j of sequence b in row
        ``cu_rows[b] + j`` (int32 [batch + 1]). Give ``out`` or its number of ``rows``. Returns out."""
        self._on(batch)
        if _ints(cu_rows, "cu_rows", 1, self._dev).numel() != batch.batch + 1:
            raise ValueError(f"cu_rows has {cu_rows.numel()} entries for {batch.batch} sequences")
        if out is None:
            if rows is None:
                raise ValueError("read needs out or rows")
            out = _new((rows, self.latent + self.rope), self.dtype, self.device, stream)
        oa, os_, n = _flat(out, "out", self.dtype, self._dev, self.latent + self.rope, rows)
        if n:
            F.ftmoe_latent_read(self._ref, batch._ref(0), cu_rows.data_ptr(), n, oa, os_, _handle(stream, self._dev))
        return out

    def attend(self, batch: KVBatch, q: torch.Tensor, q_rope: torch.Tensor, scale: float, causal: bool = True,
               out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """Absorbed attention of the new tokens' queries [tokens, heads, latent] and [tokens, heads, rope]
        over their sequences' cached tokens (``ftmoe_latent_attention``). ``lse`` fp32 [tokens, heads]
        receives the log-sum-exp; ``out`` may be q itself. Returns out [tokens, heads, latent]."""
        self._on(batch)
        qr, n, heads = _rows(q, "q", self.dtype, self._dev, self.latent)
        kr, _, _ = _rows(q_rope, "q_rope", self.dtype, self._dev, self.rope, heads, n)
        if out is None:
            out = _new(q.shape, q.dtype, q.device, stream)
        outr, _, _ = _rows(out, "out", self.dtype, self._dev, self.latent, heads, n)
        la = _lse(lse, n, heads, self._dev)
        if n == 0 or heads == 0:
            return out
        ref = batch._ref(n)
        key = ("latent", n, heads, self.latent, self.bits, self.page_size, causal)
        need = batch._bytes.get(key)
        if need is None:
            need = batch._bytes[key] = F.ftmoe_latent_attention_workspace_bytes(self._ref, ref, heads, causal)
        handle = _handle(stream, self._dev)
        with batch._lock:
            ws = batch._workspace(need, handle, stream) if need else None
            F.ftmoe_latent_attention(self._ref, ref, qr, kr, heads, scale, causal, outr, la, ws.data_ptr() if need else None, need, handle)
        return out


class ExpandedBatch(Workspaces, Status):
    """The sequences of expanded attention calls; one object serves every layer of a step.

    cu_q    int32 [batch + 1]: first row of each sequence's new tokens in the token arrays
    cu_kv   int32 [batch + 1]: first row of its keys and values, the new tokens' the last of them
    max_q   upper bound of the new tokens of one sequence, max_kv of its key rows (either may be above what a call has)
    The tensors are read when the kernels run."""

    def __init__(self, cu_q: torch.Tensor, cu_kv: torch.Tensor, max_q: int, max_kv: int):
        F.lib()
        self.cu_q = _ints(cu_q, "cu_q", 1)
        self._dev = cu_q.get_device()
        self.cu_kv = _ints(cu_kv, "cu_kv", 1, self._dev)
        self.batch = cu_q.numel() - 1
        if self.batch < 0 or cu_kv.numel() != self.batch + 1:
            raise ValueError(f"cu_q has {cu_q.numel()} entries, cu_kv {cu_kv.numel()}")
        if not 0 <= max_q <= _INT_MAX or not 0 <= max_kv <= _INT_MAX:
            raise ValueError(f"max_q={max_q}, max_kv={max_kv}: outside [0, {_INT_MAX}]")
        self.max_q, self.max_kv = int(max_q), int(max_kv)
        Workspaces.__init__(self, cu_q.device)
        Status.__init__(self, cu_q.device)
        self._refs = {}

    def _ref(self, n: int, m: int):
        ref = self._refs.get((n, m))
        if ref is None:
            ref = self._refs[n, m] = ctypes.byref(F.RowBatchView(self.cu_q.data_ptr(), self.cu_kv.data_ptr(), self.batch, n, m, self.max_q,
                                                                 min(self.max_kv, m), self._status.data_ptr()))
        return ref

    def attend(self, q: torch.Tensor, k: torch.Tensor, k_rope: torch.Tensor, v: torch.Tensor, scale: Optional[float] = None,
               causal: bool = True, out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """Attention of the new tokens' queries q [tokens, heads, nope + rope] over their sequences' rows k
        [rows, heads, nope], v [rows, heads, v_dim] and k_rope [rows, rope], which the heads share
        (``ftmoe_expanded_attention``; nope and v_dim both 128 or both 64). ``scale`` defaults to (nope + rope) ** -0.5.
        ``lse`` fp32 [tokens, heads] receives the log-sum-exp. Returns out [tokens, heads, v_dim]."""
        if q.dtype not in _DTYPES:
            raise ValueError(f"q: {q.dtype}, bfloat16 or float16")
        k_shape, v_shape, r_shape = k.shape, v.shape, k_rope.shape
        if len(k_shape) != 3 or len(v_shape) != 3 or len(r_shape) != 2:
            raise ValueError("k and v need three dimensions, k_rope two")
        dt, dev, nope, rope, vd = q.dtype, self._dev, k_shape[2], r_shape[1], v_shape[2]
        qr, n, heads = _rows(q, "q", dt, dev, nope + rope)
        kr, m, _ = _rows(k, "k", dt, dev, nope, heads)
        vr, _, _ = _rows(v, "v", dt, dev, vd, heads, m)
        ra, rs, _ = _flat(k_rope, "k_rope", dt, dev, rope, m)
        if out is None:
            out = _new((n, heads, vd), dt, self.device, stream)
        outr, _, _ = _rows(out, "out", dt, dev, vd, heads, n)
        la = _lse(lse, n, heads, dev)
        if n == 0 or heads == 0:
            return out
        ref = self._ref(n, m)
        key = (n, m, heads, nope, rope, vd, causal)
        need = self._bytes.get(key)
        if need is None:
            need = self._bytes[key] = F.ftmoe_expanded_attention_workspace_bytes(ref, _DTYPES[dt], heads, nope, rope, vd, causal)
        handle = _handle(stream, dev)
        with self._lock:
            ws = self._workspace(need, handle, stream) if need else None
            F.ftmoe_expanded_attention(ref, _DTYPES[dt], heads, nope, rope, vd, qr, kr, ra, rs, vr,
                                       (nope + rope) ** -0.5 if scale is None else scale, causal, outr, la,
                                       ws.data_ptr() if need else None, need, handle)
        return out
