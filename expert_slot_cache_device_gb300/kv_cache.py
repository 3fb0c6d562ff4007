"""Paged key/value cache of a decoder layer's attention half, next to the expert slot cache.

``PagedKVCache`` owns (or wraps) the pages of one layer; ``KVBatch`` names the sequences of one
call and serves every layer of a step; ``Rotary`` holds the rotary frequencies. A step of a layer:

    q = cache.append(batch, rotary, q, k, v, positions)    # rotate, write K and V to their slots
    y = cache.attend(batch, q, mass=mass)                   # attention of the new tokens
    cache.evict(batch, mass, new_table, budget, recent)     # now and then: keep the heavy slots

Everything is computed by libftmoe through the C-ABI binding (``ftmoe``); PyTorch provides device
memory. Arguments are checked here and in the library before anything is enqueued; what only the
device can see (a page outside the cache, lengths out of range) is recorded in the cache's status
word (``status()``). Calls go to ``stream`` (the current stream by default) and do not wait.
"""
from __future__ import annotations

import ctypes
import math
import threading
from typing import Optional

import torch

from . import ftmoe as F
from .cache import _stream

_DTYPES = {torch.bfloat16: F.DT_BF16, torch.float16: F.DT_F16}
_F32 = torch.float32
_INT_MAX = 2 ** 31 - 1  # the C calls' integers
_KEPT = 256 << 20       # the largest workspace that a batch keeps, in bytes
# The current stream's handle without a Stream object around it (3 us of a call's 13 on the host)
_current = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _handle(stream, dev: int) -> int:
    """Handle of the stream of a call on memory of device `dev`. The library's kernels go to the current
    device, so that has to be it."""
    if _current_device() != dev:
        raise ValueError(f"memory of device {dev}: make it the current device first")
    if stream is None and _current is not None:
        return _current(dev)
    if getattr(stream, "device_index", dev) != dev:
        raise ValueError(f"memory of device {dev}, a stream of device {stream.device_index}")
    return _stream(stream)


def _new(shape, dtype, device, stream):
    """Device memory that the allocator does not hand out again while `stream` still uses it."""
    t = torch.empty(shape, dtype=dtype, device=device)
    if stream is not None:
        s = torch.cuda.ExternalStream(stream, device=device) if isinstance(stream, int) else stream
        if s != torch.cuda.current_stream(device):
            s.wait_stream(torch.cuda.current_stream(device))  # memory freed there may still be in use
            t.record_stream(s)
    return t


def _ints(t: torch.Tensor, name: str, dims: int, dev: Optional[int] = None) -> torch.Tensor:
    if not isinstance(t, torch.Tensor) or t.dtype != torch.int32 or not t.is_cuda or t.dim() != dims:
        raise ValueError(f"{name}: needs an int32 device tensor of {dims} dimension(s)")
    if dev is not None and t.get_device() != dev:
        raise ValueError(f"{name}: on device {t.get_device()}, the call's is {dev}")
    if t.numel() and t.stride(-1) != 1 and t.shape[-1] != 1:
        raise ValueError(f"{name}: needs consecutive elements")
    return t


def rotary_frequencies(rot_dim: int, base: float = 10000.0, scaling: Optional[dict] = None):
    """(frequencies in radians a position, fp64 [rot_dim / 2]; factor on the rotated part).

    f_i = base^(-2i / rot_dim); ``scaling`` stretches them for contexts beyond the trained length:

    None                                   f_i
    dict(kind="linear", factor=s)          f_i / s
    dict(kind="base", factor=s)            base * s^(rot_dim / (rot_dim - 2)) in place of base
    dict(kind="yarn", factor=s, original=n, beta_fast=32, beta_slow=1, attention_factor=None)
        pairs that turn more than beta_fast times in n positions keep f_i, those that turn less
        than beta_slow times get f_i / s, a linear ramp over the pair index blends between; the
        factor is attention_factor or 0.1 ln s + 1 (1 for s <= 1)
    dict(kind="banded", factor=s, original=n, low=1, high=4)
        with r = n f_i / 2 pi turns in n positions: f_i for r > high, f_i / s for r < low, and
        between, (1 - a) f_i / s + a f_i with a = (r - low) / (high - low)
    """
    if rot_dim <= 0 or rot_dim % 2:
        raise ValueError(f"rot_dim={rot_dim}: a positive even number")
    if not base > 1.0 or not math.isfinite(base):
        raise ValueError(f"base={base}: above 1")
    i = torch.arange(rot_dim // 2, dtype=torch.float64)
    freq = lambda b: torch.exp(i * (-2.0 / rot_dim * math.log(b)))  # noqa: E731
    if scaling is None:
        return freq(base), 1.0
    known = {"linear": {"factor"}, "base": {"factor"},
             "yarn": {"factor", "original", "beta_fast", "beta_slow", "attention_factor"},
             "banded": {"factor", "original", "low", "high"}}
    a = dict(scaling)
    kind = a.pop("kind", None)
    if kind not in known:
        raise ValueError(f"unknown rotary scaling {kind!r}")
    if set(a) - known[kind] or "factor" not in a or ("original" in known[kind] and "original" not in a):
        raise ValueError(f"rotary scaling {kind!r} takes {sorted(known[kind])}, got {sorted(a)}")
    s = float(a["factor"])
    if not s > 0 or not math.isfinite(s):
        raise ValueError(f"rotary scaling factor {s}")
    if kind == "linear":
        return freq(base) / s, 1.0
    if kind == "base":
        if rot_dim == 2:
            raise ValueError("base scaling needs rot_dim above 2")
        return freq(base * s ** (rot_dim / (rot_dim - 2))), 1.0
    f, n = freq(base), float(a["original"])
    if not n > 0:
        raise ValueError(f"original={n}")
    if kind == "banded":
        low, high = float(a.get("low", 1.0)), float(a.get("high", 4.0))
        if not high > low:
            raise ValueError("banded scaling needs high above low")
        t = ((n * f / (2 * math.pi) - low) / (high - low)).clamp(0, 1)
        return (1 - t) * f / s + t * f, 1.0
    fast, slow = float(a.get("beta_fast", 32.0)), float(a.get("beta_slow", 1.0))
    if not fast > slow > 0:
        raise ValueError("yarn scaling needs beta_fast above beta_slow above 0")
    pair = lambda turns: rot_dim * math.log(n / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
    lo, hi = max(math.floor(pair(fast)), 0), min(math.ceil(pair(slow)), rot_dim - 1)
    ramp = ((i - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
    att = a.get("attention_factor")
    att = float(att) if att is not None else (0.1 * math.log(s) + 1.0 if s > 1 else 1.0)
    return f * (1 - ramp) + f / s * ramp, att


class Rotary:
    """Rotary plan of a model: ``layout`` "half" (pairs (i, i + rot_dim / 2)) or "interleaved"
    (pairs (2i, 2i + 1)), on the first ``rot_dim`` elements of a head (all by default; a multiple
    of 16), ``scaling`` as in ``rotary_frequencies``."""

    def __init__(self, head_dim: int, rot_dim: Optional[int] = None, base: float = 10000.0, layout: str = "half",
                 scaling: Optional[dict] = None, device="cuda"):
        rot_dim = head_dim if rot_dim is None else rot_dim
        if layout not in ("half", "interleaved"):
            raise ValueError(f"layout {layout!r}: half or interleaved")
        if rot_dim % 16 or not 0 < rot_dim <= head_dim:
            raise ValueError(f"rot_dim={rot_dim}: a multiple of 16, at most head_dim={head_dim}")
        self.head_dim, self.rot_dim, self.layout = head_dim, rot_dim, layout
        freq, self.factor = rotary_frequencies(rot_dim, base, scaling)
        turns = freq / (2 * math.pi)
        hi = turns.to(torch.float32)
        self.freq = torch.stack([hi, (turns - hi.double()).to(torch.float32)], -1).contiguous().to(device)
        self._dev = self.freq.get_device()
        self._view = F.RotaryView(self.freq.data_ptr(), rot_dim, layout == "interleaved", self.factor)
        self.ref = ctypes.byref(self._view)


class KVBatch:
    """The sequences of one call.

    block_table  int32 [batch, pages]: page of each block of page_size slots
    kv_lens      int32 [batch]: cached tokens, this call's new ones included (the last of them)
    cu_q         int32 [batch + 1]: first row of each sequence's new tokens in the token arrays
    max_q        upper bound of the new tokens of one sequence
    max_kv       upper bound of kv_lens
    The tensors are read when the kernels run, so one object can serve a captured step whose
    lengths change within the bounds."""

    def __init__(self, block_table: torch.Tensor, kv_lens: torch.Tensor, cu_q: torch.Tensor, max_q: int, max_kv: int):
        self.block_table = _ints(block_table, "block_table", 2)
        self._dev = block_table.get_device()
        self.kv_lens, self.cu_q = _ints(kv_lens, "kv_lens", 1, self._dev), _ints(cu_q, "cu_q", 1, self._dev)
        self.batch = block_table.shape[0]
        if kv_lens.numel() != self.batch or cu_q.numel() != self.batch + 1:
            raise ValueError(f"{self.batch} sequences: kv_lens has {kv_lens.numel()}, cu_q {cu_q.numel()} entries")
        if not 0 <= max_q <= _INT_MAX or not 0 <= max_kv <= _INT_MAX:
            raise ValueError(f"max_q={max_q}, max_kv={max_kv}: outside [0, {_INT_MAX}]")
        self.max_q, self.max_kv = int(max_q), int(max_kv)
        self.device = block_table.device
        stride = block_table.stride(0) if self.batch > 1 else block_table.shape[1]
        self._args = (block_table.data_ptr(), stride, kv_lens.data_ptr(), cu_q.data_ptr(), self.batch)
        self._views, self._bytes, self._spaces = {}, {}, {}
        self._lock = threading.Lock()

    def _ref(self, tokens: int):
        """Reference to the C view for token arrays of `tokens` rows."""
        v = self._views.get(tokens)
        if v is None:
            v = F.KVBatchView(*self._args, tokens, self.max_q, self.max_kv, self.block_table.shape[1])
            v = self._views[tokens] = (ctypes.byref(v), v)
        return v[0]

    def _workspace(self, need: int, handle: int, stream) -> torch.Tensor:
        """At least ``need`` bytes for a call on stream ``handle``, kept for the next one there: a step's layers
        run one after another (an allocation a call takes 4 us of its 12 on the host). A large one is not
        kept: 64 sequences of 128k tokens with mass need 4 GB, and their call takes longer on the GPU than
        the allocation on the host. A captured call gets its own, which lives with the graph. The caller holds ``_lock`` until the call's kernels are
        enqueued: another thread's may not come between them, which share it."""
        if need > _KEPT or torch.cuda.is_current_stream_capturing():
            return _new(need, torch.uint8, self.device, stream)
        t = self._spaces.get(handle)
        if t is None or t.numel() < need:
            t = self._spaces[handle] = _new(need, torch.uint8, self.device, stream)
        return t


class PagedKVCache:
    """Keys and values of one layer in pages.

    num_pages, page_size (a power of two, 16..256), kv_heads, head_dim (attention: 64 or 128)
    k_pages, v_pages  optional device tensors [num_pages, page_size, kv_heads, head_dim] of
                      ``dtype`` (bfloat16 or float16) in any stride order with the last axis
                      contiguous; allocated here when omitted"""

    def __init__(self, num_pages: int, page_size: int, kv_heads: int, head_dim: int, dtype=torch.bfloat16,
                 k_pages: Optional[torch.Tensor] = None, v_pages: Optional[torch.Tensor] = None, device="cuda"):
        F.lib()
        if dtype not in _DTYPES:
            raise ValueError(f"dtype {dtype}: bfloat16 or float16")
        shape = (num_pages, page_size, kv_heads, head_dim)
        pages = []
        for name, t in (("k_pages", k_pages), ("v_pages", v_pages)):
            if t is None:
                t = torch.empty(shape, dtype=dtype, device=device)
            if tuple(t.shape) != shape or t.dtype != dtype or not t.is_cuda or t.stride(3) != 1:
                raise ValueError(f"{name}: needs a {dtype} device tensor {list(shape)} with a contiguous last axis")
            pages.append(t)
        self.k_pages, self.v_pages = pages
        self._dev = self.k_pages.get_device()
        if self.v_pages.get_device() != self._dev:
            raise ValueError("k_pages and v_pages are on different devices")
        self.num_pages, self.page_size, self.kv_heads, self.head_dim, self.dtype = *shape, dtype
        self.device = self.k_pages.device
        self._scale = head_dim ** -0.5
        self._status = torch.zeros(1, dtype=torch.int32, device=self.device)
        self._view = F.KVCacheView(self.k_pages.data_ptr(), self.v_pages.data_ptr(), *self.k_pages.stride()[:3],
                                   *self.v_pages.stride()[:3], _DTYPES[dtype], num_pages, page_size, kv_heads, head_dim,
                                   self._status.data_ptr())
        self._ref = ctypes.byref(self._view)

    def _rows(self, t: torch.Tensor, name: str, heads: Optional[int] = None, tokens: Optional[int] = None):
        """(reference to the C view of t [tokens, heads, head_dim], tokens, heads)."""
        if not isinstance(t, torch.Tensor) or t.dtype is not self.dtype or t.get_device() != self._dev or len(shape := t.shape) != 3:
            raise ValueError(f"{name}: needs a {self.dtype} tensor [tokens, heads, head_dim] on device {self._dev}")
        n, h, d = shape
        st, sh, sd = t.stride()
        if d != self.head_dim or sd != 1 or (heads is not None and h != heads) or (tokens is not None and n != tokens):
            raise ValueError(f"{name}: shape {list(t.shape)} does not match the call, or rows of head_dim are not contiguous")
        # a stride over one element is never taken
        return ctypes.byref(F.RowsView(t.data_ptr(), st if n > 1 else 8, sh if h > 1 else 8)), n, h

    def append(self, batch: KVBatch, rotary: Rotary, q: Optional[torch.Tensor], k: torch.Tensor, v: torch.Tensor,
               positions: torch.Tensor, q_out: Optional[torch.Tensor] = None, stream=None) -> Optional[torch.Tensor]:
        """Rotate q and k [tokens, heads, head_dim] by ``positions`` (int32 [tokens]) and write k
        and v to their slots. Returns the rotated queries (``q_out``, which may be q itself)."""
        if batch._dev != self._dev or rotary._dev != self._dev:
            raise ValueError(f"batch on device {batch._dev}, rotary plan on {rotary._dev}, cache on {self._dev}")
        if rotary.head_dim != self.head_dim:
            raise ValueError(f"rotary plan of head_dim {rotary.head_dim}, cache of {self.head_dim}")
        kr, n, _ = self._rows(k, "k", self.kv_heads)
        vr, _, _ = self._rows(v, "v", self.kv_heads, n)
        if _ints(positions, "positions", 1, self._dev).numel() != n:
            raise ValueError(f"positions has {positions.numel()} entries for {n} tokens")
        qr = qo = None
        heads = 0
        if q is not None:
            qr, _, heads = self._rows(q, "q", None, n)
            if q_out is None:
                q_out = _new(q.shape, q.dtype, q.device, stream)
            qo, _, _ = self._rows(q_out, "q_out", heads, n)
        if n == 0:
            return q_out
        F.ftmoe_rope_append(self._ref, batch._ref(n), rotary.ref, qr, qo, heads, kr, vr, positions.data_ptr(),
                            _handle(stream, self._dev))
        return q_out

    def attend(self, batch: KVBatch, q: torch.Tensor, scale: Optional[float] = None, window: int = 0,
               sinks: Optional[torch.Tensor] = None, causal: bool = True, out: Optional[torch.Tensor] = None,
               lse: Optional[torch.Tensor] = None, mass: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """Attention of the new tokens' queries [tokens, heads, head_dim] over their sequences'
        cached slots (``ftmoe_paged_attention``). ``scale`` defaults to head_dim ** -0.5,
        ``sinks`` is fp32 [heads], ``lse`` fp32 [tokens, heads] receives the log-sum-exp, ``mass``
        fp32 [batch, kv_heads, >= max_kv] gets each slot's attention weight added. A ``window`` of any
        size above the cached tokens is none. ``out`` may be q itself. Returns out."""
        if window > _INT_MAX:
            window = _INT_MAX
        if batch._dev != self._dev:
            raise ValueError(f"batch on device {batch._dev}, cache on {self._dev}")
        qr, n, heads = self._rows(q, "q")
        if heads % self.kv_heads:
            raise ValueError(f"{heads} query heads over {self.kv_heads} key heads")
        if out is None:
            out = _new(q.shape, q.dtype, q.device, stream)
        outr, _, _ = self._rows(out, "out", heads, n)
        if sinks is not None and (sinks.dtype is not _F32 or sinks.get_device() != self._dev or sinks.shape != (heads,) or not sinks.is_contiguous()):
            raise ValueError(f"sinks: needs a contiguous fp32 tensor [{heads}] on device {self._dev}")
        if lse is not None and (lse.dtype is not _F32 or lse.get_device() != self._dev or lse.shape != (n, heads) or not lse.is_contiguous()):
            raise ValueError(f"lse: needs a contiguous fp32 tensor [{n}, {heads}] on device {self._dev}")
        ms = mh = 0
        if mass is not None:
            ms, mh = self._mass(batch, mass)
        if n == 0:
            return out
        ref = batch._ref(n)
        key = (n, heads, self.kv_heads, self.head_dim, self.page_size, window, causal, mass is not None)
        need = batch._bytes.get(key)
        if need is None:
            need = batch._bytes[key] = F.ftmoe_paged_attention_workspace_bytes(self._ref, ref, heads, window, causal,
                                                                               mass is not None)
        handle = _handle(stream, self._dev)
        with batch._lock:
            ws = batch._workspace(need, handle, stream) if need else None
            F.ftmoe_paged_attention(self._ref, ref, qr, heads, self._scale if scale is None else scale, window, causal,
                                    sinks.data_ptr() if sinks is not None else None, outr,
                                    lse.data_ptr() if lse is not None else None,
                                    mass.data_ptr() if mass is not None else None, ms, mh,
                                    ws.data_ptr() if need else None, need, handle)
        return out

    def _mass(self, batch: KVBatch, mass: torch.Tensor):
        if mass.dtype is not _F32 or mass.get_device() != self._dev or mass.dim() != 3:
            raise ValueError(f"mass: needs an fp32 tensor [{batch.batch}, {self.kv_heads}, slots] on device {self._dev}")
        b, h, n = mass.shape
        ms, mh, m1 = mass.stride()
        if b != batch.batch or h != self.kv_heads or n < batch.max_kv or (n > 1 and m1 != 1):
            raise ValueError(f"mass: shape {list(mass.shape)}, needs [{batch.batch}, {self.kv_heads}, >= max_kv={batch.max_kv}] "
                             "with consecutive slots")
        if h == 1:
            mh = n
        if mh < n or (b > 1 and ms < n):
            raise ValueError("mass: rows overlap")
        return ms, mh

    def evict(self, batch: KVBatch, mass: torch.Tensor, new_table: torch.Tensor, budget: int, recent: int,
              kept: Optional[torch.Tensor] = None, new_mass: Optional[torch.Tensor] = None,
              new_lens: Optional[torch.Tensor] = None, stream=None):
        """Keep at most ``budget`` slots of each (sequence, key head): the last ``recent`` and
        those of largest mass (``ftmoe_kv_evict``), moved in order to the pages of ``new_table``
        (int32 [batch, pages], pages that ``block_table`` does not name). Returns (kept int32
        [batch, kv_heads, budget], new_mass fp32 likewise, new_lens int32 [batch]); the old
        pages can be reused by later work on the same stream."""
        if batch._dev != self._dev:
            raise ValueError(f"batch on device {batch._dev}, cache on {self._dev}")
        ms, mh = self._mass(batch, mass)
        if _ints(new_table, "new_table", 2, self._dev).shape[0] != batch.batch:
            raise ValueError(f"new_table has {new_table.shape[0]} rows for {batch.batch} sequences")
        shape = (batch.batch, self.kv_heads, budget)
        if budget < 1 or budget > _INT_MAX or recent > _INT_MAX:
            raise ValueError(f"budget={budget}, recent={recent}")
        if kept is None:
            kept = _new(shape, torch.int32, self.device, stream)
        if new_mass is None:
            new_mass = _new(shape, torch.float32, self.device, stream)
        if new_lens is None:
            new_lens = _new(batch.batch, torch.int32, self.device, stream)
        for name, t, sh, dt in (("kept", kept, shape, torch.int32), ("new_mass", new_mass, shape, _F32),
                                ("new_lens", new_lens, shape[:1], torch.int32)):
            if t.dtype is not dt or t.get_device() != self._dev or t.shape != sh or not t.is_contiguous():
                raise ValueError(f"{name}: needs a contiguous {dt} tensor {list(sh)} on device {self._dev}")
        # the C call takes one row length for every row
        if new_table.shape[1] * self.page_size < min(budget, batch.max_kv):
            raise ValueError(f"new_table: {new_table.shape[1]} pages a row for {min(budget, batch.max_kv)} slots")
        stride = new_table.stride(0) if batch.batch > 1 else new_table.shape[1]
        F.ftmoe_kv_evict(self._ref, batch._ref(0), mass.data_ptr(), ms, mh, budget, recent, new_table.data_ptr(), stride,
                         kept.data_ptr(), new_mass.data_ptr(), new_lens.data_ptr(), _handle(stream, self._dev))
        return kept, new_mass, new_lens

    def _on(self, stream):
        if stream is None:
            return torch.cuda.current_stream(self.device)
        return torch.cuda.ExternalStream(_stream(stream), device=self.device)

    def status(self, stream=None) -> int:
        """Sticky device status of this cache's calls (synchronises the stream)."""
        with torch.cuda.stream(self._on(stream)):
            return int(self._status.item())

    def reset_status(self, stream=None) -> None:
        with torch.cuda.stream(self._on(stream)):
            self._status.zero_()
