"""Dense projections with 4-bit weights: w = (code - zero) * scale, one scale (and zero) per
``group`` consecutive k of a row. ``W4Weights`` lays the codes out once for the product kernel;
``matvec`` multiplies a decode batch. Computed by libftmoe (``ftmoe_w4_matvec``)."""
from __future__ import annotations

from typing import Optional

import torch

from . import ftmoe as F
from .kv_cache import _DTYPES, _handle, _new


class W4Weights:
    """codes   uint8 [N, K / 2], low nibble = even k
    scales  bfloat16 or float16 [N, K / group]; x and y have the same type
    zeros   uint8 [N, K / group] with values 0..15, or None for 8
    group   32, 64 or 128
    The plain arrays may be freed afterwards (by work on the same stream)."""

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, zeros: Optional[torch.Tensor] = None,
                 group: int = 128, stream=None):
        F.lib()
        if codes.dtype != torch.uint8 or codes.dim() != 2 or not codes.is_cuda or not codes.is_contiguous():
            raise ValueError("codes: needs a contiguous uint8 device tensor [N, K / 2]")
        self.N, self.K, self.group = codes.shape[0], codes.shape[1] * 2, group
        if scales.dtype not in _DTYPES:
            raise ValueError(f"scales dtype {scales.dtype}: bfloat16 or float16")
        if group not in (32, 64, 128) or self.K % group:
            raise ValueError(f"group={group}: 32, 64 or 128, dividing K={self.K}")
        shape = (self.N, self.K // group)
        for name, t, dt in (("scales", scales, scales.dtype), ("zeros", zeros, torch.uint8)):
            if t is not None and (t.dtype != dt or t.get_device() != codes.get_device() or t.shape != shape or not t.is_contiguous()):
                raise ValueError(f"{name}: needs a contiguous {dt} tensor {list(shape)} on the codes' device")
        self.dtype, self.zeros, self.device, self._dev = scales.dtype, zeros is not None, codes.device, codes.get_device()
        handle = _handle(stream, self._dev)
        nbytes = F.ftmoe_w4_packed_bytes(self.N, self.K, group, self.zeros)
        self.packed = _new(nbytes, torch.uint8, self.device, stream)
        F.ftmoe_w4_pack(codes.data_ptr(), scales.data_ptr(), zeros.data_ptr() if self.zeros else None, self.N, self.K,
                        group, self.packed.data_ptr(), nbytes, handle)
        self._row = self.K + (-self.K) % 8  # a row stride that is never taken
        self._args = (self.packed.data_ptr(), self.N, self.K, group, self.zeros, _DTYPES[self.dtype])

    def matvec(self, x: torch.Tensor, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
        """y [tokens, N] = x [tokens, K] times the weights' transpose."""
        if x.dtype is not self.dtype or x.dim() != 2 or x.get_device() != self._dev:
            raise ValueError(f"x: needs a {self.dtype} tensor [tokens, {self.K}] on device {self._dev} with contiguous rows")
        n, k = x.shape
        xs, x1 = x.stride()
        if k != self.K or x1 != 1:
            raise ValueError(f"x: needs a {self.dtype} device tensor [tokens, {self.K}] with contiguous rows")
        if out is None:
            out = _new((n, self.N), self.dtype, self.device, stream)
        elif out.dtype is not self.dtype or out.shape != (n, self.N) or out.get_device() != self._dev or (self.N > 1 and out.stride(1) != 1):
            raise ValueError(f"out: needs a {self.dtype} tensor [{n}, {self.N}] on device {self._dev} with contiguous rows")
        F.ftmoe_w4_matvec(*self._args, x.data_ptr(), xs if n > 1 else self._row, n, out.data_ptr(),
                          out.stride(0) if n > 1 else self.N, _handle(stream, self._dev))
        return out
