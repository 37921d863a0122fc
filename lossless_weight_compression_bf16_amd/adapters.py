"""Low-rank adapters of many requests beside a shared projection.

The projection's weights are shared (and may be compressed:
``gemm.decode_gemm`` adds X W^T into Y); each request's adapter is a pair of
small matrices, and its product is added into the same Y.
"""
from __future__ import annotations

import torch

from . import _binding as B
from . import _ops

MAX_RANK = 256


def add_adapters(x: torch.Tensor, y: torch.Tensor, a: torch.Tensor, b: torch.Tensor, ids: torch.Tensor,
                 scales: torch.Tensor | None = None, check: bool = True, stream=None) -> torch.Tensor:
    """y[t] += scales[i] B_i (A_i x[t]) with i = ids[t], in place; returns y.

    x: m x cols BF16 or FP16; y: m x rows, FP32 or the type of x; a: n x rank
    x cols and b: n x rows x rank in the type of x (rank at most 256, smaller
    ones padded with zeros; cols a multiple of 8); ids: m int64, -1 for a
    token without an adapter; scales: n FP32.  With check (which waits for
    the GPU) an id out of range raises; without, its row of y stays as it
    is."""
    for t, what in ((x, "x"), (y, "y"), (a, "a"), (b, "b"), (ids, "ids")):
        _ops.check_tensor(t, what, x.device)
    if x.dtype not in _ops.HALVES or a.dtype != x.dtype or b.dtype != x.dtype:
        raise TypeError("x, a and b must share a 16-bit float type")
    if y.dtype not in (x.dtype, torch.float32):
        raise TypeError("y must be float32 or of the type of x")
    if x.dim() != 2 or y.dim() != 2 or a.dim() != 3 or b.dim() != 3:
        raise ValueError("x and y must be 2-D, a and b 3-D")
    m, cols = x.shape
    n, rank, rows = a.shape[0], a.shape[1], y.shape[1]
    if y.shape[0] != m or a.shape[2] != cols or tuple(b.shape) != (n, rows, rank):
        raise ValueError(f"shapes do not match: x {tuple(x.shape)}, y {tuple(y.shape)}, a {tuple(a.shape)}, "
                         f"b {tuple(b.shape)}")
    if not 1 <= rank <= MAX_RANK or cols % 8 or not cols or not rows:
        raise ValueError(f"the rank must be 1 to {MAX_RANK} and cols a multiple of 8, got {rank} and {cols}")
    if ids.dtype != torch.int64 or ids.shape != (m,):
        raise ValueError(f"ids must be {m} int64 numbers, one per row of x")
    if not a.is_contiguous() or not b.is_contiguous() or a.data_ptr() % 16:
        raise ValueError("a and b must be contiguous, and a 16-byte aligned")
    if m and (y.stride(1) != 1 and rows > 1 or y.stride(0) < rows and m > 1):
        raise ValueError("y must have unit column stride and rows that do not overlap")
    if scales is not None:
        _ops.check_tensor(scales, "scales", x.device)
        if scales.dtype != torch.float32 or scales.shape != (n,):
            raise ValueError(f"scales must be {n} float32 numbers")
        scales = scales.contiguous()
    x = _ops.rows16(x)
    ids = ids.contiguous()

    def call(raw):
        nbytes = B.wc_add_adapters_scratch(m, rank, cols, rows)
        scratch = torch.empty(nbytes, dtype=torch.uint8, device=x.device) if nbytes else None
        err = torch.zeros(1, dtype=torch.int32, device=x.device) if check else None
        g = B.wc_adapters(x.data_ptr(), x.stride(0), y.data_ptr(), y.stride(0), a.data_ptr(), b.data_ptr(),
                          ids.data_ptr(), scales.data_ptr() if scales is not None else 0, m, n, rank, cols, rows,
                          _ops.TYPES[x.dtype], _ops.TYPES[y.dtype])
        B.wc_add_adapters(g, scratch, nbytes, err, raw)
        _ops.raise_bits(err, "add_adapters")
        return y

    return _ops.on_stream(x.device, stream, call)
