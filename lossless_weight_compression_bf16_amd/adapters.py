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


def _check(x, y, a, b, ids, scales):
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
    if ids.dtype != torch.int64 or ids.shape != (m,):
        raise ValueError(f"ids must be {m} int64 numbers, one per row of x")
    if not a.is_contiguous() or not b.is_contiguous() or a.data_ptr() % 16:
        raise ValueError("a and b must be contiguous, and a 16-byte aligned")
    if not _ops.rows_apart(y):
        raise ValueError("y must have unit column stride and rows that do not overlap")
    if scales is not None:
        _ops.check_tensor(scales, "scales", x.device)
        if scales.dtype != torch.float32 or scales.shape != (n,):
            raise ValueError(f"scales must be {n} float32 numbers")
    raise ValueError(f"the rank must be 1 to {MAX_RANK}, cols a multiple of 8 and rank * rows below 2^31, got {rank}, "
                     f"{cols} and {rows}")


def add_adapters(x: torch.Tensor, y: torch.Tensor, a: torch.Tensor, b: torch.Tensor, ids: torch.Tensor,
                 scales: torch.Tensor | None = None, check: bool = True, stream=None) -> torch.Tensor:
    """y[t] += scales[i] B_i (A_i x[t]) with i = ids[t], in place; returns y.

    x: m x cols BF16 or FP16; y: m x rows, FP32 or the type of x; a: n x rank
    x cols and b: n x rows x rank in the type of x (rank at most 256, smaller
    ones padded with zeros; cols a multiple of 8); ids: m int64, -1 for a
    token without an adapter; scales: n FP32.  y may lie in x's memory (x is
    copied first).  There is no backward pass: tensors that require a gradient
    raise unless gradients are switched off.  With check (which waits for
    the GPU) an id out of range raises; without, its row of y stays as it
    is."""
    dev, dtype, y_type = x.device, x.dtype, y.dtype
    if not (x.is_cuda and y.device == dev and a.device == dev and b.device == dev and ids.device == dev
            and dtype in _ops.HALVES and a.dtype == dtype and b.dtype == dtype
            and (y_type == dtype or y_type == torch.float32) and ids.dtype == torch.int64
            and len(shape := x.shape) == 2 and len(sy := y.shape) == 2 and len(sa := a.shape) == 3
            and sy[0] == shape[0] and sa[2] == shape[1] and b.shape == (sa[0], sy[1], sa[1]) and ids.shape == shape[:1]
            and 1 <= sa[1] <= MAX_RANK and shape[1] and not shape[1] % 8 and sy[1] and sy[1] * sa[1] < 1 << 31
            and a.is_contiguous() and b.is_contiguous() and not a.data_ptr() % 16 and _ops.rows_apart(y)
            and (scales is None or scales.dtype == torch.float32 and scales.shape == sa[:1] and scales.device == dev)):
        _check(x, y, a, b, ids, scales)
    if torch.is_grad_enabled() and (x.requires_grad or y.requires_grad or a.requires_grad or b.requires_grad
                                    or scales is not None and scales.requires_grad):
        _ops.no_backward("add_adapters")
    if _ops.forward_mode():
        _ops.no_tangents("add_adapters", x, y, a, b, scales)
    m, cols = shape
    n, rank, _ = sa
    rows = sy[1]

    def call(raw):
        lib = B.lib()
        z, i = _ops.rows16(x), ids.contiguous()
        s = scales.contiguous() if scales is not None else None
        nbytes = lib.wc_add_adapters_scratch(m, rank, cols, rows)
        scratch = torch.empty(nbytes, dtype=torch.uint8, device=dev) if nbytes else None
        err = _ops.error_word(check, dev)
        (z_row, _), (y_row, _) = z.stride(), y.stride()
        g = B.wc_adapters(z.data_ptr(), z_row, y.data_ptr(), y_row, a.data_ptr(), b.data_ptr(), i.data_ptr(),
                          s.data_ptr() if s is not None else 0, m, n, rank, cols, rows, _ops.TYPES[dtype],
                          _ops.TYPES[y_type])
        _ops.written(y)
        room, word = scratch.data_ptr() if nbytes else 0, err.data_ptr() if check else 0
        rc = lib.wc_add_adapters(g, room, nbytes, word, raw)
        if rc == B.WC_ERR_ARG and _ops.may_overlap(z, y):  # y in x's memory: from a copy of x
            z = z.clone(memory_format=torch.contiguous_format)
            g.x, g.x_stride = z.data_ptr(), cols
            rc = lib.wc_add_adapters(g, room, nbytes, word, raw)
        _ops.done(rc, err, "add_adapters")
        return y

    return _ops.on_stream(dev, stream, call)
