"""Matrix products grouped by expert over ragged rows, with their gradients:
the experts of a mixture-of-experts layer for any number of tokens, once the
rows have been sorted by expert.

Where ``moe.moe_layer`` is a whole layer for up to 64 tokens, this is its one
product for as many as there are, and it can be trained.
"""
from __future__ import annotations

import torch

from . import _binding as B
from . import _ops

MAX_EXPERTS = 1024
_MAX_STRIDE = (1 << 22) - 8


def _check(x, w, ends, out=None, grad=None):
    _ops.check_tensor(x, "x")
    _ops.check_tensor(w, "w", x.device)
    _ops.check_tensor(ends, "ends", x.device)
    if x.dtype not in _ops.HALVES or w.dtype != x.dtype:
        raise TypeError("x and w must share a 16-bit float type")
    if x.dim() != 2 or w.dim() != 3 or w.shape[2] != x.shape[1]:
        raise ValueError("x must be m x cols, w experts x rows x cols")
    experts, rows, cols = w.shape
    if not 1 <= experts <= MAX_EXPERTS:
        raise ValueError(f"1 to {MAX_EXPERTS} experts, got {experts}")
    if not cols or cols % 8 or not rows or rows % 8 or max(cols, rows) > 1 << 20:
        raise ValueError(f"cols and rows must be multiples of 8, at most 2^20, got {cols} and {rows}")
    if ends.dtype != torch.int64 or ends.shape != (experts,):
        raise ValueError(f"ends must be {experts} int64 numbers, one per expert")
    if (w.stride(2) != 1 or w.stride(1) % 8 or w.stride(0) % 8 or not cols <= w.stride(1) <= _MAX_STRIDE
            or w.data_ptr() % 16):
        raise ValueError("w must have unit column stride and 16-byte aligned rows, less than 2^22 elements apart")
    if out is not None:
        _ops.check_tensor(out, "out", x.device)
        if out.dtype != x.dtype or out.shape != (x.shape[0], rows) or not _rows_fit(out):
            raise ValueError(f"out must be {x.shape[0]} x {rows} in the type of x, with unit column stride and 16-byte "
                             "aligned rows that do not overlap, less than 2^22 elements apart")
    if grad is not None:
        _ops.check_tensor(grad, "grad", x.device)
        if grad.dtype != x.dtype or grad.shape != (x.shape[0], rows):
            raise ValueError(f"grad must be {x.shape[0]} x {rows} in the type of x")


def _rows_fit(t) -> bool:
    row, col = t.stride()
    return col == 1 and row % 8 == 0 and t.shape[1] <= row <= _MAX_STRIDE and t.data_ptr() % 16 == 0


def _rows(t: torch.Tensor) -> torch.Tensor:
    return t if _rows_fit(t) else t.clone(memory_format=torch.contiguous_format)


def _good(x, w, ends) -> bool:
    """The plain case: contiguous weights."""
    dev, dtype, s = x.device, x.dtype, w.shape
    return (x.is_cuda and w.device == dev and ends.device == dev and dtype in _ops.HALVES and w.dtype == dtype
            and x.dim() == 2 and len(s) == 3 and x.shape[1] == s[2] and 1 <= s[0] <= MAX_EXPERTS
            and 8 <= s[1] <= 1 << 20 and 8 <= s[2] <= 1 << 20 and not s[1] % 8 and not s[2] % 8
            and ends.dtype == torch.int64 and ends.shape == s[:1] and w.is_contiguous() and not w.data_ptr() % 16)


def _limit(m, w):
    raise ValueError(f"{m} rows of {w.shape[0]} experts of {w.shape[1]} x {w.shape[2]} are more tiles than one launch takes")


def _forward(x, w, ends, out, check, stream):
    (m, cols), (experts, rows, _), dev = x.shape, w.shape, x.device

    def call(raw):
        z, e = _rows(x), ends.contiguous()
        y = torch.empty((m, rows), dtype=x.dtype, device=dev) if out is None else out
        if out is not None:
            _ops.written(out)
        lib = B.lib()
        nbytes = lib.wc_grouped_linear_scratch(m, experts, rows, cols)
        scratch = torch.empty(nbytes, dtype=torch.uint8, device=dev) if nbytes else None
        err = _ops.error_word(check, dev)
        g = B.wc_grouped(z.data_ptr(), z.stride(0), w.data_ptr(), w.stride(0) if experts > 1 else 0, w.stride(1),
                         e.data_ptr(), y.data_ptr(), y.stride(0), m, experts, rows, cols, _ops.TYPES[x.dtype],
                         1 if out is None else 0, 0)
        args = scratch.data_ptr() if nbytes else 0, nbytes, err.data_ptr() if check else 0, raw
        rc = lib.wc_grouped_linear(g, *args)
        if rc == B.WC_ERR_ARG and out is not None and _ops.may_overlap(z, y):  # out across x: from a copy of it
            z = z.clone(memory_format=torch.contiguous_format)
            g.x, g.x_stride = z.data_ptr(), cols
            rc = lib.wc_grouped_linear(g, *args)
        if rc == B.WC_ERR_ARG:
            _limit(m, w)
        _ops.done(rc, err, "grouped_linear")
        return y

    return _ops.on_stream(dev, stream, call)


def grouped_linear(x: torch.Tensor, w: torch.Tensor, ends: torch.Tensor, out: torch.Tensor | None = None,
                   check: bool = True, stream=None) -> torch.Tensor:
    """y[r] = w[e] x[r] for the rows ends[e - 1] <= r < ends[e] of every
    expert e (from 0 for the first), m x rows in the type of x.

    x: m x cols BF16 or FP16, sorted by expert; w: experts x rows x cols, a
    view of a larger tensor will do; ends: experts int64 numbers on the
    device, which never have to come to the host.  rows and cols are
    multiples of 8.  Rows behind the last expert's are not read: their y is
    zero, or in a given `out` what it was.  x and w can be differentiated,
    once; captured into a graph only while autograd holds no other graph of
    them, which is looked at where they are leaves, not for leaves that they are
    made from.  With check (which waits for the GPU) ends that go back, or past
    the rows, raise; without, y is undefined."""
    if out is not None or not _good(x, w, ends):
        _check(x, w, ends, out)
    if _ops.forward_mode():
        _ops.no_tangents("grouped_linear", x, w, out)
    if torch.is_grad_enabled() and (x.requires_grad or w.requires_grad or out is not None and out.requires_grad):
        if out is not None or stream is not None:
            raise ValueError("with gradients the call runs on the current stream and makes its own result: use "
                             "torch.cuda.stream, and no out")
        _ops.fresh_under_capture("grouped_linear", x, w)
        y = _GroupedLinear.apply(x, w, ends, check)
        _ops.note_captured(x, w)
        return y
    if out is not None and (_ops.may_overlap(out, w) or _ops.may_overlap(out, ends)):
        raise ValueError("out and w or ends have memory in common")
    return _forward(x, w, ends, out, check, stream)


def grouped_linear_backward(x: torch.Tensor, w: torch.Tensor, ends: torch.Tensor, grad: torch.Tensor,
                            need_x: bool = True, need_w: bool = True, check: bool = True, stream=None):
    """The gradients of x and w from that of ``grouped_linear``'s result, in
    their type (None where not needed): w[e]^T grad[r], and the sum of
    grad[r] x[r]^T over an expert's rows, zero for an expert without any.
    Rows behind the last expert's are not read, and their gradient is zero."""
    if not (_good(x, w, ends) and grad.device == x.device and grad.dtype == x.dtype
            and grad.shape == (x.shape[0], w.shape[1])):
        _check(x, w, ends, None, grad)
    if _ops.forward_mode():
        _ops.no_tangents("grouped_linear_backward", x, w, grad)
    if torch.is_grad_enabled() and (x.requires_grad or w.requires_grad or grad.requires_grad):
        _ops.no_backward("grouped_linear_backward")
    return _backward(x, w, ends, grad, need_x, need_w, check, stream)


def _backward(x, w, ends, grad, need_x, need_w, check, stream):
    (m, cols), (experts, rows, _), dev = x.shape, w.shape, x.device
    if not need_x and not need_w:
        return None, None

    def call(raw):
        z, d, e = _rows(x), _rows(grad), ends.contiguous()
        dx = torch.empty((m, cols), dtype=x.dtype, device=dev) if need_x else None
        dw = torch.empty((experts, rows, cols), dtype=x.dtype, device=dev) if need_w else None
        lib = B.lib()
        nbytes = lib.wc_grouped_linear_backward_scratch(m, experts, rows, cols)
        scratch = torch.empty(nbytes, dtype=torch.uint8, device=dev) if nbytes else None
        err = _ops.error_word(check, dev)
        g = B.wc_grouped_grad(z.data_ptr(), z.stride(0), w.data_ptr(), w.stride(0) if experts > 1 else 0, w.stride(1),
                              e.data_ptr(), d.data_ptr(), d.stride(0), dx.data_ptr() if need_x else 0, cols,
                              dw.data_ptr() if need_w else 0, m, experts, rows, cols, _ops.TYPES[x.dtype], 1, 0)
        rc = lib.wc_grouped_linear_backward(g, scratch.data_ptr() if nbytes else 0, nbytes, err.data_ptr() if check else 0,
                                            raw)
        if rc == B.WC_ERR_ARG:
            _limit(m, w)
        _ops.done(rc, err, "grouped_linear_backward")
        return dx, dw

    return _ops.on_stream(dev, stream, call)


class _GroupedLinear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, ends, check):
        ctx.save_for_backward(x, w, ends)
        ctx.set_materialize_grads(False)
        return _forward(x, w, ends, None, check, None)

    @staticmethod
    def backward(ctx, grad):
        if grad is None:
            return None, None, None, None
        x, w, ends = ctx.saved_tensors
        need = ctx.needs_input_grad
        found = _backward(x, w, ends, grad, need[0], need[1], False, None)
        return *_ops.once("grouped_linear", found, x, w, grad), None, None
