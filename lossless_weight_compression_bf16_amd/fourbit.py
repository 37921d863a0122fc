"""Products of few rows with weights of 4 bits and group scales.

Where ``gemm.decode_gemm`` multiplies weights that were compressed without
loss, as they are decoded, this is the lossy form in which frozen weights are
served: a quarter of the bytes, and nothing unpacked in memory.
``adapters.add_adapters`` adds low-rank adapters to the result.
"""
from __future__ import annotations

from typing import NamedTuple

import torch

from . import _binding as B
from . import _ops

GROUPS = (32, 64, 128)


class Weights4(NamedTuple):
    """w[r, k] = scales[r, k // group] (q[r, k] - zeros[r, k // group]), with
    8 for the zeros where there are none."""
    q: torch.Tensor             # rows x cols / 2, uint8: the even column in the low half of a byte
    scales: torch.Tensor        # rows x cols / group, BF16 or FP16
    zeros: torch.Tensor | None  # like scales
    group: int                  # 32, 64 or 128


def _check(x, w, out):
    _ops.check_tensor(x, "x")
    if x.dtype not in _ops.HALVES or x.dim() != 2:
        raise TypeError("x must be a 2-D tensor of a 16-bit float type")
    for t, what in ((w.q, "q"), (w.scales, "scales"), (w.zeros, "zeros")):
        if t is not None:
            _ops.check_tensor(t, what, x.device)
            if t.dim() != 2 or not t.is_contiguous():
                raise ValueError(f"{what} must be 2-D and contiguous")
    if w.q.dtype != torch.uint8 or w.q.data_ptr() % 16:
        raise TypeError("q must be a 16-byte aligned uint8 tensor")
    if w.scales.dtype != x.dtype or w.zeros is not None and w.zeros.dtype != x.dtype:
        raise TypeError(f"scales and zeros must have the type of x, {x.dtype}")
    rows, cols = w.q.shape[0], 2 * w.q.shape[1]
    if w.group not in GROUPS or not cols or cols % w.group or cols > 1 << 20 or not 1 <= rows <= 1 << 24:
        raise ValueError(f"groups of 32, 64 or 128 columns, whole ones, at most 2^20 columns and 2^24 rows: got {rows} x {cols} in "
                         f"groups of {w.group}")
    if x.shape[1] != cols:
        raise ValueError(f"x must have {cols} columns, got {x.shape[1]}")
    groups = (rows, cols // w.group)
    if w.scales.shape != groups or w.zeros is not None and w.zeros.shape != groups:
        raise ValueError(f"scales and zeros must be {groups[0]} x {groups[1]}")
    if out is not None:
        _ops.check_tensor(out, "out", x.device)
        if out.dtype != x.dtype or out.shape != (x.shape[0], rows) or not _ops.rows_apart(out):
            raise ValueError(f"out must be {x.shape[0]} x {rows} in the type of x, with unit column stride and rows that do "
                             "not overlap")
        if any(t is not None and _ops.may_overlap(out, t) for t in (w.q, w.scales, w.zeros)):
            raise ValueError("out and the weights have memory in common")


def _good(x, w) -> bool:
    q, scales, zeros, group = w
    dev, dtype, s = x.device, x.dtype, q.shape
    return (x.is_cuda and q.device == dev and scales.device == dev and dtype in _ops.HALVES and scales.dtype == dtype
            and q.dtype == torch.uint8 and x.dim() == 2 and len(s) == 2 and x.shape[1] == 2 * s[1] and group in GROUPS
            and 0 < 2 * s[1] <= 1 << 20 and not 2 * s[1] % group and 1 <= s[0] <= 1 << 24
            and scales.shape == (s[0], 2 * s[1] // group) and q.is_contiguous() and scales.is_contiguous()
            and not q.data_ptr() % 16
            and (zeros is None or zeros.device == dev and zeros.dtype == dtype and zeros.shape == scales.shape
                 and zeros.is_contiguous()))


def linear4(x: torch.Tensor, w: Weights4, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """x w^T, m x rows in the type of x (BF16 or FP16): products of x with
    whole numbers, summed in fp32 over a group, then scaled and summed in fp32
    and rounded once.  An infinity in a row of x makes its row of y NaN, and
    so may BF16 numbers past 2^128 / (32 group), 8.3e34 for groups of 128,
    whose sums of (16 + q) x over a group pass fp32's range.

    Meant for few rows, where reading the weights is the time; 32 rows of x
    meet them at a time (16 of up to 16).  There is no backward pass: tensors
    that require a gradient raise unless gradients are switched off."""
    if out is not None or not _good(x, w):
        _check(x, w, out)
    if torch.is_grad_enabled() and (x.requires_grad or w.scales.requires_grad or w.zeros is not None and w.zeros.requires_grad
                                    or out is not None and out.requires_grad):
        _ops.no_backward("linear4")
    if _ops.forward_mode():
        _ops.no_tangents("linear4", x, w.scales, w.zeros, out)
    m, cols = x.shape
    rows, dev = w.q.shape[0], x.device

    def call(raw):
        z = _ops.rows16(x)
        y = torch.empty((m, rows), dtype=x.dtype, device=dev) if out is None else out
        if out is not None:
            _ops.written(out)
        a = B.wc_fourbit(z.data_ptr(), z.stride(0), w.q.data_ptr(), w.scales.data_ptr(),
                         w.zeros.data_ptr() if w.zeros is not None else 0, y.data_ptr(), y.stride(0), m, rows, cols, w.group,
                         _ops.TYPES[x.dtype])
        rc = B.lib().wc_linear4(a, raw)
        if rc == B.WC_ERR_ARG and out is not None and _ops.may_overlap(z, y):  # out across x: from a copy of it
            z = z.clone(memory_format=torch.contiguous_format)
            a.x, a.x_stride = z.data_ptr(), cols
            rc = B.lib().wc_linear4(a, raw)
        if rc == B.WC_ERR_ARG:
            raise ValueError(f"{m} rows of x and {rows} of weights are more than one launch takes")
        _ops.done(rc, None, "linear4")
        return y

    return _ops.on_stream(dev, stream, call)


def quantize4(w: torch.Tensor, group: int = 64, zeros: bool = False, stream=None) -> Weights4:
    """The 4-bit form of rows x cols BF16 or FP16 weights: of every `group`
    columns of a row, steps of a seventh of the largest size around 0, or
    with `zeros` of a fifteenth of the range, to which 0 belongs.  Each
    weight goes to the nearest step.  A group with a NaN or an infinity gets
    a scale that says so.  There is no backward pass: weights that require a
    gradient raise unless gradients are switched off."""
    _ops.check_tensor(w, "w")
    if w.dtype not in _ops.HALVES or w.dim() != 2:
        raise TypeError("w must be a 2-D tensor of a 16-bit float type")
    rows, cols = w.shape
    if group not in GROUPS or not cols or cols % group or cols > 1 << 20 or not 1 <= rows <= 1 << 24:
        raise ValueError(f"groups of 32, 64 or 128 columns, whole ones, at most 2^20 columns and 2^24 rows: got {rows} x {cols} in "
                         f"groups of {group}")
    if torch.is_grad_enabled() and w.requires_grad:
        _ops.no_backward("quantize4")
    if _ops.forward_mode():
        _ops.no_tangents("quantize4", w)
    dev = w.device

    def call(raw):
        v = _ops.rows_of(w.detach())
        q = torch.empty((rows, cols // 2), dtype=torch.uint8, device=dev)
        scales = torch.empty((rows, cols // group), dtype=w.dtype, device=dev)
        z = torch.empty_like(scales) if zeros else None
        _ops.done(B.lib().wc_quantize4(v.data_ptr(), v.stride(0), rows, cols, group, _ops.TYPES[w.dtype], q.data_ptr(),
                                       scales.data_ptr(), z.data_ptr() if zeros else 0, raw), None, "quantize4")
        return Weights4(q, scales, z, group)

    return _ops.on_stream(dev, stream, call)
