"""A whole mixture-of-experts layer for few tokens.

The experts are uncompressed tensors; ``codec.decode_batch`` with the experts
of one stacked tensor as its outputs fills them from a compressed set.
"""
from __future__ import annotations

import torch

from . import _binding as B
from . import _ops

MAX_TOKENS, MAX_TOP_K, MAX_EXPERTS = 64, 16, 1024


def _check_experts(t, what, shape, dtype, device):
    _ops.check_tensor(t, what, device)
    if t.dtype != dtype:
        raise TypeError(f"{what} must have the type of x, {dtype}")
    if tuple(t.shape) != shape:
        raise ValueError(f"{what} must be {shape}, got {tuple(t.shape)}")
    if t.stride(2) != 1 or t.stride(1) % 8 or t.stride(0) % 8 or t.stride(1) < shape[2] or t.data_ptr() % 16:
        raise ValueError(f"{what} must have unit column stride and 16-byte aligned rows")


def moe_layer(x: torch.Tensor, router: torch.Tensor, w1: torch.Tensor, w3: torch.Tensor, w2: torch.Tensor,
              top_k: int, renormalize: bool = True, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """sum over the top_k experts e of each token of weight_e W2_e
    (silu(W1_e x) * (W3_e x)), m x cols in the type of x.

    x: m x cols BF16 or FP16, m at most 64; router: experts x cols; w1 (gate)
    and w3 (up): experts x inner x cols with the same strides (views of one
    stacked tensor will do); w2 (down): experts x cols x inner; cols and
    inner multiples of 8.  The weights are the softmax over all experts,
    divided by the sum of the chosen ones with `renormalize`.  Equal logits
    go to the expert with the lower number."""
    _ops.check_tensor(x, "x")
    _ops.check_tensor(router, "router", x.device)
    if x.dtype not in _ops.HALVES or router.dtype != x.dtype:
        raise TypeError("x and router must share a 16-bit float type")
    if x.dim() != 2 or router.dim() != 2 or w1.dim() != 3 or router.shape[1] != x.shape[1]:
        raise ValueError("x must be m x cols, router experts x cols, w1 experts x inner x cols")
    m, cols = x.shape
    experts, inner = router.shape[0], w1.shape[1]
    if m > MAX_TOKENS or not 1 <= experts <= MAX_EXPERTS or not 1 <= top_k <= min(MAX_TOP_K, experts):
        raise ValueError(f"at most {MAX_TOKENS} tokens, {MAX_EXPERTS} experts and {MAX_TOP_K} (or all) of them per "
                         f"token: got {m}, {experts} and {top_k}")
    if not cols or cols % 8 or not inner or inner % 8 or max(cols, inner) > 1 << 20:
        raise ValueError(f"cols and inner must be multiples of 8, got {cols} and {inner}")
    _check_experts(w1, "w1", (experts, inner, cols), x.dtype, x.device)
    _check_experts(w3, "w3", (experts, inner, cols), x.dtype, x.device)
    _check_experts(w2, "w2", (experts, cols, inner), x.dtype, x.device)
    if w1.stride() != w3.stride():
        raise ValueError("w1 and w3 must have the same strides")
    if out is not None:
        _ops.check_tensor(out, "out", x.device)
        if out.dtype != x.dtype or out.shape != x.shape or (m and _ops.rows_of(out) is not out):
            raise ValueError("out must be like x, with unit column stride and rows that do not overlap")
    x = _ops.rows16(x)
    router = router if router.is_contiguous() and router.data_ptr() % 16 == 0 else router.clone(
        memory_format=torch.contiguous_format)

    def call(raw):
        o = torch.empty((m, cols), dtype=x.dtype, device=x.device) if out is None else out
        nbytes = B.wc_moe_layer_scratch(m, experts, top_k, cols, inner)
        scratch = torch.empty(nbytes, dtype=torch.uint8, device=x.device)
        g = B.wc_moe(x.data_ptr(), x.stride(0), router.data_ptr(), w1.data_ptr(), w3.data_ptr(), w2.data_ptr(),
                     w1.stride(0), w1.stride(1), w2.stride(0), w2.stride(1), o.data_ptr(), o.stride(0), m, experts,
                     top_k, cols, inner, _ops.TYPES[x.dtype], int(renormalize))
        B.wc_moe_layer(g, scratch, nbytes, raw)
        return o

    return _ops.on_stream(x.device, stream, call)
