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
    if (t.stride(2) != 1 or t.stride(1) % 8 or t.stride(0) % 8 or not shape[2] <= t.stride(1) <= 1 << 26
            or t.data_ptr() % 16):
        raise ValueError(f"{what} must have unit column stride and 16-byte aligned rows, at most 2^26 elements apart")


def _check(x, router, w1, w3, w2, top_k, out):
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
        if out.dtype != x.dtype or out.shape != x.shape or not _ops.rows_apart(out):
            raise ValueError("out must be like x, with unit column stride and rows that do not overlap")


def _good(x, router, w1, w3, w2, top_k) -> bool:
    """The plain case: everything contiguous."""
    dev, dtype = x.device, x.dtype
    if not (x.is_cuda and router.device == dev and w1.device == dev and w3.device == dev and w2.device == dev
            and dtype in _ops.HALVES and router.dtype == dtype and w1.dtype == dtype and w3.dtype == dtype
            and w2.dtype == dtype and x.dim() == 2 and router.dim() == 2):
        return False
    (m, cols), experts, s1 = x.shape, router.shape[0], w1.shape
    return (len(s1) == 3 and router.shape[1] == cols and s1 == (experts, s1[1], cols) and w3.shape == s1
            and w2.shape == (experts, cols, s1[1]) and m <= MAX_TOKENS and experts <= MAX_EXPERTS
            and 1 <= top_k <= experts and top_k <= MAX_TOP_K and 8 <= cols <= 1 << 20 and 8 <= s1[1] <= 1 << 20
            and not cols % 8 and not s1[1] % 8 and w1.is_contiguous() and w3.is_contiguous() and w2.is_contiguous()
            and not (w1.data_ptr() | w3.data_ptr() | w2.data_ptr()) % 16)


def moe_layer(x: torch.Tensor, router: torch.Tensor, w1: torch.Tensor, w3: torch.Tensor, w2: torch.Tensor,
              top_k: int, renormalize: bool = True, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """sum over the top_k experts e of each token of weight_e W2_e
    (silu(W1_e x) * (W3_e x)), m x cols in the type of x.

    x: m x cols BF16 or FP16, m at most 64; router: experts x cols; w1 (gate)
    and w3 (up): experts x inner x cols with the same strides (views of one
    stacked tensor will do); w2 (down): experts x cols x inner; cols and
    inner multiples of 8.  The weights are the softmax over all experts,
    divided by the sum of the chosen ones with `renormalize`.  Equal logits
    go to the expert with the lower number.  There is no backward pass:
    tensors that require a gradient raise unless gradients are switched off."""
    if out is not None or not _good(x, router, w1, w3, w2, top_k):
        _check(x, router, w1, w3, w2, top_k, out)
    if torch.is_grad_enabled() and (x.requires_grad or router.requires_grad or w1.requires_grad or w3.requires_grad
                                    or w2.requires_grad or out is not None and out.requires_grad):
        _ops.no_backward("moe_layer")
    if _ops.forward_mode():
        _ops.no_tangents("moe_layer", x, router, w1, w3, w2, out)
    (m, cols), (experts, inner, _), dev = x.shape, w1.shape, x.device

    def call(raw):
        lib = B.lib()
        z = _ops.rows16(x)
        r = router if router.is_contiguous() and router.data_ptr() % 16 == 0 else router.clone(
            memory_format=torch.contiguous_format)
        o = torch.empty((m, cols), dtype=x.dtype, device=dev) if out is None else out
        if out is not None:
            _ops.written(out)
        nbytes = lib.wc_moe_layer_scratch(m, experts, top_k, cols, inner)
        if m and not nbytes:
            raise ValueError(f"experts with tokens (at most {min(m * top_k, experts)}) times inner must be below 2^28, "
                             f"got inner {inner}")
        scratch = torch.empty(nbytes, dtype=torch.uint8, device=dev)
        up, down = w1.stride(), w2.stride()
        g = B.wc_moe(z.data_ptr(), z.stride(0), r.data_ptr(), w1.data_ptr(), w3.data_ptr(), w2.data_ptr(),
                     up[0], up[1], down[0], down[1], o.data_ptr(), o.stride(0), m, experts, top_k, cols, inner,
                     _ops.TYPES[x.dtype], 1 if renormalize else 0)
        _ops.done(lib.wc_moe_layer(g, scratch.data_ptr(), nbytes, raw), None, "moe_layer")
        return o

    return _ops.on_stream(dev, stream, call)
