"""Softmax cross entropy over a large vocabulary from hidden states and the
output weights: the logits are made a tile at a time, and again for the
gradient, and are never in memory.

Where ``logprobs.token_logprobs`` takes logits that a program has, this takes
what they are made from.
"""
from __future__ import annotations

from typing import NamedTuple

import torch

from . import _binding as B
from . import _ops
from .grouped import _MAX_STRIDE, _rows, _rows_fit

MAX_ROWS, MAX_VOCAB = 1 << 19, 1 << 22


class LinearCrossEntropy(NamedTuple):
    loss: torch.Tensor  # m, fp32: minus the log probability of each row's token (0 for token -1)
    lse: torch.Tensor   # m, fp32: log of the sum of the exponentials of the row's logits


def _check(hidden, weight, tokens):
    _ops.check_tensor(hidden, "hidden")
    _ops.check_tensor(weight, "weight", hidden.device)
    _ops.check_tensor(tokens, "tokens", hidden.device)
    if hidden.dtype not in _ops.HALVES or weight.dtype != hidden.dtype:
        raise TypeError("hidden and weight must share a 16-bit float type")
    if hidden.dim() != 2 or weight.dim() != 2 or weight.shape[1] != hidden.shape[1]:
        raise ValueError("hidden must be m x cols, weight vocabulary x cols")
    m, cols = hidden.shape
    if not cols or cols % 8 or cols > 1 << 20:
        raise ValueError(f"cols must be a multiple of 8, at most 2^20, got {cols}")
    if m > MAX_ROWS or not 1 <= weight.shape[0] <= MAX_VOCAB:
        raise ValueError(f"at most {MAX_ROWS} rows, and a vocabulary of 1 to {MAX_VOCAB}: got {m} and {weight.shape[0]}")
    if tokens.dtype != torch.int64 or tokens.shape != (m,):
        raise ValueError(f"tokens must be {m} int64 numbers, one per row")
    if not _rows_fit(weight):
        raise ValueError("weight must have unit column stride and 16-byte aligned rows that do not overlap, less than "
                         "2^22 elements apart")


def _good(hidden, weight, tokens) -> bool:
    dev, dtype, s, v = hidden.device, hidden.dtype, hidden.shape, weight.shape
    return (hidden.is_cuda and weight.device == dev and tokens.device == dev and dtype in _ops.HALVES
            and weight.dtype == dtype and len(s) == 2 and len(v) == 2 and v[1] == s[1] and 8 <= s[1] <= 1 << 20
            and not s[1] % 8 and s[0] <= MAX_ROWS and 1 <= v[0] <= MAX_VOCAB and tokens.dtype == torch.int64
            and tokens.shape == s[:1] and weight.is_contiguous() and not weight.data_ptr() % 16)


def _forward(hidden, weight, tokens, check, stream, views=True):
    (m, cols), vocab, dev = hidden.shape, weight.shape[0], hidden.device

    def call(raw):
        h, t = _rows(hidden), tokens.contiguous()
        if views:  # one allocation
            loss, lse = torch.empty((2, m), dtype=torch.float32, device=dev).unbind(0)
        else:      # autograd's outputs are tensors of their own
            loss, lse = (torch.empty(m, dtype=torch.float32, device=dev) for _ in range(2))
        lib = B.lib()
        nbytes = lib.wc_linear_cross_entropy_scratch(m, vocab, cols)
        scratch = torch.empty(nbytes, dtype=torch.uint8, device=dev)
        err = _ops.error_word(check, dev)
        a = B.wc_linear_loss(h.data_ptr(), h.stride(0), weight.data_ptr(), weight.stride(0), t.data_ptr(), m, vocab, cols,
                             _ops.TYPES[h.dtype], 0, loss.data_ptr(), lse.data_ptr())
        _ops.done(lib.wc_linear_cross_entropy(a, scratch.data_ptr(), nbytes, err.data_ptr() if check else 0, raw), err,
                  "linear_cross_entropy")
        return LinearCrossEntropy(loss, lse)

    return _ops.on_stream(dev, stream, call)


def linear_cross_entropy(hidden: torch.Tensor, weight: torch.Tensor, tokens: torch.Tensor, check: bool = True,
                         stream=None, rounded: bool = False) -> LinearCrossEntropy:
    """loss[r] = lse[r] - z[r, tokens[r]] and lse[r] = log sum_v exp z[r, v]
    of the logits z = hidden weight^T, which are not kept.

    hidden: m x cols and weight: vocabulary x cols, BF16 or FP16, cols a
    multiple of 8; the logits are sums in fp32 and are not rounded.  Token -1
    stands for no token (loss 0, whatever the row holds).  hidden and weight
    can be differentiated, once, through loss and lse (a penalty on the
    size of the logits is a function of lse); captured into a graph only
    while autograd holds no other graph of them, which is looked at where they
    are leaves, not for leaves that they are made from.  `rounded` is the gradients':
    see linear_cross_entropy_backward.  With check (which waits for
    the GPU) a token out of range raises; without, its loss is NaN."""
    if not _good(hidden, weight, tokens):
        _check(hidden, weight, tokens)
    if _ops.forward_mode():
        _ops.no_tangents("linear_cross_entropy", hidden, weight)
    if torch.is_grad_enabled() and (hidden.requires_grad or weight.requires_grad):
        if stream is not None:
            raise ValueError("with gradients the call runs on the current stream: use torch.cuda.stream")
        _ops.fresh_under_capture("linear_cross_entropy", hidden, weight)
        r = LinearCrossEntropy(*_LinearCrossEntropy.apply(hidden, weight, tokens, check, rounded))
        _ops.note_captured(hidden, weight)
        return r
    return _forward(hidden, weight, tokens, check, stream)


def linear_cross_entropy_backward(hidden: torch.Tensor, weight: torch.Tensor, tokens: torch.Tensor, lse: torch.Tensor,
                                  grad_loss=None, grad_lse=None, need_hidden: bool = True, need_weight: bool = True,
                                  check: bool = True, stream=None, rounded: bool = False):
    """The gradients of hidden and weight, in their type (None where not
    needed), from those of loss and lse (either may be None) and the lse that
    ``linear_cross_entropy`` gave.  The gradient of the logits is made for
    a piece of the vocabulary at a time, as a sum of two numbers of the type of
    hidden (16 bits of it in BF16, 22 in FP16), and both products sum it in fp32.
    With `rounded` it is one such number, and both products take half as
    long, but a gradient's error then is about that of two roundings to the type, not of one.  A
    row without a token and without a gradient of lse has no part in them, whatever it holds."""
    if not _good(hidden, weight, tokens):
        _check(hidden, weight, tokens)
    m, dev = hidden.shape[0], hidden.device
    for v, what in ((lse, "lse"), (grad_loss, "grad_loss"), (grad_lse, "grad_lse")):
        if v is None:
            if what == "lse":
                raise ValueError("lse is needed")
        elif not (v.dtype == torch.float32 and v.shape == (m,) and v.device == dev):
            _ops.check_tensor(v, what, dev)
            raise ValueError(f"{what} must be {m} float32 numbers")
    given = [t for t in (hidden, weight, lse, grad_loss, grad_lse) if t is not None]
    if _ops.forward_mode():
        _ops.no_tangents("linear_cross_entropy_backward", *given)
    if torch.is_grad_enabled() and any(t.requires_grad for t in given):
        _ops.no_backward("linear_cross_entropy_backward")
    return _backward(hidden, weight, tokens, lse, grad_loss, grad_lse, need_hidden, need_weight, check, stream, rounded)


def _backward(hidden, weight, tokens, lse, grad_loss, grad_lse, need_hidden, need_weight, check, stream, rounded):
    (m, cols), vocab, dev = hidden.shape, weight.shape[0], hidden.device
    if not need_hidden and not need_weight:
        return None, None

    def call(raw):
        dh = torch.empty((m, cols), dtype=hidden.dtype, device=dev) if need_hidden else None
        if not m:
            return dh, torch.zeros((vocab, cols), dtype=hidden.dtype, device=dev) if need_weight else None
        dw = torch.empty((vocab, cols), dtype=hidden.dtype, device=dev) if need_weight else None
        h, t, s = _rows(hidden), tokens.contiguous(), lse.contiguous()
        gl = grad_loss.contiguous() if grad_loss is not None else None
        gz = grad_lse.contiguous() if grad_lse is not None else None
        lib = B.lib()
        nbytes = lib.wc_linear_cross_entropy_backward_scratch(m, vocab, cols)
        scratch = torch.empty(nbytes, dtype=torch.uint8, device=dev)
        err = _ops.error_word(check, dev)
        a = B.wc_linear_loss_grad(h.data_ptr(), h.stride(0), weight.data_ptr(), weight.stride(0), t.data_ptr(), s.data_ptr(),
                                  gl.data_ptr() if gl is not None else 0, gz.data_ptr() if gz is not None else 0,
                                  dh.data_ptr() if need_hidden else 0, cols, dw.data_ptr() if need_weight else 0, m, vocab,
                                  cols, _ops.TYPES[h.dtype], 1 if rounded else 0)
        _ops.done(lib.wc_linear_cross_entropy_backward(a, scratch.data_ptr(), nbytes, err.data_ptr() if check else 0, raw),
                  err, "linear_cross_entropy_backward")
        return dh, dw

    return _ops.on_stream(dev, stream, call)


class _LinearCrossEntropy(torch.autograd.Function):
    @staticmethod
    def forward(ctx, hidden, weight, tokens, check, rounded):
        ctx.rounded = rounded
        r = _forward(hidden, weight, tokens, check, None, views=False)
        ctx.save_for_backward(hidden, weight, tokens, r.lse)
        ctx.set_materialize_grads(False)
        return tuple(r)

    @staticmethod
    def backward(ctx, grad_loss, grad_lse):
        if grad_loss is None and grad_lse is None:
            return (None,) * 5
        hidden, weight, tokens, lse = ctx.saved_tensors
        need = ctx.needs_input_grad
        found = _backward(hidden, weight, tokens, lse, grad_loss, grad_lse, need[0], need[1], False, None,
                          ctx.rounded)
        return *_ops.once("linear_cross_entropy", found, hidden, weight, grad_loss, grad_lse), None, None, None
