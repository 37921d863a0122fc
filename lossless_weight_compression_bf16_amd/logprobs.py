"""Log probabilities of given tokens, with entropy and the most likely
alternatives, and the gradient of the logits.

``token_logprobs`` reads the logits once; autograd runs
``token_logprobs_backward`` for logits that require a gradient.
"""
from __future__ import annotations

from typing import NamedTuple

import torch

from . import _binding as B
from . import _ops

MAX_TOP = 64


class TokenLogprobs(NamedTuple):
    logprob: torch.Tensor        # m, fp32: log probability of each row's token (0 for token -1)
    entropy: torch.Tensor        # m, fp32, in nats
    lse: torch.Tensor            # m, fp32: log of the sum of the exponentials
    top_logprobs: torch.Tensor | None   # m x top, fp32, largest first; None without alternatives
    top_ids: torch.Tensor | None        # m x top, int64; equal logits by their index, NaN last


def _check(logits, tokens):
    _ops.check_tensor(logits, "logits")
    _ops.check_tensor(tokens, "tokens", logits.device)
    if logits.dim() != 2 or logits.dtype not in _ops.TYPES:
        raise TypeError("logits must be a 2-D bfloat16, float16 or float32 tensor (rows x vocabulary)")
    if tokens.dtype != torch.int64 or tokens.shape != logits.shape[:1]:
        raise ValueError(f"tokens must be {logits.shape[0]} int64 numbers, one per row")
    if not logits.shape[1]:
        raise ValueError("the vocabulary is empty")


def _good(logits, tokens, device) -> bool:
    return (logits.is_cuda and tokens.device == device and logits.dim() == 2 and logits.dtype in _ops.TYPES
            and tokens.dtype == torch.int64 and tokens.shape == logits.shape[:1] and logits.shape[1] > 0)


def _forward(logits, tokens, top, check, stream, views=True):
    m, vocab = logits.shape
    dev = logits.device

    def call(raw):
        z, t = _ops.rows_of(logits), tokens.contiguous()
        best = ids = None
        if not views:  # autograd's outputs are tensors of their own
            rows = [torch.empty(m, dtype=torch.float32, device=dev) for _ in range(3)]
            if top:
                best = torch.empty((m, top), dtype=torch.float32, device=dev)
        elif top:  # one allocation for the fp32 outputs
            *rows, best = torch.empty(m * (3 + top), dtype=torch.float32, device=dev).split_with_sizes(
                (m, m, m, m * top))
            best = best.view(m, top)
        else:
            rows = torch.empty((3, m), dtype=torch.float32, device=dev).unbind(0)
        if top:
            ids = torch.empty((m, top), dtype=torch.int64, device=dev)
        lib = B.lib()
        nbytes = lib.wc_token_logprobs_scratch(m, vocab, top)
        scratch = torch.empty(nbytes, dtype=torch.uint8, device=dev) if nbytes else None
        err = _ops.error_word(check, dev)
        a = B.wc_logprobs(z.data_ptr(), z.stride(0), t.data_ptr(), m, vocab, top, _ops.TYPES[z.dtype], 0,
                          rows[0].data_ptr(), rows[1].data_ptr(), rows[2].data_ptr(),
                          best.data_ptr() if top else 0, ids.data_ptr() if top else 0)
        _ops.done(lib.wc_token_logprobs(a, scratch.data_ptr() if nbytes else 0, nbytes,
                                        err.data_ptr() if check else 0, raw), err, "token_logprobs")
        return TokenLogprobs(*rows, best, ids)

    return _ops.on_stream(dev, stream, call)


def token_logprobs(logits: torch.Tensor, tokens: torch.Tensor, top: int = 0, check: bool = True,
                   stream=None) -> TokenLogprobs:
    """Log probability of tokens[r] under softmax(logits[r]), the row's
    entropy, and its `top` (at most 64) most likely alternatives.

    Token -1 stands for no token (logprob 0).  -inf masks a logit; a row of
    nothing but -inf has lse and log probabilities -inf and entropy 0; a row
    with NaN or +inf has NaN statistics.  logprob and entropy can be
    differentiated, once; lse and top_logprobs raise when a gradient comes
    back to them.  With check (which waits for the
    GPU) a token out of range raises; without, its logprob is NaN."""
    if not _good(logits, tokens, logits.device):
        _check(logits, tokens)
    if not 0 <= top <= min(MAX_TOP, logits.shape[1]):
        raise ValueError(f"top must be between 0 and {min(MAX_TOP, logits.shape[1])}, got {top}")
    if _ops.forward_mode():
        _ops.no_tangents("token_logprobs", logits)
    if logits.requires_grad and torch.is_grad_enabled():
        if stream is not None:
            raise ValueError("with gradients the call runs on the current stream: use torch.cuda.stream")
        return TokenLogprobs(*_TokenLogprobs.apply(logits, tokens, top, check))
    return _forward(logits, tokens, top, check, stream)


def _check_row_values(v, m, what, device):
    if v is not None and not (v.dtype == torch.float32 and v.shape == (m,) and v.device == device):
        _ops.check_tensor(v, what, device)
        raise ValueError(f"{what} must be {m} float32 numbers")


def token_logprobs_backward(logits: torch.Tensor, tokens: torch.Tensor, lse: torch.Tensor, entropy=None,
                            grad_logprob=None, grad_entropy=None, out=None, check: bool = True,
                            stream=None) -> torch.Tensor:
    """The gradient of the logits, in their type, from the gradients of
    logprob and entropy (either may be None) and the lse and entropy that
    ``token_logprobs`` gave.  `out` may be the logits themselves (elsewhere
    in their memory, they are copied first)."""
    dev = logits.device
    if not _good(logits, tokens, dev):
        _check(logits, tokens)
    m, vocab = logits.shape
    if lse is None:
        raise ValueError("lse is needed")
    if grad_entropy is not None and entropy is None:
        raise ValueError("the gradient of the entropy needs the entropy")
    _check_row_values(lse, m, "lse", dev)
    _check_row_values(entropy, m, "entropy", dev)
    _check_row_values(grad_logprob, m, "grad_logprob", dev)
    _check_row_values(grad_entropy, m, "grad_entropy", dev)
    if _ops.forward_mode():
        _ops.no_tangents("token_logprobs_backward", logits, lse, entropy, grad_logprob, grad_entropy, out)
    if out is not None:
        _ops.check_tensor(out, "out", dev)
        if out.dtype != logits.dtype or out.shape != logits.shape or not _ops.rows_apart(out):
            raise ValueError("out must be like the logits, with unit column stride and rows that do not overlap")
        if out.requires_grad and torch.is_grad_enabled():
            raise RuntimeError("out requires a gradient: call token_logprobs_backward under torch.no_grad(), or with "
                               "another out")

    def call(raw):
        z, t = _ops.rows_of(logits), tokens.contiguous()
        s = lse.contiguous()  # each copy is kept until the call is on the stream
        ent = entropy.contiguous() if entropy is not None else None
        gl = grad_logprob.contiguous() if grad_logprob is not None else None
        ge = grad_entropy.contiguous() if grad_entropy is not None else None
        o = torch.empty((m, vocab), dtype=z.dtype, device=dev) if out is None else out
        if out is not None:
            _ops.written(out)
        err = _ops.error_word(check, dev)
        a = B.wc_logprobs_grad(z.data_ptr(), z.stride(0), o.data_ptr(), o.stride(0), t.data_ptr(), s.data_ptr(),
                               ent.data_ptr() if ent is not None else 0, gl.data_ptr() if gl is not None else 0,
                               ge.data_ptr() if ge is not None else 0, m, vocab, _ops.TYPES[z.dtype])
        rc = B.lib().wc_token_logprobs_backward(a, err.data_ptr() if check else 0, raw)
        if rc == B.WC_ERR_ARG and _ops.may_overlap(z, o):  # out across the logits: from a copy of them
            z = z.clone(memory_format=torch.contiguous_format)
            a.logits, a.stride = z.data_ptr(), vocab
            rc = B.lib().wc_token_logprobs_backward(a, err.data_ptr() if check else 0, raw)
        _ops.done(rc, err, "token_logprobs_backward")
        return o

    return _ops.on_stream(dev, stream, call)


class _TokenLogprobs(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, tokens, top, check):
        r = _forward(logits, tokens, top, check, None, views=False)
        ctx.save_for_backward(logits, tokens, r.lse, r.entropy)
        if r.top_ids is not None:
            ctx.mark_non_differentiable(r.top_ids)
        ctx.set_materialize_grads(False)
        return tuple(r)

    @staticmethod
    def backward(ctx, grad_logprob, grad_entropy, grad_lse, grad_top, _):
        if grad_lse is not None or grad_top is not None:
            raise RuntimeError("token_logprobs has gradients of logprob and entropy only: detach lse and top_logprobs, "
                               "or take them from torch where a loss needs them")
        logits, tokens, lse, entropy = ctx.saved_tensors
        if grad_logprob is None and grad_entropy is None:
            return None, None, None, None
        grad = token_logprobs_backward(logits, tokens, lse, entropy, grad_logprob, grad_entropy, check=False)
        if torch.is_grad_enabled():  # create_graph: the kernel's result has no graph of its own
            grad = _Once.apply(grad, logits, grad_logprob, grad_entropy)
        return grad, None, None, None


class _Once(torch.autograd.Function):
    """A gradient that depends on its inputs, and whose own gradient is an error rather than nothing."""
    @staticmethod
    def forward(ctx, grad, *inputs):
        return grad.view_as(grad)

    @staticmethod
    def backward(ctx, *_):
        raise RuntimeError("token_logprobs cannot be differentiated twice")
