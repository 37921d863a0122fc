"""Log probabilities of given tokens, with entropy and the most likely
alternatives, and the gradient of the logits.

``token_logprobs`` reads the logits once; autograd runs
``token_logprobs_backward`` for logits that require a gradient.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple

import torch

from . import _binding as B
from . import _ops

MAX_TOP = 64


class TokenLogprobs(NamedTuple):
    logprob: torch.Tensor        # m, fp32: log probability of each row's token (0 for token -1)
    entropy: torch.Tensor        # m, fp32, in nats
    lse: torch.Tensor            # m, fp32: log of the sum of the exponentials
    top_logprobs: torch.Tensor   # m x top, fp32, largest first
    top_ids: torch.Tensor        # m x top, int64; equal logits by their index, NaN last


def _check(logits, tokens):
    _ops.check_tensor(logits, "logits")
    _ops.check_tensor(tokens, "tokens", logits.device)
    if logits.dim() != 2 or logits.dtype not in _ops.TYPES:
        raise TypeError("logits must be a 2-D bfloat16, float16 or float32 tensor (rows x vocabulary)")
    if tokens.dtype != torch.int64 or tokens.shape != logits.shape[:1]:
        raise ValueError(f"tokens must be {logits.shape[0]} int64 numbers, one per row")
    if not logits.shape[1]:
        raise ValueError("the vocabulary is empty")


def _forward(logits, tokens, top, check, stream, views=True):
    z, t = _ops.rows_of(logits), tokens.contiguous()
    m, vocab = z.shape

    def call(raw):
        dev = z.device
        if not views:  # autograd's outputs are tensors of their own
            rows = [torch.empty(m, dtype=torch.float32, device=dev) for _ in range(3)]
            best = torch.empty((m, top), dtype=torch.float32, device=dev)
        elif top:  # one allocation for the fp32 outputs
            *rows, best = torch.empty(m * (3 + top), dtype=torch.float32, device=dev).split((m, m, m, m * top))
            best = best.view(m, top)
        else:
            rows = torch.empty((3, m), dtype=torch.float32, device=dev).unbind(0)
            best = torch.empty((m, 0), dtype=torch.float32, device=dev)
        out = TokenLogprobs(*rows, best, torch.empty((m, top), dtype=torch.int64, device=dev))
        nbytes = B.wc_token_logprobs_scratch(m, vocab, top)
        scratch = torch.empty(nbytes, dtype=torch.uint8, device=dev) if nbytes else None
        err = torch.zeros(1, dtype=torch.int32, device=dev) if check else None
        a = B.wc_logprobs(z.data_ptr(), z.stride(0), t.data_ptr(), m, vocab, top, _ops.TYPES[z.dtype], 0,
                          out.logprob.data_ptr(), out.entropy.data_ptr(), out.lse.data_ptr(),
                          out.top_logprobs.data_ptr(), out.top_ids.data_ptr())
        B.wc_token_logprobs(a, scratch, nbytes, err, raw)
        _ops.raise_bits(err, "token_logprobs")
        return out

    return _ops.on_stream(z.device, stream, call)


def token_logprobs(logits: torch.Tensor, tokens: torch.Tensor, top: int = 0, check: bool = True,
                   stream=None) -> TokenLogprobs:
    """Log probability of tokens[r] under softmax(logits[r]), the row's
    entropy, and its `top` (at most 64) most likely alternatives.

    Token -1 stands for no token (logprob 0).  -inf masks a logit; a row of
    nothing but -inf has lse and log probabilities -inf and entropy 0; a row
    with NaN or +inf has NaN statistics.  With check (which waits for the
    GPU) a token out of range raises; without, its logprob is NaN."""
    _check(logits, tokens)
    if not 0 <= top <= min(MAX_TOP, logits.shape[1]):
        raise ValueError(f"top must be between 0 and {min(MAX_TOP, logits.shape[1])}, got {top}")
    if logits.requires_grad and torch.is_grad_enabled():
        if stream is not None:
            raise ValueError("with gradients the call runs on the current stream: use torch.cuda.stream")
        return TokenLogprobs(*_TokenLogprobs.apply(logits, tokens, top, check))
    return _forward(logits, tokens, top, check, stream)


def token_logprobs_backward(logits: torch.Tensor, tokens: torch.Tensor, lse: torch.Tensor, entropy=None,
                            grad_logprob=None, grad_entropy=None, out=None, check: bool = True,
                            stream=None) -> torch.Tensor:
    """The gradient of the logits, in their type, from the gradients of
    logprob and entropy (either may be None) and the lse and entropy that
    ``token_logprobs`` gave.  `out` may be the logits themselves."""
    _check(logits, tokens)
    z, t = _ops.rows_of(logits), tokens.contiguous()
    m, vocab = z.shape
    if grad_entropy is not None and entropy is None:
        raise ValueError("the gradient of the entropy needs the entropy")
    kept = []  # contiguous copies live until the call is enqueued

    def row_values(v, what):
        if v is None:
            return 0
        _ops.check_tensor(v, what, z.device)
        if v.dtype != torch.float32 or v.shape != (m,):
            raise ValueError(f"{what} must be {m} float32 numbers")
        kept.append(v if v.is_contiguous() else v.contiguous())
        return kept[-1].data_ptr()

    if lse is None:
        raise ValueError("lse is needed")
    p_lse, p_ent = row_values(lse, "lse"), row_values(entropy, "entropy")
    p_glp, p_gent = row_values(grad_logprob, "grad_logprob"), row_values(grad_entropy, "grad_entropy")
    if out is not None:
        _ops.check_tensor(out, "out", z.device)
        if out.dtype != z.dtype or out.shape != z.shape or (out.numel() and _ops.rows_of(out) is not out):
            raise ValueError("out must be like the logits, with unit column stride and rows that do not overlap")

    def call(raw):
        o = torch.empty((m, vocab), dtype=z.dtype, device=z.device) if out is None else out
        err = torch.zeros(1, dtype=torch.int32, device=z.device) if check else None
        a = B.wc_logprobs_grad(z.data_ptr(), z.stride(0), o.data_ptr(), o.stride(0), t.data_ptr(), p_lse, p_ent,
                               p_glp, p_gent, m, vocab, _ops.TYPES[z.dtype])
        B.wc_token_logprobs_backward(a, err, raw)
        _ops.raise_bits(err, "token_logprobs_backward")
        return o

    return _ops.on_stream(z.device, stream, call)


class _TokenLogprobs(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, tokens, top, check):
        r = _forward(logits, tokens, top, check, None, views=False)
        ctx.save_for_backward(logits, tokens, r.lse, r.entropy)
        ctx.mark_non_differentiable(r.lse, r.top_logprobs, r.top_ids)
        ctx.set_materialize_grads(False)
        return tuple(r)

    @staticmethod
    def backward(ctx, grad_logprob, grad_entropy, *_):
        logits, tokens, lse, entropy = ctx.saved_tensors
        if grad_logprob is None and grad_entropy is None:
            return None, None, None, None
        return (token_logprobs_backward(logits, tokens, lse, entropy, grad_logprob, grad_entropy, check=False),
                None, None, None)
