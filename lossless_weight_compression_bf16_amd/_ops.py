"""What the operators beside the weights share: element types, streams,
error words and the checks of a call.

A call's checks are one expression over the tensors' attributes; only when it
is false are they gone through one by one, to say what is wrong.  (An
attribute of a tensor takes 0.1 us to read, and the smallest calls take 5 us
on the GPU.)
"""
from __future__ import annotations

import torch
from torch.autograd import forward_ad
from torch.autograd.graph import increment_version

from . import _binding as B

TYPES = {torch.bfloat16: B.WC_T_BF16, torch.float16: B.WC_T_FP16, torch.float32: B.WC_T_FP32}
HALVES = (torch.bfloat16, torch.float16)


def check_tensor(t, what: str, device=None):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{what} must be a tensor on a HIP device")
    if device is not None and t.device != device:
        raise ValueError(f"{what} is on {t.device}, not on {device}")


def rows_of(t: torch.Tensor) -> torch.Tensor:
    """t (2-D) with unit column stride and rows that do not overlap: itself, or a copy."""
    if rows_apart(t):
        return t
    return t.contiguous()


def rows_apart(t: torch.Tensor) -> bool:
    """Whether t (2-D) has unit column stride and rows that do not overlap."""
    (m, n), (row, col) = t.shape, t.stride()
    return (col == 1 or n == 1) and (row >= n or m == 1) or m == 0 or n == 0


def rows16(t: torch.Tensor) -> torch.Tensor:
    """t (2-D, 16-bit) with 16-byte aligned rows of unit column stride: itself, or a copy."""
    row, col = t.stride()
    if col == 1 and row % 8 == 0 and row >= t.shape[1] and t.data_ptr() % 16 == 0:
        return t
    return t.clone(memory_format=torch.contiguous_format)


# the current stream's handle without a stream object (2.7 us of a call's host time)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def on_stream(device: torch.device, stream, call):
    """call(raw stream) with the device and stream of the call current, so
    that what it allocates and copies belongs to that stream: copies of
    arguments are made within call.  stream: None (the device's current one),
    a torch stream or a raw hipStream_t."""
    if stream is None:
        if device.index == torch.cuda.current_device():
            return call(_raw_stream(device.index))
        stream = torch.cuda.current_stream(device)
    elif isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=device)
    if stream.device != device:
        raise ValueError(f"the stream is on {stream.device}, the tensors on {device}")
    with torch.cuda.stream(stream):
        return call(stream.cuda_stream)


def may_overlap(a: torch.Tensor, b: torch.Tensor) -> bool:
    """Whether the memory from the first to the last element of a and of b (2-D) has a byte in common."""
    def ends(t):
        return t.data_ptr(), t.data_ptr() + t.element_size() * (1 + sum((n - 1) * s for n, s in zip(t.shape, t.stride())))
    (a0, a1), (b0, b1) = ends(a), ends(b)
    return a0 < b1 and b0 < a1


def no_backward(what: str):
    """For a call that autograd would have to follow, and cannot."""
    raise RuntimeError(f"{what} has no backward pass: call it under torch.no_grad(), or with tensors that do not require "
                       "a gradient")


def forward_mode() -> bool:
    """Whether the call is made within a level of forward-mode differentiation (a look at a number: asking every
    tensor would take as long as the checks of a call)."""
    return getattr(forward_ad, "_current_level", 0) >= 0


def no_tangents(what: str, *tensors):
    """Raises where a tensor carries a forward-mode tangent, which the call would drop."""
    if any(t is not None and forward_ad.unpack_dual(t).tangent is not None for t in tensors):
        raise RuntimeError(f"{what} has no forward-mode derivative")


_increment_version = getattr(torch._C, "_increment_version", None) or (lambda tensors: increment_version(*tensors))


def written(t: torch.Tensor):
    """What autograd has to know of a tensor that a call writes in place.  (increment_version without its own check
    of a type, half of its time.)"""
    _increment_version((t,))


def error_word(check: bool, device):
    return torch.zeros(1, dtype=torch.int32, device=device) if check else None


def done(rc: int, err, what: str):
    """The call's status, and with an error word (which waits for the GPU)
    what its kernels reported."""
    if rc:
        B._check(rc, "wc_" + what)
    if err is not None:
        bits = int(err.item())
        if bits:
            raise B.WcError(f"{what}: device reported {', '.join(B.error_names(bits))} (bits {bits:#x})")
