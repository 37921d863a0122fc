"""What the operators beside the weights share: element types, streams and
error words of a call."""
from __future__ import annotations

import torch

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
    if t.stride(1) == 1 and t.stride(0) >= t.shape[1] or t.numel() == 0:
        return t
    return t.contiguous()


def rows16(t: torch.Tensor) -> torch.Tensor:
    """t (2-D, 16-bit) with 16-byte aligned rows of unit column stride: itself, or a copy."""
    if t.stride(1) == 1 and t.stride(0) % 8 == 0 and t.stride(0) >= t.shape[1] and t.data_ptr() % 16 == 0:
        return t
    return t.clone(memory_format=torch.contiguous_format)


# the current stream's handle without a stream object (2.7 us of a call's host time)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def on_stream(device: torch.device, stream, call):
    """call(raw stream) with the device and stream of the call current, so
    that what it allocates belongs to that stream.  stream: None (the
    device's current one), a torch stream or a raw hipStream_t."""
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


def raise_bits(err, what: str):
    """Waits for the call and raises what its kernels reported."""
    if err is not None:
        bits = int(err.item())
        if bits:
            raise B.WcError(f"{what}: device reported {', '.join(B.error_names(bits))} (bits {bits:#x})")
