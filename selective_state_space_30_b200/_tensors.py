"""Checks and launch context that the torch front ends of the slot and convolution operators share."""
from __future__ import annotations

from . import _abi


def io_code(t) -> int:
    """The library's code of an I/O tensor's dtype."""
    import torch
    if t.dtype == torch.bfloat16:
        return _abi.SSM_BF16
    if t.dtype == torch.float32:
        return _abi.SSM_F32
    raise ValueError("inputs must be bfloat16 or float32")


def need(name: str, t, dtype, shape, device) -> None:
    """t is None, or a contiguous tensor of this dtype and shape on this device."""
    if t is None:
        return
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def need_cuda(name: str, t, dims: int) -> None:
    if t.dim() != dims:
        raise ValueError(f"{name} must have {dims} dimensions")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def need_pool(name: str, t, dtype, slot_shape, device) -> None:
    """A pool (n_slots, *slot_shape) whose slots are contiguous; the slots may lie apart."""
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}")
    if t.dim() != 1 + len(slot_shape) or t.shape[1:] != slot_shape:
        raise ValueError(f"{name} must have shape (n_slots, {', '.join(map(str, slot_shape))}), not {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}")
    if not inner_contiguous(t, 1):
        raise ValueError(f"every slot of {name} must be contiguous")


def inner_contiguous(t, first: int) -> bool:
    """Whether the dimensions from `first` on are laid out without gaps."""
    if t.is_contiguous():
        return True
    want = 1
    for i in range(t.dim() - 1, first - 1, -1):
        if t.shape[i] != 1 and t.stride(i) != want:
            return False
        want *= t.shape[i]
    return True


def launch(fn, device, stream, *args):
    """fn(*args, raw stream) on `stream` (None: the device's current one), with that stream and its
    device current, so what fn allocates belongs to the stream that uses it."""
    import torch
    if stream is None:
        if device.index == torch.cuda.current_device():
            return fn(*args, torch.cuda.current_stream(device).cuda_stream)
        with torch.cuda.device(device):
            return fn(*args, torch.cuda.current_stream(device).cuda_stream)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(_abi._stream(stream) or 0, device=device)
    if stream.device != device:
        raise ValueError(f"stream must be on {device}")
    with torch.cuda.stream(stream):
        return fn(*args, stream.cuda_stream)
