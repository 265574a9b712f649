"""Checks and launch context that the torch front ends of the slot and convolution operators share.

The front ends of single tokens run once per layer and step, so these checks are written to cost
little where they pass; what is wrong is found out only once something is."""
from __future__ import annotations

from . import _abi


def io_code(t) -> int:
    """The library's code of an I/O tensor's dtype."""
    import torch
    if t.dtype is torch.bfloat16:
        return _abi.SSM_BF16
    if t.dtype is torch.float32:
        return _abi.SSM_F32
    raise ValueError("inputs must be bfloat16 or float32")


def need(name: str, t, dtype, shape, device: int) -> None:
    """t is None, or a contiguous tensor of this dtype and shape (a tuple) on this CUDA device."""
    if t is None or (t.dtype is dtype and t.shape == shape and t.get_device() == device and t.is_contiguous()):
        return
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    if t.get_device() != device:
        raise ValueError(f"{name} must be on cuda:{device}")
    raise ValueError(f"{name} must be contiguous")


def need_cuda(name: str, t, dims: int) -> int:
    """t is a contiguous CUDA tensor of this many dimensions; returns its device's index."""
    if t.dim() != dims:
        raise ValueError(f"{name} must have {dims} dimensions")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.get_device()


def pool_stride(name: str, t, dtype, n: int, last: int, device: int) -> int:
    """t is a pool (n_slots, n, last) whose slots are contiguous and may lie apart; returns the elements
    from one slot to the next."""
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}")
    if t.dim() != 3 or t.shape[1:] != (n, last):
        raise ValueError(f"{name} must have shape (n_slots, {n}, {last}), not {tuple(t.shape)}")
    if t.get_device() != device:
        raise ValueError(f"{name} must be on cuda:{device}")
    if t.is_contiguous():
        return n * last
    if not inner_contiguous(t, 1):
        raise ValueError(f"every slot of {name} must be contiguous")
    # a single slot's stride says nothing
    return t.stride(0) if t.shape[0] > 1 else n * last


def inner_contiguous(t, first: int) -> bool:
    """Whether the dimensions from `first` on are laid out without gaps."""
    want = 1
    for i in range(t.dim() - 1, first - 1, -1):
        if t.shape[i] != 1 and t.stride(i) != want:
            return False
        want *= t.shape[i]
    return True


def ptr(t):
    return None if t is None else t.data_ptr()


def launch(fn, device: int, stream, *args):
    """fn(*args, raw stream) on `stream` (None: the device's current one), with that stream and its
    device current, so what fn allocates belongs to the stream that uses it."""
    import torch
    if stream is None:
        if device == torch.cuda.current_device():
            return fn(*args, torch._C._cuda_getCurrentRawStream(device))
        with torch.cuda.device(device):
            return fn(*args, torch._C._cuda_getCurrentRawStream(device))
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(_abi._stream(stream) or 0, device=device)
    if stream.device.index != device:
        raise ValueError(f"stream must be on cuda:{device}")
    with torch.cuda.stream(stream):
        return fn(*args, stream.cuda_stream)
