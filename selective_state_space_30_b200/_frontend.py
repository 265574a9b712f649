"""Loads the compiled front ends (_front.so, csrc/front.cpp) and runs their calls on a stream."""
from __future__ import annotations

import ctypes

from . import _abi

_ENTRIES = ("ssm_causal_conv1d_fwd", "ssm_causal_conv1d_bwd_workspace_size", "ssm_causal_conv1d_bwd",
            "ssm_causal_conv1d_packed_fwd", "ssm_causal_conv1d_update", "ssm_selective_scan_packed_workspace_size",
            "ssm_selective_scan_packed_fwd", "ssm_selective_state_update_slots", "ssm_state_slots_copy")

_front = None


def load():
    """The module, bound to the library that the package has loaded (raises if either has not been built)."""
    global _front
    if _front is None:
        import torch  # noqa: F401  (its libraries are what the module is linked to)
        lib = _abi.load_library()
        try:
            from . import _front as front
        except ImportError as e:
            raise RuntimeError("the compiled front ends are missing: build them with `python -m "
                               f"selective_state_space_30_b200.build` ({e})") from e
        front.bind({n: ctypes.cast(getattr(lib, n), ctypes.c_void_p).value for n in _ENTRIES}, _abi.SsmError)
        _front = front
    return _front


def on_stream(fn, stream, like, *args):
    """fn(*args) with `stream` current, so what it allocates belongs to the stream that uses it.  stream:
    a torch stream, or a raw handle of `like`'s device.  The tensors given are recorded as in use on it, so
    that torch does not hand their memory out again before the call has run."""
    import torch
    if not isinstance(like, torch.Tensor) or not like.is_cuda:
        return fn(*args)                                 # which refuses it
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(_abi._stream(stream) or 0, device=like.device)
    if stream.device != like.device:
        raise ValueError(f"stream must be on {like.device}")
    with torch.cuda.stream(stream):
        result = fn(*args)
    if stream.cuda_stream != torch.cuda.current_stream(like.device).cuda_stream:
        for t in args:
            if isinstance(t, torch.Tensor):
                t.record_stream(stream)
    return result
