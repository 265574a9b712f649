"""Torch front ends of the operators that keep each sequence's state in a slot of a pool.

Layouts, slots and lengths are those of include/ssm_scan.h ("packed prompts and state slots"):
`cu_seqlens` and `slots` are int32 and `has_state` uint8 or bool CUDA tensors, read on the device;
a negative slot marks a padding row.  Pools are (n_slots, ...) tensors whose slots are contiguous
and may lie apart (a layer's view of a pool that holds several layers).  The calls update the
pools in place, run on `stream` (default: the device's current one) and can be captured into a
CUDA graph.  `out` is allocated with torch unless given, zeroed so that padding reads as zero; a
workspace is allocated unless given.
"""
from __future__ import annotations

from ctypes import byref

from . import _abi
from ._tensors import inner_contiguous, io_code, launch, need, need_cuda, pool_stride, ptr


def _n_seq(cu_seqlens) -> int:
    if cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 1:
        raise ValueError("cu_seqlens must have n_seq + 1 entries")
    return cu_seqlens.shape[0] - 1


def _need_indices(n, device, cu_seqlens, slots, has_state):
    import torch
    need("cu_seqlens", cu_seqlens, torch.int32, (n + 1,), device)
    need("slots", slots, torch.int32, (n,), device)
    if has_state is not None:
        need("has_state", has_state, torch.bool if has_state.dtype is torch.bool else torch.uint8, (n,), device)


def _width(w, bias, dim, device) -> int:
    import torch
    if w.dim() != 2:
        raise ValueError("w must have shape (dim, width)")
    width = w.shape[1]
    if not 1 <= width <= 4:
        raise ValueError("w must have a width of 1 to 4")
    need("w", w, torch.float32, (dim, width), device)
    need("bias", bias, torch.float32, (dim,), device)
    return width


def causal_conv1d_packed(x, w, cu_seqlens, conv_states, slots=None, has_state=None, bias=None, silu: bool = True,
                         out=None, stream=None):
    """The causal convolution over prompts packed along time: x (dim, total) -> out.  Each sequence's
    earlier inputs come from its slot of conv_states (n_slots, dim, width - 1; x's dtype, the oldest
    first) where has_state is nonzero, and its last width - 1 inputs replace them."""
    dev = need_cuda("x", x, 2)
    dim, total = x.shape
    io, n, width = io_code(x), _n_seq(cu_seqlens), _width(w, bias, dim, dev)
    need("out", out, x.dtype, (dim, total), dev)
    stride = pool_stride("conv_states", conv_states, x.dtype, dim, width - 1, dev)
    _need_indices(n, dev, cu_seqlens, slots, has_state)

    def call(raw):
        o = x.new_zeros(dim, total) if out is None else out
        lib = _abi._lib or _abi.load_library()
        _abi._check(lib.ssm_causal_conv1d_packed_fwd(
            dim, total, n, width, io, x.data_ptr(), w.data_ptr(), ptr(bias), 1 if silu else 0, cu_seqlens.data_ptr(),
            ptr(slots), ptr(has_state), conv_states.data_ptr(), conv_states.shape[0], stride, o.data_ptr(), raw),
            "ssm_causal_conv1d_packed_fwd")
        return o
    return launch(call, dev, stream)


def causal_conv1d_update(x, w, conv_states, slots=None, bias=None, silu: bool = True, out=None, stream=None):
    """The causal convolution of one new token per row: x (batch, dim) -> out, each row's slot of
    conv_states moved on by its token."""
    import torch
    dev = need_cuda("x", x, 2)
    batch, dim = x.shape
    io, width = io_code(x), _width(w, bias, dim, dev)
    need("out", out, x.dtype, (batch, dim), dev)
    stride = pool_stride("conv_states", conv_states, x.dtype, dim, width - 1, dev)
    need("slots", slots, torch.int32, (batch,), dev)

    def call(raw):
        o = x.new_zeros(batch, dim) if out is None else out
        lib = _abi._lib or _abi.load_library()
        _abi._check(lib.ssm_causal_conv1d_update(
            batch, dim, width, io, x.data_ptr(), w.data_ptr(), ptr(bias), 1 if silu else 0, ptr(slots),
            conv_states.data_ptr(), conv_states.shape[0], stride, o.data_ptr(), raw), "ssm_causal_conv1d_update")
        return o
    return launch(call, dev, stream)


def selective_scan_packed(u, delta, A, B, C, cu_seqlens, states, slots=None, has_state=None, D=None, z=None,
                          delta_bias=None, softplus: bool = True, max_seqlen: int = 0, out=None, workspace=None,
                          stream=None):
    """The forward scan over prompts packed along time: u (dim, total), delta (nheads, total), B and C
    (ngroups, dstate, total) -> out.  Each sequence starts from its slot of states (n_slots, dim, dstate;
    fp32) where has_state is nonzero, else from zero, and leaves its final state there.  max_seqlen, if
    known, only saves the cutting of sequences that are all short.  The workspace (uint8, at least
    ssm_selective_scan_packed_workspace_size bytes) must not serve two calls, or two graphs, at once."""
    import torch
    dev = need_cuda("u", u, 2)
    need_cuda("delta", delta, 2)
    need_cuda("B", B, 3)
    dim, total = u.shape
    nheads, (ngroups, dstate) = delta.shape[0], B.shape[:2]
    io, dtype, n, f32 = io_code(u), u.dtype, _n_seq(cu_seqlens), torch.float32
    need("delta", delta, dtype, (nheads, total), dev)
    need("A", A, f32, (dim, dstate) if nheads == dim else (nheads,), dev)
    need("B", B, dtype, (ngroups, dstate, total), dev)
    need("C", C, dtype, (ngroups, dstate, total), dev)
    need("D", D, f32, (dim,), dev)
    need("z", z, dtype, (dim, total), dev)
    need("delta_bias", delta_bias, f32, (nheads,), dev)
    need("out", out, dtype, (dim, total), dev)
    stride = pool_stride("states", states, f32, dim, dstate, dev)
    _need_indices(n, dev, cu_seqlens, slots, has_state)
    if workspace is not None and (workspace.get_device() != dev or not workspace.is_contiguous()):
        raise ValueError(f"workspace must be a contiguous tensor on cuda:{dev}")
    dims = _abi.make_dims(n, dim, total, dstate, nheads, ngroups, io)
    longest = max(int(max_seqlen or 0), 0)

    def call(raw):
        nbytes = _abi.ssm_selective_scan_packed_workspace_size(dims, longest)
        ws = torch.empty(nbytes, dtype=torch.uint8, device=u.device) if workspace is None and nbytes else workspace
        o = u.new_zeros(dim, total) if out is None else out
        _abi._check(_abi._lib.ssm_selective_scan_packed_fwd(
            byref(dims), u.data_ptr(), delta.data_ptr(), A.data_ptr(), B.data_ptr(), C.data_ptr(), ptr(D), ptr(z),
            ptr(delta_bias), 1 if softplus else 0, cu_seqlens.data_ptr(), ptr(slots), ptr(has_state), states.data_ptr(),
            states.shape[0], stride, longest, o.data_ptr(), ptr(ws), ws.numel() * ws.element_size() if ws is not None else 0,
            raw), "ssm_selective_scan_packed_fwd")
        return o
    return launch(call, dev, stream)


def selective_state_update_slots(states, u, delta, A, B, C, slots=None, D=None, z=None, delta_bias=None,
                                 softplus: bool = True, out=None, stream=None):
    """One step of the recurrence for rows whose states sit in slots: u (batch, dim), delta (batch, nheads),
    B and C (batch, ngroups, dstate) -> out, each row's slot of states (n_slots, dim, dstate; fp32) updated
    in place."""
    import torch
    dev = need_cuda("u", u, 2)
    need_cuda("delta", delta, 2)
    need_cuda("B", B, 3)
    batch, dim = u.shape
    nheads, (ngroups, dstate) = delta.shape[1], B.shape[1:]
    io, dtype, f32 = io_code(u), u.dtype, torch.float32
    need("delta", delta, dtype, (batch, nheads), dev)
    need("A", A, f32, (dim, dstate) if nheads == dim else (nheads,), dev)
    need("B", B, dtype, (batch, ngroups, dstate), dev)
    need("C", C, dtype, (batch, ngroups, dstate), dev)
    need("D", D, f32, (dim,), dev)
    need("z", z, dtype, (batch, dim), dev)
    need("delta_bias", delta_bias, f32, (nheads,), dev)
    need("out", out, dtype, (batch, dim), dev)
    need("slots", slots, torch.int32, (batch,), dev)
    stride = pool_stride("states", states, f32, dim, dstate, dev)
    dims = _abi.ssm_dims_t(batch, dim, 1, dstate, nheads, ngroups, io, 0)

    def call(raw):
        o = u.new_zeros(batch, dim) if out is None else out
        lib = _abi._lib or _abi.load_library()
        _abi._check(lib.ssm_selective_state_update_slots(
            byref(dims), states.data_ptr(), ptr(slots), states.shape[0], stride, u.data_ptr(), delta.data_ptr(),
            A.data_ptr(), B.data_ptr(), C.data_ptr(), ptr(D), ptr(z), ptr(delta_bias), 1 if softplus else 0, o.data_ptr(),
            raw), "ssm_selective_state_update_slots")
        return o
    return launch(call, dev, stream)


def state_slots_copy(pool, src, dst, slot_dim: int = 0, stream=None):
    """Slot dst[i] of the pool becomes what slot src[i] held before the call, or zeros for src[i] = -1, for
    all i at once: forks, moves and clears, in every layer.  slot_dim is the pool's dimension that counts
    slots; the dimension before it, if any (slot_dim = 1), counts layers.  Returns the pool."""
    import torch
    if not pool.is_cuda:
        raise ValueError("pool must be a CUDA tensor")
    if slot_dim not in (0, 1) or pool.dim() <= slot_dim:
        raise ValueError("slot_dim must be 0, or 1 behind a dimension of layers")
    if not pool.is_contiguous() and not inner_contiguous(pool, slot_dim + 1):
        raise ValueError("every slot of pool must be contiguous")
    dev, n = pool.get_device(), src.numel()
    need("src", src, torch.int32, (n,), dev)
    need("dst", dst, torch.int32, (n,), dev)
    e, n_slots = pool.element_size(), pool.shape[slot_dim]
    slot_bytes = e
    for s in pool.shape[slot_dim + 1:]:
        slot_bytes *= s
    layers, layer_stride = (pool.shape[0], pool.stride(0) * e) if slot_dim else (1, 0)
    # a single slot's stride says nothing
    slot_stride = pool.stride(slot_dim) * e if n_slots > 1 else slot_bytes

    def call(raw):
        lib = _abi._lib or _abi.load_library()
        _abi._check(lib.ssm_state_slots_copy(pool.data_ptr(), layers, n_slots, slot_bytes, slot_stride, layer_stride,
                                             src.data_ptr(), dst.data_ptr(), n, raw), "ssm_state_slots_copy")
        return pool
    return launch(call, dev, stream)
