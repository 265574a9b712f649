"""Torch front ends of the operators that keep each sequence's state in a slot of a pool.

Layouts, slots and lengths are those of include/ssm_scan.h ("packed prompts and state slots"):
`cu_seqlens` and `slots` are int32 and `has_state` uint8 or bool CUDA tensors, read on the device;
a negative slot marks a padding row.  Pools are (n_slots, ...) tensors whose slots are contiguous
and may lie apart (a layer's view of a pool that holds several layers).  The calls update the
pools in place, allocate `out` (and a workspace) with torch unless given, run on `stream` (default:
the device's current one) and can be captured into a CUDA graph.
"""
from __future__ import annotations

from . import _abi
from ._tensors import inner_contiguous, io_code, launch, need, need_cuda, need_pool


def _indices(n, device, cu_seqlens=None, slots=None, has_state=None):
    import torch
    need("cu_seqlens", cu_seqlens, torch.int32, (n + 1,), device)
    need("slots", slots, torch.int32, (n,), device)
    if has_state is not None:
        need("has_state", has_state, torch.bool if has_state.dtype == torch.bool else torch.uint8, (n,), device)


def _n_seq(cu_seqlens) -> int:
    if cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 1:
        raise ValueError("cu_seqlens must have n_seq + 1 entries")
    return cu_seqlens.shape[0] - 1


def causal_conv1d_packed(x, w, cu_seqlens, conv_states, slots=None, has_state=None, bias=None, silu: bool = True,
                         out=None, stream=None):
    """The causal convolution over prompts packed along time: x (dim, total) -> out.  Each sequence's
    earlier inputs come from its slot of conv_states (n_slots, dim, width - 1; x's dtype, the oldest
    first) where has_state is nonzero, and its last width - 1 inputs replace them."""
    import torch
    need_cuda("x", x, 2)
    dim, total = x.shape
    io, dev, n = io_code(x), x.device, _n_seq(cu_seqlens)
    if w.dim() != 2:
        raise ValueError("w must have shape (dim, width)")
    width = w.shape[1]
    need("w", w, torch.float32, (dim, width), dev)
    need("bias", bias, torch.float32, (dim,), dev)
    need("out", out, x.dtype, (dim, total), dev)
    need_pool("conv_states", conv_states, x.dtype, (dim, max(width - 1, 0)), dev)
    _indices(n, dev, cu_seqlens, slots, has_state)

    def call(out, raw):
        if out is None:
            out = torch.zeros_like(x)
        _abi.ssm_causal_conv1d_packed_fwd(dim, total, n, width, io, x, w, bias, silu, cu_seqlens, slots, has_state,
                                          conv_states, conv_states.shape[0], max(conv_states.stride(0), dim * (width - 1)),
                                          out, raw)
        return out
    return launch(call, dev, stream, out)


def causal_conv1d_update(x, w, conv_states, slots=None, bias=None, silu: bool = True, out=None, stream=None):
    """The causal convolution of one new token per row: x (batch, dim) -> out, each row's slot of
    conv_states moved on by its token."""
    import torch
    need_cuda("x", x, 2)
    batch, dim = x.shape
    io, dev = io_code(x), x.device
    if w.dim() != 2:
        raise ValueError("w must have shape (dim, width)")
    width = w.shape[1]
    need("w", w, torch.float32, (dim, width), dev)
    need("bias", bias, torch.float32, (dim,), dev)
    need("out", out, x.dtype, (batch, dim), dev)
    need_pool("conv_states", conv_states, x.dtype, (dim, max(width - 1, 0)), dev)
    need("slots", slots, torch.int32, (batch,), dev)

    def call(out, raw):
        if out is None:
            out = torch.zeros_like(x)
        _abi.ssm_causal_conv1d_update(batch, dim, width, io, x, w, bias, silu, slots, conv_states, conv_states.shape[0],
                                      max(conv_states.stride(0), dim * (width - 1)), out, raw)
        return out
    return launch(call, dev, stream, out)


def selective_scan_packed(u, delta, A, B, C, cu_seqlens, states, slots=None, has_state=None, D=None, z=None,
                          delta_bias=None, softplus: bool = True, max_seqlen: int = 0, out=None, workspace=None,
                          stream=None):
    """The forward scan over prompts packed along time: u (dim, total), delta (nheads, total), B and C
    (ngroups, dstate, total) -> out.  Each sequence starts from its slot of states (n_slots, dim, dstate;
    fp32) where has_state is nonzero, else from zero, and leaves its final state there.  max_seqlen, if
    known, only saves the cutting of sequences that are all short.  The workspace (uint8, at least
    ssm_selective_scan_packed_workspace_size bytes) must not serve two calls, or two graphs, at once."""
    import torch
    need_cuda("u", u, 2)
    need_cuda("delta", delta, 2)
    need_cuda("B", B, 3)
    dim, total = u.shape
    nheads, (ngroups, dstate) = delta.shape[0], B.shape[:2]
    io, dev, n, f32 = io_code(u), u.device, _n_seq(cu_seqlens), torch.float32
    need("delta", delta, u.dtype, (nheads, total), dev)
    need("A", A, f32, (dim, dstate) if nheads == dim else (nheads,), dev)
    need("B", B, u.dtype, (ngroups, dstate, total), dev)
    need("C", C, u.dtype, (ngroups, dstate, total), dev)
    need("D", D, f32, (dim,), dev)
    need("z", z, u.dtype, (dim, total), dev)
    need("delta_bias", delta_bias, f32, (nheads,), dev)
    need("out", out, u.dtype, (dim, total), dev)
    need_pool("states", states, f32, (dim, dstate), dev)
    _indices(n, dev, cu_seqlens, slots, has_state)
    if workspace is not None and (workspace.device != dev or not workspace.is_contiguous()):
        raise ValueError(f"workspace must be a contiguous tensor on {dev}")
    dims = _abi.make_dims(n, dim, total, dstate, nheads, ngroups, io)
    longest = max(int(max_seqlen or 0), 0)

    def call(out, workspace, raw):
        nbytes = _abi.ssm_selective_scan_packed_workspace_size(dims, longest)
        if workspace is None and nbytes:
            workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev)
        if out is None:
            out = torch.zeros_like(u)
        have = workspace.numel() * workspace.element_size() if workspace is not None else 0
        _abi.ssm_selective_scan_packed_fwd(dims, u, delta, A, B, C, D, z, delta_bias, softplus, cu_seqlens, slots,
                                           has_state, states, states.shape[0], max(states.stride(0), dim * dstate),
                                           longest, out, workspace, have, raw)
        return out
    return launch(call, dev, stream, out, workspace)


def selective_state_update_slots(states, u, delta, A, B, C, slots=None, D=None, z=None, delta_bias=None,
                                 softplus: bool = True, out=None, stream=None):
    """One step of the recurrence for rows whose states sit in slots: u (batch, dim), delta (batch, nheads),
    B and C (batch, ngroups, dstate) -> out, each row's slot of states (n_slots, dim, dstate; fp32) updated
    in place."""
    import torch
    need_cuda("u", u, 2)
    need_cuda("delta", delta, 2)
    need_cuda("B", B, 3)
    batch, dim = u.shape
    nheads, (ngroups, dstate) = delta.shape[1], B.shape[1:]
    io, dev, f32 = io_code(u), u.device, torch.float32
    need("delta", delta, u.dtype, (batch, nheads), dev)
    need("A", A, f32, (dim, dstate) if nheads == dim else (nheads,), dev)
    need("B", B, u.dtype, (batch, ngroups, dstate), dev)
    need("C", C, u.dtype, (batch, ngroups, dstate), dev)
    need("D", D, f32, (dim,), dev)
    need("z", z, u.dtype, (batch, dim), dev)
    need("delta_bias", delta_bias, f32, (nheads,), dev)
    need("out", out, u.dtype, (batch, dim), dev)
    need("slots", slots, torch.int32, (batch,), dev)
    need_pool("states", states, f32, (dim, dstate), dev)
    dims = _abi.make_dims(batch, dim, 1, dstate, nheads, ngroups, io)

    def call(out, raw):
        if out is None:
            out = torch.zeros_like(u)
        _abi.ssm_selective_state_update_slots(dims, states, slots, states.shape[0], max(states.stride(0), dim * dstate),
                                              u, delta, A, B, C, D, z, delta_bias, softplus, out, raw)
        return out
    return launch(call, dev, stream, out)


def state_slots_copy(pool, src, dst, slot_dim: int = 0, stream=None):
    """Slot dst[i] of the pool becomes what slot src[i] held before the call, or zeros for src[i] = -1, for
    all i at once: forks, moves and clears, in every layer.  slot_dim is the pool's dimension that counts
    slots; the dimension before it, if any (slot_dim = 1), counts layers.  Returns the pool."""
    import torch
    if not pool.is_cuda:
        raise ValueError("pool must be a CUDA tensor")
    if slot_dim not in (0, 1) or pool.dim() <= slot_dim:
        raise ValueError("slot_dim must be 0, or 1 behind a dimension of layers")
    if not inner_contiguous(pool, slot_dim + 1):
        raise ValueError("every slot of pool must be contiguous")
    n = src.numel()
    need("src", src, torch.int32, (n,), pool.device)
    need("dst", dst, torch.int32, (n,), pool.device)
    e, n_slots = pool.element_size(), pool.shape[slot_dim]
    slot_bytes = e
    for s in pool.shape[slot_dim + 1:]:
        slot_bytes *= s
    layers, layer_stride = (pool.shape[0], pool.stride(0) * e) if slot_dim else (1, 0)
    # a single slot's stride says nothing
    slot_stride = pool.stride(slot_dim) * e if n_slots > 1 else slot_bytes

    def call(raw):
        _abi.ssm_state_slots_copy(pool, layers, n_slots, slot_bytes, slot_stride, layer_stride, src, dst, n, raw)
        return pool
    return launch(call, pool.device, stream)
