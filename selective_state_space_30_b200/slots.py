"""Torch front ends of the operators that keep each sequence's state in a slot of a pool.

Layouts, slots and lengths are those of include/ssm_scan.h ("packed prompts and state slots"):
`cu_seqlens` and `slots` are int32 and `has_state` uint8 or bool CUDA tensors, read on the device;
a negative slot marks a padding row.  Pools are (n_slots, ...) tensors whose slots are contiguous
and may lie apart (a layer's view of a pool that holds several layers).  The calls update the
pools in place, run on `stream` (default: the device's current one) and can be captured into a
CUDA graph.  `out` is allocated with torch unless given, zeroed where a call may leave some of it as
it was, so that padding reads as zero; a workspace is allocated unless given.  An `out` that is given
shares no memory with what the call reads (the single-token calls may write over x, u or z: out being
that very tensor).  Tensors of another type, shape, device or layout are refused with ValueError, what
the library refuses with SsmError.  The checks and calls are compiled (csrc/front.cpp).
"""
from __future__ import annotations

from ._frontend import load, on_stream


def causal_conv1d_packed(x, w, cu_seqlens, conv_states, slots=None, has_state=None, bias=None, silu: bool = True,
                         out=None, stream=None):
    """The causal convolution over prompts packed along time: x (dim, total) -> out.  Each sequence's
    earlier inputs come from its slot of conv_states (n_slots, dim, width - 1; x's dtype, the oldest
    first) where has_state is nonzero, and its last width - 1 inputs replace them."""
    f = load().conv_packed
    if stream is None:
        return f(x, w, cu_seqlens, conv_states, slots, has_state, bias, silu, out)
    return on_stream(f, stream, x, x, w, cu_seqlens, conv_states, slots, has_state, bias, silu, out)


def causal_conv1d_update(x, w, conv_states, slots=None, bias=None, silu: bool = True, out=None, stream=None):
    """The causal convolution of one new token per row: x (batch, dim) -> out, each row's slot of
    conv_states moved on by its token."""
    f = load().conv_update
    if stream is None:
        return f(x, w, conv_states, slots, bias, silu, out)
    return on_stream(f, stream, x, x, w, conv_states, slots, bias, silu, out)


def selective_scan_packed(u, delta, A, B, C, cu_seqlens, states, slots=None, has_state=None, D=None, z=None,
                          delta_bias=None, softplus: bool = True, max_seqlen: int = 0, out=None, workspace=None,
                          stream=None):
    """The forward scan over prompts packed along time: u (dim, total), delta (nheads, total), B and C
    (ngroups, dstate, total) -> out.  Each sequence starts from its slot of states (n_slots, dim, dstate;
    fp32) where has_state is nonzero, else from zero, and leaves its final state there.  max_seqlen, if
    known, only saves the cutting of sequences that are all short.  The workspace (uint8, at least
    ssm_selective_scan_packed_workspace_size bytes) must not serve two calls, or two graphs, at once.
    ssm_selective_scan_packed_device_status tells whether a kernel gave up on a wait."""
    f = load().scan_packed
    if stream is None:
        return f(u, delta, A, B, C, cu_seqlens, states, slots, has_state, D, z, delta_bias, softplus, max_seqlen, out,
                 workspace)
    return on_stream(f, stream, u, u, delta, A, B, C, cu_seqlens, states, slots, has_state, D, z, delta_bias, softplus,
                     max_seqlen, out, workspace)


def selective_state_update_slots(states, u, delta, A, B, C, slots=None, D=None, z=None, delta_bias=None,
                                 softplus: bool = True, out=None, stream=None):
    """One step of the recurrence for rows whose states sit in slots: u (batch, dim), delta (batch, nheads),
    B and C (batch, ngroups, dstate) -> out, each row's slot of states (n_slots, dim, dstate; fp32) updated
    in place."""
    f = load().state_update
    if stream is None:
        return f(states, u, delta, A, B, C, slots, D, z, delta_bias, softplus, out)
    return on_stream(f, stream, u, states, u, delta, A, B, C, slots, D, z, delta_bias, softplus, out)


def state_slots_copy(pool, src, dst, slot_dim: int = 0, stream=None):
    """Slot dst[i] of the pool becomes what slot src[i] held before the call, or zeros for src[i] = -1, for
    all i at once: forks, moves and clears, in every layer.  slot_dim is the pool's dimension that counts
    slots; the dimension before it, if any (slot_dim = 1), counts layers.  Returns the pool."""
    f = load().slots_copy
    if stream is None:
        return f(pool, src, dst, slot_dim)
    return on_stream(f, stream, pool, pool, src, dst, slot_dim)
