"""Torch front ends of the causal convolution in front of the scan and of its gradients
(ssm_causal_conv1d_fwd and ssm_causal_conv1d_bwd of include/ssm_scan.h)."""
from __future__ import annotations

from ._frontend import load, on_stream


def causal_conv1d_fwd(x, w, bias=None, silu: bool = True, out=None, stream=None):
    """out[b,d,t] = act(bias[d] + sum_k w[d,k] x[b,d,t-width+1+k]) on CUDA tensors: x (batch, dim, seqlen)
    bf16 or fp32, w (dim, width) and bias fp32.  out must not overlap an input: each output needs the inputs
    before its own."""
    f = load().conv_fwd
    return f(x, w, bias, silu, out) if stream is None else on_stream(f, stream, x, x, w, bias, silu, out)


def causal_conv1d_bwd(x, w, dout, bias=None, silu: bool = True, workspace=None, stream=None) -> dict:
    """Gradients of causal_conv1d_fwd: {"dx": x's dtype, "dw": fp32, "dbias": fp32} (dbias is the gradient
    at zero where bias is None).  The workspace (uint8, at least ssm_causal_conv1d_bwd_workspace_size bytes)
    is allocated with torch unless given."""
    f = load().conv_bwd
    args = (x, w, dout, bias, silu, workspace)
    dx, dw, dbias = f(*args) if stream is None else on_stream(f, stream, x, *args)
    return {"dx": dx, "dw": dw, "dbias": dbias}


_fn_cls = None


def _causal_conv1d_function():
    """The torch.autograd.Function (built on first use, so that importing the package does not import torch)."""
    global _fn_cls
    if _fn_cls is not None:
        return _fn_cls
    import torch
    from torch.autograd.function import once_differentiable

    class CausalConv1dFn(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, w, bias, silu):
            ctx.save_for_backward(x, w, bias)
            ctx.silu = silu
            return causal_conv1d_fwd(x, w, bias, silu)

        @staticmethod
        @once_differentiable
        def backward(ctx, dout):
            x, w, bias = ctx.saved_tensors
            g = causal_conv1d_bwd(x, w, dout.contiguous(), bias, ctx.silu)
            return g["dx"], g["dw"], g["dbias"] if bias is not None else None, None

    _fn_cls = CausalConv1dFn
    return _fn_cls


def causal_conv1d_fn(x, w, bias=None, silu: bool = True):
    """The convolution as a differentiable torch operation; its backward runs ssm_causal_conv1d_bwd.

    In a CUDA graph, capture the forward and its backward together, once the results of eager calls on the
    same leaves are gone: torch ties a leaf's accumulation to the stream that first used it."""
    return _causal_conv1d_function().apply(x, w, bias, silu)
