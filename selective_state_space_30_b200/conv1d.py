"""Torch front ends of the causal convolution in front of the scan and of its gradients
(ssm_causal_conv1d_fwd and ssm_causal_conv1d_bwd of include/ssm_scan.h)."""
from __future__ import annotations

from . import _abi
from ._tensors import io_code, launch, need, need_cuda


def _checked(x, w, bias):
    import torch
    need_cuda("x", x, 3)
    if w.dim() != 2:
        raise ValueError("w must have shape (dim, width)")
    need("w", w, torch.float32, (x.shape[1], w.shape[1]), x.device)
    need("bias", bias, torch.float32, (x.shape[1],), x.device)
    return (*x.shape, w.shape[1], io_code(x))


def causal_conv1d_fwd(x, w, bias=None, silu: bool = True, out=None, stream=None):
    """out[b,d,t] = act(bias[d] + sum_k w[d,k] x[b,d,t-width+1+k]) on CUDA tensors: x (batch, dim, seqlen)
    bf16 or fp32, w (dim, width) and bias fp32."""
    import torch
    batch, dim, seqlen, width, io = _checked(x, w, bias)
    need("out", out, x.dtype, x.shape, x.device)

    def call(out, raw):
        out = torch.empty_like(x) if out is None else out
        _abi.ssm_causal_conv1d_fwd(batch, dim, seqlen, width, io, x, w, bias, silu, out, raw)
        return out
    return launch(call, x.device, stream, out)


def causal_conv1d_bwd(x, w, dout, bias=None, silu: bool = True, workspace=None, stream=None) -> dict:
    """Gradients of causal_conv1d_fwd: {"dx": x's dtype, "dw": fp32, "dbias": fp32} (dbias is the gradient
    at zero where bias is None).  The workspace (uint8, at least ssm_causal_conv1d_bwd_workspace_size bytes)
    is allocated with torch unless given."""
    import torch
    batch, dim, seqlen, width, io = _checked(x, w, bias)
    need("dout", dout, x.dtype, x.shape, x.device)
    if workspace is not None and (workspace.device != x.device or not workspace.is_contiguous()):
        raise ValueError(f"workspace must be a contiguous tensor on {x.device}")

    def call(workspace, raw):
        if workspace is None:
            nbytes = _abi.ssm_causal_conv1d_bwd_workspace_size(batch, dim, seqlen, width, io)
            workspace = torch.empty(nbytes, dtype=torch.uint8, device=x.device)
        g = {"dx": torch.empty_like(x), "dw": torch.empty_like(w),
             "dbias": torch.empty((dim,), dtype=torch.float32, device=x.device)}
        _abi.ssm_causal_conv1d_bwd(batch, dim, seqlen, width, io, x, w, bias, silu, dout, g["dx"], g["dw"], g["dbias"],
                                   workspace, workspace.numel() * workspace.element_size(), raw)
        return g
    return launch(call, x.device, stream, workspace)


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
    """The convolution as a differentiable torch operation; its backward runs ssm_causal_conv1d_bwd."""
    return _causal_conv1d_function().apply(x, w, bias, silu)
