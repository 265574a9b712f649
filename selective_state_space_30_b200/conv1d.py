"""Torch front ends of the causal convolution in front of the scan and of its gradients
(ssm_causal_conv1d_fwd and ssm_causal_conv1d_bwd of include/ssm_scan.h)."""
from __future__ import annotations

from . import _abi
from ._tensors import io_code, launch, need, need_cuda, ptr


def _checked(x, w, bias):
    import torch
    dev = need_cuda("x", x, 3)
    if w.dim() != 2:
        raise ValueError("w must have shape (dim, width)")
    need("w", w, torch.float32, (x.shape[1], w.shape[1]), dev)
    need("bias", bias, torch.float32, (x.shape[1],), dev)
    return (*x.shape, w.shape[1], io_code(x))


def causal_conv1d_fwd(x, w, bias=None, silu: bool = True, out=None, stream=None):
    """out[b,d,t] = act(bias[d] + sum_k w[d,k] x[b,d,t-width+1+k]) on CUDA tensors: x (batch, dim, seqlen)
    bf16 or fp32, w (dim, width) and bias fp32."""
    import torch
    batch, dim, seqlen, width, io = _checked(x, w, bias)
    need("out", out, x.dtype, x.shape, x.get_device())

    def call(raw):
        o = torch.empty_like(x) if out is None else out
        _abi.ssm_causal_conv1d_fwd(batch, dim, seqlen, width, io, x, w, bias, silu, o, raw)
        return o
    return launch(call, x.get_device(), stream)


def causal_conv1d_bwd(x, w, dout, bias=None, silu: bool = True, workspace=None, stream=None) -> dict:
    """Gradients of causal_conv1d_fwd: {"dx": x's dtype, "dw": fp32, "dbias": fp32} (dbias is the gradient
    at zero where bias is None).  The workspace (uint8, at least ssm_causal_conv1d_bwd_workspace_size bytes)
    is allocated with torch unless given."""
    import torch
    batch, dim, seqlen, width, io = _checked(x, w, bias)
    dev = x.get_device()
    need("dout", dout, x.dtype, x.shape, dev)
    if workspace is not None and (workspace.get_device() != dev or not workspace.is_contiguous()):
        raise ValueError(f"workspace must be a contiguous tensor on cuda:{dev}")

    def call(raw):
        ws = workspace
        if ws is None:
            nbytes = _abi.ssm_causal_conv1d_bwd_workspace_size(batch, dim, seqlen, width, io)
            ws = torch.empty(nbytes, dtype=torch.uint8, device=x.device)
        dx, dw, dbias = torch.empty_like(x), torch.empty_like(w), w.new_empty(dim)
        lib = _abi._lib or _abi.load_library()
        _abi._check(lib.ssm_causal_conv1d_bwd(
            batch, dim, seqlen, width, io, x.data_ptr(), w.data_ptr(), ptr(bias), 1 if silu else 0, dout.data_ptr(),
            dx.data_ptr(), dw.data_ptr(), dbias.data_ptr(), ws.data_ptr(), ws.numel() * ws.element_size(), raw),
            "ssm_causal_conv1d_bwd")
        return {"dx": dx, "dw": dw, "dbias": dbias}
    return launch(call, dev, stream)


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
