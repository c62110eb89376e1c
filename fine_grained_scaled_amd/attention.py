"""Causal attention over packed sequences with grouped heads, forward and
backward (the kernels behind fgs_attention_fwd / fgs_attention_bwd), and its
autograd form.

A pack holds sequences of different lengths one after the other:
cu_seqlens (int32 [S + 1] on the GPU) says where each begins and ends, and is
read on the device, so no call waits for the GPU.  attention_fwd and
attention_bwd keep no state and can be captured into a graph.  So can
attention() and its backward pass, as any of torch's operations, once no eager
graph of the same leaves is alive (its loss deleted): a leaf's AccumulateGrad
node keeps the stream on which it was made for as long as a graph holds it, a
captured backward pass would have to wait for that stream, which capture does
not allow, and torch's backward thread ends the process with the error.
"""
from __future__ import annotations

import array
from typing import Optional

import torch

from . import _lib
from .ops import _readable, _stream_of

_LIMIT = "must be a [tokens x heads x head_dim] bfloat16 tensor"
_HEADS = 24      # bytes of an fgs_heads: pointer and two strides


def _heads(t: torch.Tensor, name: str):
    """The fgs_heads of t: pointer, token stride, head stride."""
    if t.dtype != torch.bfloat16 or t.dim() != 3:
        raise TypeError(f"{name} {_LIMIT}")
    if not t.is_cuda:
        raise ValueError("fine_grained_scaled_amd operates on GPU tensors only")
    token, head, value = t.stride()
    if value != 1 and t.shape[2] > 1:
        raise ValueError(f"{name} must have unit stride along head_dim")
    return t.data_ptr(), token, head


def _check(q, k, v, cu_seqlens, softmax_scale):
    T, H, D = q.shape
    Tk, Hk, Dk = shape = k.shape
    if shape != v.shape or Tk != T or Dk != D:
        raise ValueError(f"k and v must be [{T} x kv_heads x {D}] (got {tuple(k.shape)} and {tuple(v.shape)})")
    if Hk == 0 or H % Hk:
        raise ValueError(f"heads ({H}) must be a multiple of kv_heads ({Hk})")
    if cu_seqlens.dtype != torch.int32 or cu_seqlens.dim() != 1 or not cu_seqlens.is_contiguous() \
            or cu_seqlens.numel() < 1:
        raise TypeError("cu_seqlens must be a contiguous 1-D int32 tensor of one entry at least")
    gpu = q.get_device()
    if k.get_device() != gpu or v.get_device() != gpu or cu_seqlens.get_device() != gpu:
        raise ValueError("q, k, v and cu_seqlens must be on one GPU")
    return T, H, Hk, D, (max(D, 1) ** -0.5 if softmax_scale is None else float(softmax_scale))


def attention_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_seqlens: torch.Tensor,
                  softmax_scale: Optional[float] = None):
    """Causal attention of every sequence of the pack: returns (out [T x H x D]
    bfloat16, lse [H x T] float32, the natural logarithm of the row sums).
    q is [T x H x D], k and v [T x Hk x D] (H a multiple of Hk, D 64 or 128),
    views of a fused projection among them.  softmax_scale: 1 / sqrt(D)
    unless given (2^-100 to 2^100).
    Tokens of no sequence get out = 0 and lse = -inf."""
    views = _heads(q, "q") + _heads(k, "k") + _heads(v, "v")
    T, H, Hk, D, scale = _check(q, k, v, cu_seqlens, softmax_scale)
    out = q.new_empty(T, H, D)               # half of what torch.empty takes
    lse = q.new_empty(H, T, dtype=torch.float32)
    views = array.array("q", views + (out.data_ptr(), H * D, D))
    at = views.buffer_info()[0]
    _lib.check(_lib.load().fgs_attention_fwd(
        at, at + _HEADS, at + 2 * _HEADS, cu_seqlens.data_ptr(), cu_seqlens.numel() - 1, T, H, Hk, D, scale,
        at + 3 * _HEADS, lse.data_ptr(), _stream_of(q)))
    return out, lse


def attention_bwd(dout: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, out: torch.Tensor,
                  lse: torch.Tensor, cu_seqlens: torch.Tensor, softmax_scale: Optional[float] = None,
                  workspace: Optional[torch.Tensor] = None):
    """dq, dk, dv of attention_fwd from its inputs, its out and lse, and dout
    [T x H x D].  workspace: optional uint8 device scratch of
    fgs_attention_workspace_bytes() bytes.  The same inputs give the same
    bits; tokens of no sequence get zeros."""
    views = _heads(q, "q") + _heads(k, "k") + _heads(v, "v") + _heads(out, "out") + _heads(dout, "dout")
    T, H, Hk, D, scale = _check(q, k, v, cu_seqlens, softmax_scale)
    if out.shape != q.shape or dout.shape != q.shape:
        raise ValueError(f"out and dout must be {tuple(q.shape)} (got {tuple(out.shape)} and {tuple(dout.shape)})")
    if lse.dtype != torch.float32 or tuple(lse.shape) != (H, T) or not lse.is_contiguous():
        raise TypeError(f"lse must be a contiguous [{H} x {T}] float32 tensor")
    gpu = q.get_device()
    if out.get_device() != gpu or dout.get_device() != gpu or lse.get_device() != gpu:
        raise ValueError("all tensors must be on one GPU")
    dq, dk, dv = q.new_empty(T, H, D), q.new_empty(T, Hk, D), q.new_empty(T, Hk, D)
    lib = _lib.load()
    need = lib.fgs_attention_workspace_bytes(T, H)
    if workspace is None:
        workspace = lse.new_empty(-(-need // 4))
    elif workspace.get_device() != gpu or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the same GPU")
    views = array.array("q", views + (dq.data_ptr(), H * D, D, dk.data_ptr(), Hk * D, D, dv.data_ptr(), Hk * D, D))
    at = [views.buffer_info()[0] + i * _HEADS for i in range(8)]
    _lib.check(lib.fgs_attention_bwd(
        at[4], *at[:4], lse.data_ptr(), cu_seqlens.data_ptr(), cu_seqlens.numel() - 1, T, H, Hk, D, scale, *at[5:],
        workspace.data_ptr(), workspace.numel() * workspace.element_size(), _stream_of(q)))
    return dq, dk, dv


class _Attention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, cu_seqlens, softmax_scale):
        out, lse = attention_fwd(q, k, v, cu_seqlens, softmax_scale)
        ctx.save_for_backward(q, k, v, out, lse, cu_seqlens)
        ctx.scale = softmax_scale
        return out

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dout):
        q, k, v, out, lse, cu = ctx.saved_tensors
        dq, dk, dv = attention_bwd(_readable(dout.to(torch.bfloat16), 0), q, k, v, out, lse, cu, ctx.scale)
        return dq, dk, dv, None, None


def attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_seqlens: torch.Tensor,
              softmax_scale: Optional[float] = None) -> torch.Tensor:
    """attention_fwd's out with autograd: gradients for q, k and v."""
    return _Attention.apply(q, k, v, cu_seqlens, softmax_scale)
