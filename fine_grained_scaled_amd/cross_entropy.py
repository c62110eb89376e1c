"""The output head with softmax cross entropy, without keeping the logits (the
kernels behind fgs_linear_cross_entropy_fwd / fgs_linear_cross_entropy_bwd), and
its autograd form."""
from __future__ import annotations

from typing import Optional

import torch

from . import _lib
from .ops import _need_gpu, _readable, _stream_of

_INDEX = {torch.int32: _lib.INDEX_I32, torch.int64: _lib.INDEX_I64}


def _check(x, w, targets):
    """Shapes, types and places; returns T, V, K, the GPU and the targets' type."""
    for t, name in ((x, "x"), (w, "w")):
        if t.dtype != torch.bfloat16 or t.dim() != 2:
            raise TypeError(f"{name} must be a 2-D bfloat16 tensor")
        if t.stride(1) != 1:
            raise ValueError(f"{name} must have unit stride along columns")
    (T, K), V = x.shape, w.shape[0]
    if w.shape[1] != K:
        raise ValueError(f"w must be [vocab x {K}] (got {tuple(w.shape)})")
    if targets.dtype not in _INDEX or targets.dim() != 1 or targets.numel() != T or not targets.is_contiguous():
        raise TypeError(f"targets must be a contiguous int32 or int64 tensor of {T} values")
    _need_gpu(x)
    gpu = x.get_device()
    if w.get_device() != gpu or targets.get_device() != gpu:
        raise ValueError("all tensors must be on one GPU")
    return T, V, K, gpu, _INDEX[targets.dtype]


def _workspace(given: Optional[torch.Tensor], like: torch.Tensor, need: int):
    if given is None:
        return like.new_empty(need, dtype=torch.uint8)
    if given.get_device() != like.get_device() or not given.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the same GPU")
    return given


def _floats(t: torch.Tensor, name: str, count: int, gpu: int) -> None:
    if t.dtype != torch.float32 or t.dim() != 1 or t.numel() != count or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous float32 tensor of {count} values")
    if t.get_device() != gpu:
        raise ValueError("all tensors must be on one GPU")


def linear_cross_entropy_fwd(x: torch.Tensor, w: torch.Tensor, targets: torch.Tensor,
                             workspace: Optional[torch.Tensor] = None):
    """z = x w^T, lse = log sum exp z, loss = lse - z[target] for every token
    (row of x): returns (loss, lse), float32 [T]; z is not kept.  x [T x K]
    and w [V x K] bfloat16 (K a multiple of 64), targets int32 or int64 [T]; a
    target outside [0, V) (-100, say) takes no part: loss and lse 0.
    workspace: optional uint8 device scratch of
    fgs_linear_cross_entropy_workspace_bytes() bytes."""
    T, V, K, gpu, index = _check(x, w, targets)
    lib = _lib.load()
    loss, lse = x.new_empty(T, dtype=torch.float32), x.new_empty(T, dtype=torch.float32)
    workspace = _workspace(workspace, x, lib.fgs_linear_cross_entropy_workspace_bytes(T, V, K, 0))
    _lib.check(lib.fgs_linear_cross_entropy_fwd(
        x.data_ptr(), x.stride(0), w.data_ptr(), w.stride(0), targets.data_ptr(), index, T, V, K, loss.data_ptr(),
        lse.data_ptr(), workspace.data_ptr(), workspace.numel() * workspace.element_size(), _stream_of(x)))
    return loss, lse


def linear_cross_entropy_bwd(dloss: torch.Tensor, x: torch.Tensor, w: torch.Tensor, targets: torch.Tensor,
                             lse: torch.Tensor, dlse: Optional[torch.Tensor] = None,
                             workspace: Optional[torch.Tensor] = None):
    """dx [T x K], dw [V x K] (bfloat16) of linear_cross_entropy_fwd from its
    inputs, its lse, and the gradients dloss and dlse (None: zero) of its two
    results, float32 [T].  The logits are formed again, a piece of the
    vocabulary at a time.  The same inputs give the same bits.  workspace:
    optional uint8 device scratch of
    fgs_linear_cross_entropy_workspace_bytes() bytes."""
    T, V, K, gpu, index = _check(x, w, targets)
    for t, name in ((dloss, "dloss"), (lse, "lse"), (dlse, "dlse")):
        if t is not None:
            _floats(t, name, T, gpu)
    lib = _lib.load()
    dx, dw = x.new_empty(T, K), w.new_empty(V, K)
    workspace = _workspace(workspace, x, lib.fgs_linear_cross_entropy_workspace_bytes(T, V, K, 1))
    _lib.check(lib.fgs_linear_cross_entropy_bwd(
        dloss.data_ptr(), 0 if dlse is None else dlse.data_ptr(), x.data_ptr(), x.stride(0), w.data_ptr(), w.stride(0),
        targets.data_ptr(), index, lse.data_ptr(), T, V, K, dx.data_ptr(), dw.data_ptr(), workspace.data_ptr(),
        workspace.numel() * workspace.element_size(), _stream_of(x)))
    return dx, dw


class _LinearCrossEntropy(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, targets):
        ctx.w_dtype, ctx.x_dtype = w.dtype, x.dtype
        x, w = _readable(x.to(torch.bfloat16), x.shape[-1]), _readable(w.to(torch.bfloat16), w.shape[-1])
        targets = targets.contiguous()
        loss, lse = linear_cross_entropy_fwd(x, w, targets)
        ctx.save_for_backward(x, w, targets, lse)
        return loss, lse

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dloss, dlse):
        x, w, targets, lse = ctx.saved_tensors
        dx, dw = linear_cross_entropy_bwd(dloss.contiguous(), x, w, targets, lse, dlse.contiguous())
        return dx.to(ctx.x_dtype), dw.to(ctx.w_dtype), None


def linear_cross_entropy(x: torch.Tensor, w: torch.Tensor, targets: torch.Tensor, return_lse: bool = False):
    """linear_cross_entropy_fwd's loss for each token, float32 [T], with
    autograd: gradients for x and w.  w is BF16 or an FP32 master weight (its
    BF16 cast is multiplied; its gradient is rounded to BF16 as a BF16 weight's
    is, and cast to its type).  Both gradients are formed.  Layouts that
    the kernels do not read are copied.  return_lse: (loss, lse), both with
    gradients, for a penalty on lse."""
    loss, lse = _LinearCrossEntropy.apply(x, w, targets)
    return (loss, lse) if return_lse else loss
