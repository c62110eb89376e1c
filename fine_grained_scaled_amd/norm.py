"""The boundary between two transformer blocks (the kernels behind
fgs_residual_norm_fwd / fgs_residual_norm_bwd): norm of the block's output,
gate, scaled residual and the norm for the next block in one pass, its
gradients, and its autograd form."""
from __future__ import annotations

from typing import NamedTuple, Optional

import torch

from . import _lib
from .ops import _need_gpu, _readable, _stream_of

_RESIDUAL = {torch.float32: _lib.OUT_FP32, torch.bfloat16: _lib.OUT_BF16}


class ResidualNormGrads(NamedTuple):
    """Gradients of residual_norm_fwd: for the residual x, the block's output
    y, the gate and the two weights (None where there is none)."""
    residual: torch.Tensor
    y: torch.Tensor
    gate: Optional[torch.Tensor]
    w_post: Optional[torch.Tensor]
    w_pre: torch.Tensor


def _at(t: Optional[torch.Tensor]) -> int:
    return 0 if t is None else t.data_ptr()


def _matrix(t: torch.Tensor, name: str, shape, dtype, gpu: int) -> int:
    """t's row stride."""
    if t.dtype != dtype or t.shape != shape:
        raise TypeError(f"{name} must be a [{shape[0]} x {shape[1]}] {dtype} tensor (got {tuple(t.shape)} {t.dtype})")
    row, value = t.stride()
    if value != 1:
        raise ValueError(f"{name} must have unit stride along columns")
    if t.get_device() != gpu:
        raise ValueError("all tensors must be on one GPU")
    return row


def _weight(t: torch.Tensor, name: str, width: int, gpu: int) -> None:
    if t.dtype != torch.float32 or t.dim() != 1 or t.numel() != width or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous float32 tensor of {width} values")
    if t.get_device() != gpu:
        raise ValueError("all tensors must be on one GPU")


def _check(y, x, w_post, gate, w_pre):
    """Shapes, types and places of the inputs; returns the shape, the GPU, the
    residual's type, the gate's kind and the row strides of y, x and gate."""
    if y.dim() != 2:
        raise TypeError("y must be a [tokens x width] bfloat16 tensor")
    shape, kind, gpu = y.shape, x.dtype, y.get_device()
    if kind not in _RESIDUAL:
        raise TypeError("the residual must be float32 or bfloat16")
    ldy = _matrix(y, "y", shape, torch.bfloat16, gpu)
    width = shape[1]
    for t, name in ((w_pre, "w_pre"), (w_post, "w_post")):
        if t is not None:
            _weight(t, name, width, gpu)
    if not y.is_cuda:
        _need_gpu(y)
    ldx = _matrix(x, "the residual", shape, kind, gpu)
    if gate is None:
        return shape, gpu, _RESIDUAL[kind], _lib.GATE_NONE, ldy, ldx, 0
    if gate.dim() == 1:
        _weight(gate, "gate", width, gpu)
        return shape, gpu, _RESIDUAL[kind], _lib.GATE_CHANNEL, ldy, ldx, 0
    return shape, gpu, _RESIDUAL[kind], _lib.GATE_TOKEN, ldy, ldx, _matrix(gate, "gate", shape, torch.bfloat16, gpu)


def residual_norm_fwd(y: torch.Tensor, x: torch.Tensor, *, w_pre: torch.Tensor, w_post: Optional[torch.Tensor] = None,
                      gate: Optional[torch.Tensor] = None, alpha: float = 1.0, eps: float = 1e-6):
    """r = alpha x + gate * (y / rms(y) * w_post), n = r / rms(r) * w_pre:
    returns (r, n).  y [tokens x width] bfloat16 is the block's output, x the
    residual (float32 or bfloat16, r in its type, rounded before it is
    normed), n bfloat16.  w_post None: y is not normed.  gate: None, float32
    [width] or bfloat16 [tokens x width].  Weights are float32 [width]."""
    (T, W), gpu, residual, kind, ldy, ldx, ldg = _check(y, x, w_post, gate, w_pre)
    r, n = x.new_empty(T, W), y.new_empty(T, W)      # a call of few rows is bound by this: torch.empty takes twice as long
    _lib.check(_lib.load().fgs_residual_norm_fwd(
        y.data_ptr(), ldy, x.data_ptr(), ldx, residual, T, W, _at(w_post), _at(gate), ldg, kind,
        alpha, w_pre.data_ptr(), eps, r.data_ptr(), n.data_ptr(), _stream_of(y)))
    return r, n


def residual_norm_bwd(dr: torch.Tensor, dn: torch.Tensor, y: torch.Tensor, r: torch.Tensor, *, w_pre: torch.Tensor,
                      w_post: Optional[torch.Tensor] = None, gate: Optional[torch.Tensor] = None, alpha: float = 1.0,
                      eps: float = 1e-6, workspace: Optional[torch.Tensor] = None) -> ResidualNormGrads:
    """Gradients of residual_norm_fwd from its y, the r it returned, and the
    gradients dr (r's type) and dn (bfloat16) of its two outputs.  Weight and
    channel-gate gradients are float32, the others have their input's type.
    workspace: optional uint8 device scratch of
    fgs_residual_norm_workspace_bytes() bytes."""
    shape, gpu, residual, kind, ldy, ldr, ldg = _check(y, r, w_post, gate, w_pre)
    T, W = shape
    lddr = _matrix(dr, "dr", shape, r.dtype, gpu)
    lddn = _matrix(dn, "dn", shape, torch.bfloat16, gpu)
    dx, dy = r.new_empty(T, W), y.new_empty(T, W)
    dgate = gate.new_empty(gate.shape) if gate is not None else None
    dw_post = w_post.new_empty(W) if w_post is not None else None
    dw_pre = w_pre.new_empty(W)
    lib = _lib.load()
    if workspace is None:
        workspace = w_pre.new_empty(-(-lib.fgs_residual_norm_workspace_bytes(T, W) // 4))
    elif workspace.get_device() != gpu or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the same GPU")
    _lib.check(lib.fgs_residual_norm_bwd(
        dr.data_ptr(), lddr, dn.data_ptr(), lddn, y.data_ptr(), ldy, r.data_ptr(), ldr, residual,
        T, W, _at(w_post), _at(gate), ldg, kind, alpha, w_pre.data_ptr(), eps, dx.data_ptr(), dy.data_ptr(), _at(dgate),
        _at(dw_post), dw_pre.data_ptr(), workspace.data_ptr(), workspace.numel() * workspace.element_size(),
        _stream_of(y)))
    return ResidualNormGrads(dx, dy, dgate, dw_post, dw_pre)


class _ResidualNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, y, x, w_pre, w_post, gate, alpha, eps):
        r, n = residual_norm_fwd(y, x, w_pre=w_pre, w_post=w_post, gate=gate, alpha=alpha, eps=eps)
        ctx.save_for_backward(y, r, w_pre, w_post, gate)
        ctx.alpha, ctx.eps = alpha, eps
        return r, n

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dr, dn):
        y, r, w_pre, w_post, gate = ctx.saved_tensors
        dr, dn = _readable(dr, y.shape[1]), _readable(dn, y.shape[1])
        g = residual_norm_bwd(dr, dn, y, r, w_pre=w_pre, w_post=w_post, gate=gate, alpha=ctx.alpha, eps=ctx.eps)
        return g.y, g.residual, g.w_pre, g.w_post, g.gate, None, None


def residual_norm(y: torch.Tensor, x: torch.Tensor, *, w_pre: torch.Tensor, w_post: Optional[torch.Tensor] = None,
                  gate: Optional[torch.Tensor] = None, alpha: float = 1.0, eps: float = 1e-6):
    """residual_norm_fwd with autograd: returns (r, n), gradients for y, x,
    the weights and the gate."""
    return _ResidualNorm.apply(y, x, w_pre, w_post, gate, alpha, eps)
