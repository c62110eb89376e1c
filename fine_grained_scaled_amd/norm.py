"""The boundary between two transformer blocks (the kernels behind
fgs_residual_norm_fwd / fgs_residual_norm_bwd): norm of the block's output,
gate, scaled residual and the norm for the next block in one pass, its
gradients, and its autograd form."""
from __future__ import annotations

from typing import NamedTuple, Optional

import torch

from . import _lib
from .ops import _need_gpu, _stream_of

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


def _matrix(t: torch.Tensor, name: str, shape, dtype) -> None:
    if t.dtype != dtype or t.shape != shape:
        raise TypeError(f"{name} must be a [{shape[0]} x {shape[1]}] {dtype} tensor (got {tuple(t.shape)} {t.dtype})")
    if t.stride(1) != 1:
        raise ValueError(f"{name} must have unit stride along columns")


def _weight(t: Optional[torch.Tensor], name: str, width: int) -> None:
    if t is not None and (t.dtype != torch.float32 or t.dim() != 1 or t.numel() != width or not t.is_contiguous()):
        raise TypeError(f"{name} must be a contiguous float32 tensor of {width} values")


def _check(y, x, w_post, gate, w_pre):
    """Shapes and types of the inputs; returns the gate's kind and row stride."""
    if y.dim() != 2:
        raise TypeError("y must be a [tokens x width] bfloat16 tensor")
    shape = y.shape
    if x.dtype not in _RESIDUAL:
        raise TypeError("the residual must be float32 or bfloat16")
    _matrix(y, "y", shape, torch.bfloat16)
    _matrix(x, "the residual", shape, x.dtype)
    _weight(w_pre, "w_pre", shape[1])
    _weight(w_post, "w_post", shape[1])
    _need_gpu(y)
    gpu = y.get_device()
    for t in (x, w_pre, w_post, gate):
        if t is not None and t.get_device() != gpu:
            raise ValueError("all tensors must be on one GPU")
    if gate is None:
        return _lib.GATE_NONE, 0
    if gate.dim() == 1:
        _weight(gate, "gate", shape[1])
        return _lib.GATE_CHANNEL, 0
    _matrix(gate, "gate", shape, torch.bfloat16)
    return _lib.GATE_TOKEN, gate.stride(0)


def residual_norm_fwd(y: torch.Tensor, x: torch.Tensor, *, w_pre: torch.Tensor, w_post: Optional[torch.Tensor] = None,
                      gate: Optional[torch.Tensor] = None, alpha: float = 1.0, eps: float = 1e-6):
    """r = alpha x + gate * (y / rms(y) * w_post), n = r / rms(r) * w_pre:
    returns (r, n).  y [tokens x width] bfloat16 is the block's output, x the
    residual (float32 or bfloat16, r in its type, rounded before it is
    normed), n bfloat16.  w_post None: y is not normed.  gate: None, float32
    [width] or bfloat16 [tokens x width].  Weights are float32 [width]."""
    kind, ldg = _check(y, x, w_post, gate, w_pre)
    T, W = y.shape
    r = torch.empty((T, W), dtype=x.dtype, device=y.device)
    n = torch.empty((T, W), dtype=torch.bfloat16, device=y.device)
    _lib.check(_lib.load().fgs_residual_norm_fwd(
        _at(y), y.stride(0), _at(x), x.stride(0), _RESIDUAL[x.dtype], T, W, _at(w_post), _at(gate), ldg, kind,
        alpha, _at(w_pre), eps, _at(r), _at(n), _stream_of(y)))
    return r, n


def residual_norm_bwd(dr: torch.Tensor, dn: torch.Tensor, y: torch.Tensor, r: torch.Tensor, *, w_pre: torch.Tensor,
                      w_post: Optional[torch.Tensor] = None, gate: Optional[torch.Tensor] = None, alpha: float = 1.0,
                      eps: float = 1e-6, workspace: Optional[torch.Tensor] = None) -> ResidualNormGrads:
    """Gradients of residual_norm_fwd from its y, the r it returned, and the
    gradients dr (r's type) and dn (bfloat16) of its two outputs.  Weight and
    channel-gate gradients are float32, the others have their input's type.
    workspace: optional uint8 device scratch of
    fgs_residual_norm_workspace_bytes() bytes."""
    kind, ldg = _check(y, r, w_post, gate, w_pre)
    T, W = y.shape
    _matrix(dr, "dr", y.shape, r.dtype)
    _matrix(dn, "dn", y.shape, torch.bfloat16)
    if dr.get_device() != y.get_device() or dn.get_device() != y.get_device():
        raise ValueError("all tensors must be on one GPU")
    dev = y.device
    dx = torch.empty((T, W), dtype=r.dtype, device=dev)
    dy = torch.empty((T, W), dtype=torch.bfloat16, device=dev)
    dgate = torch.empty_like(gate, memory_format=torch.contiguous_format) if gate is not None else None
    dw_post = torch.empty_like(w_post) if w_post is not None else None
    dw_pre = torch.empty_like(w_pre)
    lib = _lib.load()
    if workspace is None:
        workspace = torch.empty(lib.fgs_residual_norm_workspace_bytes(T, W), dtype=torch.uint8, device=dev)
    elif workspace.device != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the same GPU")
    _lib.check(lib.fgs_residual_norm_bwd(
        _at(dr), dr.stride(0), _at(dn), dn.stride(0), _at(y), y.stride(0), _at(r), r.stride(0), _RESIDUAL[r.dtype],
        T, W, _at(w_post), _at(gate), ldg, kind, alpha, _at(w_pre), eps, _at(dx), _at(dy), _at(dgate),
        _at(dw_post), _at(dw_pre), _at(workspace), workspace.numel() * workspace.element_size(), _stream_of(y)))
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
        g = residual_norm_bwd(dr.contiguous(), dn.contiguous(), y, r, w_pre=w_pre, w_post=w_post, gate=gate,
                              alpha=ctx.alpha, eps=ctx.eps)
        return g.y, g.residual, g.w_pre, g.w_post, g.gate, None, None


def residual_norm(y: torch.Tensor, x: torch.Tensor, *, w_pre: torch.Tensor, w_post: Optional[torch.Tensor] = None,
                  gate: Optional[torch.Tensor] = None, alpha: float = 1.0, eps: float = 1e-6):
    """residual_norm_fwd with autograd: returns (r, n), gradients for y, x,
    the weights and the gate."""
    return _ResidualNorm.apply(y, x, w_pre, w_post, gate, alpha, eps)
