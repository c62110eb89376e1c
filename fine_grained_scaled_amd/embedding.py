"""Token embedding and its gradient by sorted tokens (the kernels behind
fgs_embedding_fwd / fgs_embedding_bwd), and its autograd form."""
from __future__ import annotations

from typing import Optional

import torch

from . import _lib
from .cross_entropy import _INDEX, _workspace
from .ops import _need_gpu, _readable, _stream_of

_TYPE = {torch.float32: _lib.OUT_FP32, torch.bfloat16: _lib.OUT_BF16}


def _type(dtype, name: str) -> int:
    if dtype not in _TYPE:
        raise TypeError(f"{name} must be float32 or bfloat16 (got {dtype})")
    return _TYPE[dtype]


def _tokens(tokens: torch.Tensor) -> int:
    if tokens.dtype not in _INDEX or not tokens.is_contiguous():
        raise TypeError("tokens must be a contiguous int32 or int64 tensor")
    _need_gpu(tokens)
    return _INDEX[tokens.dtype]


def embedding_fwd(tokens: torch.Tensor, weight: torch.Tensor, scale: float = 1.0,
                  out_dtype: Optional[torch.dtype] = None) -> torch.Tensor:
    """scale * weight[tokens], [*tokens.shape x width] in out_dtype (float32
    or bfloat16; the weight's type unless given), zeros for tokens outside
    [0, vocab).  tokens: int32 or int64 of any shape, contiguous; weight [vocab x width]
    float32 or bfloat16, width a multiple of 8."""
    index = _tokens(tokens)
    kind = _type(weight.dtype, "weight")
    out_dtype = weight.dtype if out_dtype is None else out_dtype
    out_kind = _type(out_dtype, "out_dtype")
    if weight.dim() != 2 or weight.stride(1) != 1:
        raise ValueError("weight must be [vocab x width] with unit stride along columns")
    if weight.get_device() != tokens.get_device():
        raise ValueError("tokens and weight must be on one GPU")
    V, W = weight.shape
    out = weight.new_empty(*tokens.shape, W, dtype=out_dtype)
    _lib.check(_lib.load().fgs_embedding_fwd(
        tokens.data_ptr(), index, tokens.numel(), weight.data_ptr(), weight.stride(0), kind, V, W, scale,
        out.data_ptr(), out_kind, _stream_of(tokens)))
    return out


def embedding_bwd(dout: torch.Tensor, tokens: torch.Tensor, vocab: int, scale: float = 1.0,
                  dtype: torch.dtype = torch.float32, out: Optional[torch.Tensor] = None,
                  workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The gradient [vocab x width] of embedding_fwd for its weight: row v is
    scale times the sum of dout over the tokens that are v.  dout is
    [*tokens.shape x width], float32 or bfloat16.  A new tensor of `dtype`
    with zeros in the other rows; or, with `out` given (contiguous, float32
    or bfloat16), the sums are added to it, which touches the tokens' rows
    alone.  The same inputs give the same bits.  workspace: optional uint8
    device scratch of fgs_embedding_workspace_bytes() bytes."""
    index = _tokens(tokens)
    kind = _type(dout.dtype, "dout")
    if dout.dim() < 1 or dout.shape[:-1] != tokens.shape:
        raise ValueError(f"dout must be [{' x '.join(map(str, tokens.shape))} x width] (got {tuple(dout.shape)})")
    gpu = tokens.get_device()
    if dout.get_device() != gpu:
        raise ValueError("dout and tokens must be on one GPU")
    count, W = tokens.numel(), dout.shape[-1]
    rows = dout if dout.dim() == 2 else dout.reshape(count, W)
    if rows.stride(1) != 1 and W > 1:
        raise ValueError("dout must have unit stride along columns")
    dw = out
    if out is None:
        dw = dout.new_empty(vocab, W, dtype=dtype)
    elif tuple(out.shape) != (vocab, W) or not out.is_contiguous() or out.get_device() != gpu:
        raise ValueError(f"out must be a contiguous [{vocab} x {W}] tensor on the same GPU")
    lib = _lib.load()
    workspace = _workspace(workspace, dout, lib.fgs_embedding_workspace_bytes(count, W))
    _lib.check(lib.fgs_embedding_bwd(
        rows.data_ptr(), rows.stride(0), kind, tokens.data_ptr(), index, count, vocab, W, scale, dw.data_ptr(),
        _type(dw.dtype, "the gradient"), out is not None, workspace.data_ptr(),
        workspace.numel() * workspace.element_size(), _stream_of(tokens)))
    if out is not None:
        torch.autograd.graph.increment_version(out)      # written behind torch's back
    return dw


class _Embedding(torch.autograd.Function):
    @staticmethod
    def forward(ctx, tokens, weight, scale, out_dtype):
        tokens, weight = tokens.contiguous(), _readable(weight, weight.shape[-1])
        ctx.save_for_backward(tokens)
        ctx.vocab, ctx.scale, ctx.dtype = weight.shape[0], scale, weight.dtype
        return embedding_fwd(tokens, weight, scale, out_dtype)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dout):
        tokens, = ctx.saved_tensors
        W = dout.shape[-1]
        dout = _readable(dout.reshape(-1, W), W)
        return None, embedding_bwd(dout, tokens.view(-1), ctx.vocab, ctx.scale, ctx.dtype), None, None


def embedding(tokens: torch.Tensor, weight: torch.Tensor, scale: float = 1.0,
              out_dtype: Optional[torch.dtype] = None) -> torch.Tensor:
    """embedding_fwd with autograd: a gradient for the weight, in its type.
    Layouts that the kernels do not read are copied."""
    return _Embedding.apply(tokens, weight, scale, out_dtype)
