"""SwiGLU with its input kept in 8 bits for the backward pass (the kernels
behind fgs_swiglu_fwd / fgs_swiglu_bwd), and its autograd form."""
from __future__ import annotations

from typing import Union

import torch

from . import _lib
from .ops import Quantized, _bf16_matrix, _readable, _stream_of


def _halves(cols: int) -> int:
    if cols % 2:
        raise ValueError("gate_up must have an even number of columns")
    return cols // 2


class _Halves(Quantized):
    """Codes of [g | u] whose halves end inside a tile: the scales belong to
    the halves' tiles and not to those of whole rows, which a GEMM reads."""

    def rowwise(self):
        raise ValueError("SwiGLU's codes are a GEMM operand only where its halves are whole tiles of 128 columns")


def swiglu_fwd(gate_up: torch.Tensor, checkpoint: bool = True):
    """h = g sigmoid(g) u of gate_up = [g | u], bfloat16 [T x 2I] (I a
    multiple of 8): returns (h [T x I], kept), kept being gate_up's 1x128
    E4M3 quantization, half by half, for swiglu_bwd (half of gate_up's bytes;
    an operand of a GEMM too where I is a multiple of 128), or None without
    checkpoint."""
    T, cols, ld = _bf16_matrix(gate_up)
    inter = _halves(cols)
    h = gate_up.new_empty(T, inter)
    q = scales = None
    if checkpoint:
        q = gate_up.new_empty(T, cols, dtype=torch.uint8)
        scales = gate_up.new_empty(2 * -(-inter // 128), T, dtype=torch.float32)
    _lib.check(_lib.load().fgs_swiglu_fwd(
        gate_up.data_ptr(), T, inter, ld, h.data_ptr(), q.data_ptr() if checkpoint else 0,
        scales.data_ptr() if checkpoint else 0, _stream_of(gate_up)))
    if not checkpoint:
        return h, None
    return h, (_Halves if inter % 128 else Quantized)(q, scales, None, None, _lib.SCALE_TILE_1x128)


def swiglu_bwd(dh: torch.Tensor, kept: Union[Quantized, torch.Tensor]) -> torch.Tensor:
    """dgate_up [T x 2I] of swiglu_fwd from dh [T x I] and what was kept: the
    codes that it returned (the gradients are those at the values that the
    codes stand for), or gate_up itself.  bfloat16."""
    T, inter, lddh = _bf16_matrix(dh)
    gpu = dh.get_device()
    q = scales = x = 0
    ld = 2 * inter
    if isinstance(kept, Quantized):
        for t, name, dtype, shape in ((kept.q, "codes", torch.uint8, (T, 2 * inter)),
                                      (kept.scales, "scales", torch.float32, (2 * -(-inter // 128), T))):
            if t is None or t.dtype != dtype or tuple(t.shape) != shape or not t.is_contiguous() or t.get_device() != gpu:
                raise ValueError(f"the kept {name} must be a contiguous {shape} {dtype} tensor on dh's GPU")
        q, scales = kept.q.data_ptr(), kept.scales.data_ptr()
    else:
        rows, cols, ld = _bf16_matrix(kept)
        if (rows, cols) != (T, 2 * inter) or kept.get_device() != gpu:
            raise ValueError(f"gate_up must be a [{T} x {2 * inter}] tensor on dh's GPU (got {tuple(kept.shape)})")
        x = kept.data_ptr()
    out = dh.new_empty(T, 2 * inter)
    _lib.check(_lib.load().fgs_swiglu_bwd(dh.data_ptr(), lddh, x, ld, q, scales, T, inter, out.data_ptr(),
                                          _stream_of(dh)))
    return out


class _Swiglu(torch.autograd.Function):
    @staticmethod
    def forward(ctx, gate_up, checkpoint):
        gate_up = _readable(gate_up, gate_up.shape[-1])
        h, kept = swiglu_fwd(gate_up, checkpoint)
        ctx.checkpoint = checkpoint
        ctx.save_for_backward(*((kept.q, kept.scales) if checkpoint else (gate_up,)))
        return h

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dh):
        kept = ctx.saved_tensors
        kept = Quantized(*kept, None, None, _lib.SCALE_TILE_1x128) if ctx.checkpoint else kept[0]
        return swiglu_bwd(_readable(dh.to(torch.bfloat16), dh.shape[1]), kept), None


def swiglu(gate_up: torch.Tensor, checkpoint: bool = True) -> torch.Tensor:
    """swiglu_fwd's h with autograd.  checkpoint: what the backward pass
    needs of gate_up is kept in 8 bits, so gate_up itself need not be
    (False: it is kept as it is, and nothing is quantized, which is the form
    for passes without a gradient).  Layouts that the kernels do not read are
    copied."""
    return _Swiglu.apply(gate_up, checkpoint)
