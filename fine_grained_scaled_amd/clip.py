"""The global gradient norm over many tensors, and clipping (the kernels
behind fgs_clip_grad_norm)."""
from __future__ import annotations

import array
import ctypes
from typing import Optional, Sequence

import torch

from . import _lib
from .ops import _ptr, _stream

_ELEM = {torch.float32: _lib.OUT_FP32, torch.bfloat16: _lib.OUT_BF16}


def clip_grad_norm(grads: Sequence[torch.Tensor], max_norm: float, out: Optional[Sequence[torch.Tensor]] = None,
                   workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Scale all gradients by max_norm / norm where their global norm is above
    max_norm, in place or into `out` (one tensor for each gradient, of its
    type and size), and return the norm before clipping (float32, on the GPU;
    nothing waits for it).  grads: contiguous float32 and bfloat16 GPU
    tensors.  workspace: optional uint8 device scratch of
    fgs_clip_workspace_bytes() bytes."""
    grads = list(grads)
    out = grads if out is None else list(out)
    if len(out) != len(grads):
        raise ValueError(f"out must hold one tensor for each of the {len(grads)} gradients (got {len(out)})")
    table = array.array("q")
    device = grads[0].device if grads else torch.device("cuda", torch.cuda.current_device())
    for g, o in zip(grads, out):
        kind, n = g.dtype, g.numel()
        if kind not in _ELEM:
            raise TypeError(f"gradients must be float32 or bfloat16 (got {kind})")
        if g.device != device or device.type != "cuda":
            raise ValueError("gradients must be on one GPU")
        if not g.is_contiguous():
            raise ValueError("gradients must be contiguous")
        if o is not g and (o.dtype != kind or o.numel() != n or o.device != device or not o.is_contiguous()):
            raise ValueError("each out tensor must be contiguous, of its gradient's type, size and GPU")
        table.extend((g.data_ptr(), o.data_ptr(), n, _ELEM[kind]))
    lib = _lib.load()
    norm = torch.empty((), dtype=torch.float32, device=device)
    if workspace is None:
        workspace = torch.empty(lib.fgs_clip_workspace_bytes(len(grads)), dtype=torch.uint8, device=device)
    elif workspace.device != device or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the gradients' GPU")
    _lib.check(lib.fgs_clip_grad_norm(ctypes.c_void_p(table.buffer_info()[0]), len(grads), max_norm, _ptr(norm),
                                      _ptr(workspace), workspace.numel() * workspace.element_size(), _stream()))
    return norm
