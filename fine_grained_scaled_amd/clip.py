"""The global gradient norm over many tensors, and clipping (the kernels
behind fgs_clip_grad_norm)."""
from __future__ import annotations

import array
from typing import Optional, Sequence

import torch

from . import _lib
from .ops import _stream_of

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
    device = grads[0].device if grads else torch.device("cuda", torch.cuda.current_device())
    gpu = device.index if device.type == "cuda" else None
    # whole lists at a time: a call over hundreds of tensors is bound by this
    Tensor = torch.Tensor
    kinds, counts = [g.dtype for g in grads], [*map(Tensor.numel, grads)]
    if not set(kinds) <= _ELEM.keys():
        raise TypeError(f"gradients must be float32 or bfloat16 (got {set(kinds) - _ELEM.keys()})")
    if gpu is None or not set(map(Tensor.get_device, grads)) <= {gpu}:
        raise ValueError("gradients must be on one GPU")
    if not all(map(Tensor.is_contiguous, grads)):
        raise ValueError("gradients must be contiguous")
    data = to = [*map(Tensor.data_ptr, grads)]
    if out is not grads:
        if [o.dtype for o in out] != kinds or [*map(Tensor.numel, out)] != counts \
                or not set(map(Tensor.get_device, out)) <= {gpu} or not all(map(Tensor.is_contiguous, out)):
            raise ValueError("each out tensor must be contiguous, of its gradient's type, size and GPU")
        to = [*map(Tensor.data_ptr, out)]
    table = array.array("q", bytes(32 * len(grads)))
    table[0::4], table[1::4], table[2::4] = (array.array("q", v) for v in (data, to, counts))
    table[3::4] = array.array("q", map(_ELEM.__getitem__, kinds))
    lib = _lib.load()
    norm = torch.empty((), dtype=torch.float32, device=device)
    if workspace is None:
        workspace = torch.empty(lib.fgs_clip_workspace_bytes(len(grads)), dtype=torch.uint8, device=device)
    elif workspace.device != device or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the gradients' GPU")
    _lib.check(lib.fgs_clip_grad_norm(
        table.buffer_info()[0], len(grads), max_norm, norm.data_ptr(), workspace.data_ptr(),
        workspace.numel() * workspace.element_size(), _stream_of(norm)))
    torch.autograd.graph.increment_version(out)      # written behind torch's back: graphs that saved them have to know
    return norm
