"""Attention's sequence offsets: packs of more sequences than the backward
pass sorts, packs with much padding, and offsets that are no offsets, with
which every access stays inside the tensors (their rows are gone through on
the CPU in test_attention_tiles.py)."""
import ctypes

import pytest
import torch

import fine_grained_scaled_amd as fgs
from fine_grained_scaled_amd import _lib
from _operator_refs import attention, pack_offsets, within

pytestmark = pytest.mark.gpu
EDGE = 4096      # bytes kept free around every tensor


def _apart(shape, dtype, fill=None):
    """A tensor of the shape inside a buffer of 0x5B bytes, and the buffer."""
    size = torch.empty(0, dtype=dtype).element_size() * torch.Size(shape).numel()
    flat = torch.full((size + 2 * EDGE,), 0x5B, dtype=torch.uint8, device="cuda")
    t = flat[EDGE:EDGE + size].view(dtype).view(shape)
    if fill is not None:
        t.copy_(fill)
    return t, flat


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T,H,Hk", [(1100, 4, 2), (300, 3, 3), (1500, 8, 1)])
@pytest.mark.parametrize("offsets", [
    [0, "T", 0, "T", "T+5"], ["T", 0], ["T", 0, "T"], [-7, "T/2", "T/3", "T+9"], [2 ** 31 - 1, -2 ** 31, 50],
    ["T/2"] * 3 + [3], [0, "T"] * 30, [0, "T"] * 31, [0, "T"] * 127, ["T", 0] * 127, [0, "T"] * 150, ["T", 1] * 150],
    ids=lambda o: str(o[:5]) + f"x{len(o)}")
def test_no_offsets_leave_the_tensors(offsets, T, H, Hk, D):
    at = {"T": T, "T+5": T + 5, "T+9": T + 9, "T/2": T // 2, "T/3": T // 3}
    cu, cu_flat = _apart((len(offsets),), torch.int32, torch.tensor([at.get(o, o) for o in offsets]))
    g = torch.Generator().manual_seed(T)
    heads = dict(q=H, k=Hk, v=Hk, out=H, dout=H, dq=H, dk=Hk, dv=Hk)
    ten = {n: _apart((T, h, D), torch.bfloat16,
                     torch.randn(T, h, D, generator=g) if n in ("q", "k", "v", "dout") else 0.0)
           for n, h in heads.items()}
    lse, lse_flat = _apart((H, T), torch.float32, 0.0)
    lib = _lib.load()
    ws, ws_flat = _apart((lib.fgs_attention_workspace_bytes(T, H),), torch.uint8, 0)
    view = {n: (ctypes.c_int64 * 3)(t.data_ptr(), heads[n] * D, D) for n, (t, _) in ten.items()}
    P = ctypes.c_void_p
    stream = P(torch.cuda.current_stream().cuda_stream)
    shape = (P(cu.data_ptr()), len(offsets) - 1, T, H, Hk, D, D ** -0.5)
    _lib.check(lib.fgs_attention_fwd(view["q"], view["k"], view["v"], *shape, view["out"], P(lse.data_ptr()), stream))
    _lib.check(lib.fgs_attention_bwd(view["dout"], view["q"], view["k"], view["v"], view["out"], P(lse.data_ptr()), *shape,
                                     view["dq"], view["dk"], view["dv"], P(ws.data_ptr()), ws.numel(), stream))
    torch.cuda.synchronize()
    for name, flat in [(n, f) for n, (_, f) in ten.items()] + [("lse", lse_flat), ("ws", ws_flat), ("cu", cu_flat)]:
        assert (flat[:EDGE] == 0x5B).all() and (flat[-EDGE:] == 0x5B).all(), name


def _check(lengths, H, Hk, D, after=0, seed=0):
    g = torch.Generator().manual_seed(seed)
    T = sum(lengths) + after
    q, k, v, dout = (torch.randn(T, h, D, generator=g).to(torch.bfloat16) for h in (H, Hk, Hk, H))
    cu = pack_offsets(lengths)
    want = attention(q, k, v, cu, D ** -0.5, dout)
    on = [t.cuda() for t in (q, k, v)]
    out, lse = fgs.attention_fwd(*on, cu.cuda())
    got = dict(zip(("dq", "dk", "dv"), fgs.attention_bwd(dout.cuda(), *on, out, lse, cu.cuda())), out=out, lse=lse)
    for name, t in got.items():
        within(name, t, want[name])


@pytest.mark.parametrize("lengths,H,Hk,D", [([3] * 150 + [1300] + [2] * 149, 2, 1, 64), ([1, 0] * 140 + [1030, 17], 4, 2, 128),
                                            ([1100] + [5] * 253, 2, 2, 64), ([1100] + [5] * 254, 2, 2, 64)],
                         ids=["300", "282", "254", "255"])
def test_many_sequences_and_a_long_one(lengths, H, Hk, D):
    _check(lengths, H, Hk, D, seed=len(lengths))


@pytest.mark.parametrize("after", [1300, 9000])
def test_a_long_sequence_and_padding(after):
    _check([1300], 2, 1, 64, after=after)
