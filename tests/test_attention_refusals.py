"""Arguments that attention refuses, before any HIP call (no GPU needed)."""
import ctypes

import pytest
import torch

from fine_grained_scaled_amd import _lib, attention_bwd, attention_fwd

FAKE, NULL = 0x10000, 0


def _view(data=FAKE, token=1024, head=128):
    return (ctypes.c_int64 * 3)(data, token, head)


def _fwd(q=None, k=None, v=None, cu=FAKE, S=1, T=64, H=8, Hk=2, D=128, scale=0.1, out=None, lse=FAKE):
    lib = _lib.load()
    return lib.fgs_attention_fwd(q or _view(), k or _view(), v or _view(), ctypes.c_void_p(cu), S, T, H, Hk, D, scale,
                                 out or _view(), ctypes.c_void_p(lse), ctypes.c_void_p(0))


def _bwd(T=64, ws=FAKE, ws_bytes=None, **views):
    lib = _lib.load()
    a = {n: views.get(n) or _view() for n in ("dout", "q", "k", "v", "out", "dq", "dk", "dv")}
    if ws_bytes is None:
        ws_bytes = lib.fgs_attention_workspace_bytes(T, 8)
    return lib.fgs_attention_bwd(a["dout"], a["q"], a["k"], a["v"], a["out"], ctypes.c_void_p(FAKE),
                                 ctypes.c_void_p(FAKE), 1, T, 8, 2, 128, 0.1, a["dq"], a["dk"], a["dv"],
                                 ctypes.c_void_p(ws), ws_bytes, ctypes.c_void_p(0))


@pytest.mark.parametrize("how", [dict(T=-1), dict(S=-1), dict(H=0), dict(Hk=0), dict(H=7), dict(scale=0.0),
                                 dict(scale=float("nan")), dict(scale=float("inf")), dict(cu=NULL), dict(cu=FAKE + 2),
                                 dict(q=_view(NULL)), dict(k=_view(token=-8)), dict(lse=NULL),
                                 dict(out=_view(token=64)), dict(out=_view(head=64))], ids=str)
def test_invalid(how):
    assert _fwd(**how) == _lib.FGS_ERR_INVALID_ARG
    assert _lib.load().fgs_last_error()


@pytest.mark.parametrize("how", [dict(D=96), dict(D=256), dict(q=_view(FAKE + 8)), dict(v=_view(token=1028)),
                                 dict(k=_view(token=1 << 23)), dict(T=0x7FFFFFFF), dict(T=1 << 30, H=128, Hk=128)], ids=str)
def test_unsupported(how):
    assert _fwd(**how) == _lib.FGS_ERR_UNSUPPORTED


def test_no_tokens_is_nothing():
    assert _fwd(T=0, cu=NULL, q=_view(NULL)) == _lib.FGS_OK
    assert _bwd(T=0, ws=NULL, ws_bytes=0) == _lib.FGS_OK


def test_workspace():
    lib = _lib.load()
    assert lib.fgs_attention_workspace_bytes(64, 8) == 64 * 8 * 8
    assert lib.fgs_attention_workspace_bytes(-1, 8) == 0
    assert _bwd(ws=NULL) == _lib.FGS_ERR_INVALID_ARG
    assert _bwd(ws_bytes=64 * 8 * 8 - 1) == _lib.FGS_ERR_INVALID_ARG
    assert b"workspace" in lib.fgs_last_error()
    assert _bwd(ws=FAKE + 4) == _lib.FGS_ERR_INVALID_ARG
    assert _bwd(dk=_view(head=0)) == _lib.FGS_ERR_INVALID_ARG
    assert _bwd(dout=_view(FAKE + 2)) == _lib.FGS_ERR_UNSUPPORTED


def test_python_refuses():
    q, k = torch.zeros(4, 8, 64, dtype=torch.bfloat16), torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    cu = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU"):
        attention_fwd(q, k, k, cu)
    with pytest.raises(TypeError):
        attention_fwd(q.float(), k, k, cu)
    with pytest.raises(TypeError):
        attention_bwd(q, q[0], k, k, q, torch.zeros(8, 4), cu)
