"""Arguments that the block boundary and the clipping refuse, before any HIP
call (no GPU needed)."""
import ctypes

import pytest
import torch

import fine_grained_scaled_amd as fgs
from fine_grained_scaled_amd import _lib

FAKE, NULL = 0x10000, 0
P = ctypes.c_void_p


def _fwd(y=FAKE, ldy=64, x=FAKE, ldx=64, res=0, rows=4, width=64, w_post=FAKE, gate=FAKE, ldg=64, kind=2, alpha=1.0,
         w_pre=FAKE, eps=1e-6, r=FAKE, n=FAKE):
    return _lib.load().fgs_residual_norm_fwd(P(y), ldy, P(x), ldx, res, rows, width, P(w_post), P(gate), ldg, kind,
                                             alpha, P(w_pre), eps, P(r), P(n), P(0))


def _bwd(rows=4, width=64, w_post=FAKE, kind=1, dgate=FAKE, dw_post=FAKE, dw_pre=FAKE, ws=FAKE, ws_bytes=None, dr=FAKE,
         lddn=64):
    lib = _lib.load()
    if ws_bytes is None:
        ws_bytes = lib.fgs_residual_norm_workspace_bytes(rows, width)
    return lib.fgs_residual_norm_bwd(P(dr), 64, P(FAKE), lddn, P(FAKE), 64, P(FAKE), 64, 0, rows, width, P(w_post),
                                     P(FAKE), 64, kind, 1.0, P(FAKE), 1e-6, P(FAKE), P(FAKE), P(dgate), P(dw_post),
                                     P(dw_pre), P(ws), ws_bytes, P(0))


@pytest.mark.parametrize("how", [dict(res=2), dict(kind=3), dict(rows=-1), dict(width=0), dict(eps=-1.0),
                                 dict(eps=float("nan")), dict(alpha=float("inf")), dict(w_pre=NULL),
                                 dict(y=NULL), dict(x=NULL), dict(r=NULL), dict(n=NULL), dict(ldy=56),
                                 dict(gate=NULL), dict(gate=NULL, kind=1)], ids=str)
def test_norm_invalid(how):
    assert _fwd(**how) == _lib.FGS_ERR_INVALID_ARG
    assert _lib.load().fgs_last_error()


@pytest.mark.parametrize("how", [dict(width=60), dict(width=16392, ldy=16392, ldx=16392, ldg=16392), dict(ldx=68),
                                 dict(y=FAKE + 8), dict(w_post=FAKE + 4), dict(ldg=68)], ids=str)
def test_norm_unsupported(how):
    assert _fwd(**how) == _lib.FGS_ERR_UNSUPPORTED


def test_norm_no_rows_is_nothing():
    assert _fwd(rows=0, y=NULL, x=NULL, r=NULL, n=NULL, w_pre=NULL) == _lib.FGS_OK


@pytest.mark.parametrize("how", [dict(dw_pre=NULL), dict(dw_post=NULL), dict(dgate=NULL), dict(dgate=NULL, kind=2),
                                 dict(ws=NULL), dict(ws_bytes=100), dict(ws=FAKE + 4), dict(dr=NULL), dict(lddn=8)],
                         ids=str)
def test_norm_backward_invalid(how):
    assert _bwd(**how) == _lib.FGS_ERR_INVALID_ARG


def _clip(entries, max_norm=1.0, norm=FAKE, ws=FAKE, ws_bytes=1 << 20, count=None):
    table = (ctypes.c_int64 * max(1, 4 * len(entries)))(*[v for e in entries for v in e])
    return _lib.load().fgs_clip_grad_norm(table, len(entries) if count is None else count, max_norm, P(norm), P(ws),
                                          ws_bytes, P(0))


@pytest.mark.parametrize("entry", [(NULL, FAKE, 4, 0), (FAKE, NULL, 4, 0), (FAKE, FAKE, -1, 0), (FAKE, FAKE, 4, 2),
                                   (FAKE, FAKE, 1 << 41, 0)], ids=str)
def test_clip_invalid(entry):
    assert _clip([(FAKE, FAKE, 4, 0), entry]) == _lib.FGS_ERR_INVALID_ARG
    assert b"grads[1]" in _lib.load().fgs_last_error()


def test_clip_more():
    assert _clip([(FAKE + 2, FAKE, 4, 0)]) == _lib.FGS_ERR_UNSUPPORTED
    assert _clip([(FAKE, FAKE + 1, 4, 1)]) == _lib.FGS_ERR_UNSUPPORTED
    assert _clip([], count=-1) == _lib.FGS_ERR_INVALID_ARG
    for how in (dict(max_norm=-1.0), dict(max_norm=float("nan")), dict(norm=NULL), dict(ws=NULL), dict(ws_bytes=8)):
        assert _clip([(FAKE, FAKE, 4, 0)], **how) == _lib.FGS_ERR_INVALID_ARG
    lib = _lib.load()
    assert lib.fgs_clip_workspace_bytes(-1) == 0 and lib.fgs_clip_workspace_bytes(0) > 0
    assert lib.fgs_clip_workspace_bytes(129) > lib.fgs_clip_workspace_bytes(128)


def test_python_refuses():
    y, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.ones(64)
    with pytest.raises(ValueError, match="GPU"):
        fgs.residual_norm_fwd(y, y, w_pre=w)
    for bad in (dict(w_pre=w.half()), dict(w_pre=w[:8]), dict(w_pre=w, w_post=w.double()),
                dict(w_pre=w, gate=torch.zeros(4, 64))):
        with pytest.raises((TypeError, ValueError)):
            fgs.residual_norm_fwd(y, y, **bad)
    with pytest.raises(TypeError):
        fgs.residual_norm_fwd(y, y.half(), w_pre=w)
    with pytest.raises(ValueError):
        fgs.clip_grad_norm([w], 1.0)
    with pytest.raises(ValueError):
        fgs.clip_grad_norm([w], 1.0, out=[])
