"""Arguments that the embedding's and SwiGLU's entry points refuse, before any
HIP call (no GPU needed)."""
import ctypes

import pytest
import torch

import fine_grained_scaled_amd as fgs
from fine_grained_scaled_amd import _lib

FAKE, NULL = 0x10000, 0
P = ctypes.c_void_p
NAN = float("nan")


def _fwd(tokens=FAKE, index=1, T=4, w=FAKE, ldw=64, wt=0, V=100, W=64, scale=1.0, out=FAKE, ot=0):
    return _lib.load().fgs_embedding_fwd(P(tokens), index, T, P(w), ldw, wt, V, W, scale, P(out), ot, P(0))


def _bwd(dout=FAKE, ldd=64, ot=0, tokens=FAKE, index=1, T=4, V=100, W=64, scale=1.0, dw=FAKE, wt=0, add=0, ws=FAKE, ws_bytes=1 << 40):
    return _lib.load().fgs_embedding_bwd(P(dout), ldd, ot, P(tokens), index, T, V, W, scale, P(dw), wt, add, P(ws), ws_bytes, P(0))


COMMON = [dict(T=-1), dict(V=0), dict(W=0), dict(index=3), dict(ot=2), dict(wt=-1), dict(scale=NAN), dict(scale=float("inf")),
          dict(tokens=NULL), dict(tokens=FAKE + 4)]


@pytest.mark.parametrize("how", COMMON + [dict(w=NULL), dict(out=NULL), dict(ldw=56)], ids=str)
def test_embedding_forward_invalid(how):
    assert _fwd(**how) == _lib.FGS_ERR_INVALID_ARG
    assert _lib.load().fgs_last_error()


@pytest.mark.parametrize("how", COMMON + [dict(dout=NULL), dict(dw=NULL), dict(ldd=56), dict(ws=NULL), dict(ws=FAKE + 8), dict(ws_bytes=16)],
                         ids=str)
def test_embedding_backward_invalid(how):
    assert _bwd(**how) == _lib.FGS_ERR_INVALID_ARG


@pytest.mark.parametrize("how", [dict(W=60), dict(W=65544, ldw=65544), dict(ldw=68), dict(w=FAKE + 8), dict(out=FAKE + 4),
                                 dict(T=1 << 24), dict(V=0x7FFFFFFF)], ids=str)
def test_embedding_forward_unsupported(how):
    assert _fwd(**how) == _lib.FGS_ERR_UNSUPPORTED


@pytest.mark.parametrize("how", [dict(W=60), dict(W=65544, ldd=65544), dict(ldd=68), dict(dw=FAKE + 8), dict(dout=FAKE + 4),
                                 dict(T=(1 << 22) + 1), dict(V=0x7FFFFFFF)], ids=str)
def test_embedding_backward_unsupported(how):
    assert _bwd(**how) == _lib.FGS_ERR_UNSUPPORTED


def test_embedding_no_tokens():
    assert _fwd(T=0, tokens=NULL, w=NULL, out=NULL) == _lib.FGS_OK
    assert _bwd(T=0, tokens=NULL, dout=NULL, ws=NULL, ws_bytes=0, add=1) == _lib.FGS_OK      # nothing to add


def test_embedding_workspace_sizes():
    need = _lib.load().fgs_embedding_workspace_bytes
    assert need(-1, 64) == need(1, 60) == need((1 << 22) + 1, 64) == 0
    for T in (1, 16, 17, 4096, 4097, 100000):
        assert need(T, 64) >= 8 * T


def _sfwd(x=FAKE, T=4, I=64, ld=128, h=FAKE, q=FAKE, s=FAKE):
    return _lib.load().fgs_swiglu_fwd(P(x), T, I, ld, P(h), P(q), P(s), P(0))


def _sbwd(dh=FAKE, ldh=64, x=NULL, ld=128, q=FAKE, s=FAKE, T=4, I=64, out=FAKE):
    return _lib.load().fgs_swiglu_bwd(P(dh), ldh, P(x), ld, P(q), P(s), T, I, P(out), P(0))


@pytest.mark.parametrize("how", [dict(x=NULL), dict(h=NULL), dict(T=-1), dict(I=-8), dict(ld=120), dict(s=NULL), dict(s=FAKE + 2)], ids=str)
def test_swiglu_forward_invalid(how):
    assert _sfwd(**how) == _lib.FGS_ERR_INVALID_ARG


@pytest.mark.parametrize("how", [dict(dh=NULL), dict(out=NULL), dict(T=-1), dict(ldh=56), dict(s=NULL), dict(q=NULL),
                                 dict(x=FAKE), dict(x=FAKE, q=NULL, ld=64)], ids=str)
def test_swiglu_backward_invalid(how):
    assert _sbwd(**how) == _lib.FGS_ERR_INVALID_ARG


@pytest.mark.parametrize("how", [dict(I=60), dict(ld=132), dict(x=FAKE + 8), dict(q=FAKE + 8), dict(T=1 << 26), dict(T=1 << 40),
                                 dict(T=8192, I=1 << 23, ld=1 << 24)], ids=str)
def test_swiglu_unsupported(how):
    assert _sfwd(**how) == _lib.FGS_ERR_UNSUPPORTED


def test_swiglu_nothing():
    assert _sfwd(T=0, x=NULL, h=NULL) == _sfwd(I=0, x=NULL, h=NULL) == _sbwd(T=0, dh=NULL, out=NULL) == _lib.FGS_OK


def test_python_arguments():
    w, t = torch.zeros(10, 8), torch.zeros(4, dtype=torch.int64)
    with pytest.raises(TypeError):
        fgs.embedding_fwd(t.float(), w)
    with pytest.raises(ValueError):
        fgs.embedding_fwd(t, w)                    # not on a GPU
    with pytest.raises(TypeError):
        fgs.embedding_bwd(torch.zeros(4, 8), t.repeat(2)[::2], 10)
    for bad in (torch.zeros(4, 6).bfloat16(), torch.zeros(4, 6)):
        with pytest.raises((TypeError, ValueError)):
            fgs.swiglu_fwd(bad)
    with pytest.raises((TypeError, ValueError)):
        fgs.swiglu_bwd(torch.zeros(4, 8).bfloat16(), torch.zeros(4, 16).bfloat16())
