"""Arguments that the output head's entry points refuse, before any HIP call
(no GPU needed)."""
import ctypes

import pytest
import torch

import fine_grained_scaled_amd as fgs
from fine_grained_scaled_amd import _lib

FAKE, NULL = 0x10000, 0
P = ctypes.c_void_p


def _need(T, V, K, backward):
    return _lib.load().fgs_linear_cross_entropy_workspace_bytes(T, V, K, backward)


def _fwd(x=FAKE, ldx=128, w=FAKE, ldw=128, targets=FAKE, index=1, T=4, V=100, K=128, loss=FAKE, lse=FAKE, ws=FAKE, ws_bytes=None):
    return _lib.load().fgs_linear_cross_entropy_fwd(P(x), ldx, P(w), ldw, P(targets), index, T, V, K, P(loss), P(lse), P(ws),
                                                    1 << 40 if ws_bytes is None else ws_bytes, P(0))


def _bwd(dloss=FAKE, dlse=FAKE, x=FAKE, ldx=128, w=FAKE, ldw=128, targets=FAKE, index=1, lse=FAKE, T=4, V=100, K=128,
         dx=FAKE, dw=FAKE, ws=FAKE, ws_bytes=None):
    return _lib.load().fgs_linear_cross_entropy_bwd(P(dloss), P(dlse), P(x), ldx, P(w), ldw, P(targets), index, P(lse),
                                                    T, V, K, P(dx), P(dw), P(ws), 1 << 40 if ws_bytes is None else ws_bytes,
                                                    P(0))


COMMON = [dict(T=-1), dict(V=0), dict(V=-3), dict(K=0), dict(index=2), dict(x=NULL), dict(w=NULL), dict(targets=NULL),
          dict(targets=FAKE + 4), dict(targets=FAKE + 2, index=0), dict(ldx=64), dict(ldw=120), dict(ws=NULL), dict(ws=FAKE + 8),
          dict(ws_bytes=1000)]


@pytest.mark.parametrize("how", COMMON + [dict(loss=NULL), dict(lse=NULL), dict(lse=FAKE + 2)], ids=str)
def test_forward_invalid(how):
    assert _fwd(**how) == _lib.FGS_ERR_INVALID_ARG
    assert _lib.load().fgs_last_error()


@pytest.mark.parametrize("how", COMMON + [dict(dloss=NULL), dict(lse=NULL), dict(dlse=FAKE + 2), dict(dx=NULL), dict(dw=NULL)],
                         ids=str)
def test_backward_invalid(how):
    assert _bwd(**how) == _lib.FGS_ERR_INVALID_ARG


UNSUPPORTED = [dict(K=96), dict(K=65600, ldx=65600, ldw=65600), dict(ldx=132), dict(ldw=130), dict(x=FAKE + 8), dict(w=FAKE + 2),
               dict(T=(1 << 23) + 1), dict(V=(1 << 24) + 1), dict(T=1 << 22, V=1 << 20),
               dict(T=1 << 20, K=32768, ldx=32768, ldw=32768), dict(V=1 << 23, K=65536, ldx=65536, ldw=65536)]


@pytest.mark.parametrize("how", UNSUPPORTED, ids=str)
def test_unsupported(how):
    assert _fwd(**how) == _lib.FGS_ERR_UNSUPPORTED
    assert _bwd(**how) == _lib.FGS_ERR_UNSUPPORTED


def test_no_tokens():
    assert _fwd(T=0, x=NULL, targets=NULL, loss=NULL, lse=NULL) == _lib.FGS_OK


def test_workspace_sizes():
    assert _need(0, 100, 128, 0) > 0 and _need(-1, 100, 128, 0) == _need(5, 100, 100, 1) == 0
    # a few tokens' parts, and one piece of the vocabulary at a time: far below the logits of a large call
    assert _need(16384, 128000, 4096, 1) < 16384 * 128000 * 2 // 2
    for T in (1, 64, 65, 257, 5000):
        assert _need(T, 1000, 256, 0) >= 8 * T and _need(T, 1000, 256, 1) >= 2 * T * (1000 + 256)


def _tensors(T=4, V=100, K=128):
    return torch.zeros(T, K, dtype=torch.bfloat16), torch.zeros(V, K, dtype=torch.bfloat16), torch.zeros(T, dtype=torch.int64)


def test_python_arguments():
    x, w, t = _tensors()
    for bad, error in (((x.float(), w, t), TypeError), ((x, w.half(), t), TypeError), ((x, w, t.float()), TypeError),
                       ((x, w, t[:3]), TypeError), ((x[:, :64], w, t), ValueError), ((x.t(), w, t), ValueError),
                       ((x, w, t.repeat(2)[::2]), TypeError), ((x[None], w, t), TypeError),
                       ((x, w, t), ValueError)):      # the last: right, but not on a GPU
        with pytest.raises(error):
            fgs.linear_cross_entropy_fwd(*bad)
        with pytest.raises(error):
            fgs.linear_cross_entropy_bwd(torch.zeros(4), *bad, torch.zeros(4))
