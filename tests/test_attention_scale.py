"""The scales that attention takes: those with which scale * log2(e) and the
backward pass's lse / scale stay within FP32."""
import ctypes

import numpy as np
import pytest
import torch

from fine_grained_scaled_amd import _lib
from fine_grained_scaled_amd.attention import _check

FAKE = ctypes.c_void_p(0x10000)


def _refused(scale):
    lib = _lib.load()
    view = lambda: (ctypes.c_int64 * 3)(0x10000, 1024, 128)
    ws = lib.fgs_attention_workspace_bytes(64, 8)
    # a NULL lse ends the calls that are not refused for their scale before any HIP call
    null = ctypes.c_void_p(0)
    fwd = lib.fgs_attention_fwd(view(), view(), view(), FAKE, 1, 64, 8, 2, 128, scale, view(), null, null)
    bwd = lib.fgs_attention_bwd(view(), view(), view(), view(), view(), null, FAKE, 1, 64, 8, 2, 128, scale, view(),
                                view(), view(), FAKE, ws, null)
    assert fwd == bwd
    return fwd == _lib.FGS_ERR_UNSUPPORTED


@pytest.mark.parametrize("scale", [2.0 ** -101, 1e-38, 1e-45, 2.0 ** 101, 3e38])
def test_refused(scale):
    assert _refused(scale)
    assert b"scale" in _lib.load().fgs_last_error()


@pytest.mark.parametrize("scale", [2.0 ** -100, 1e-3, 0.088, 1.0, 2.0 ** 100])
def test_taken(scale):
    assert not _refused(scale)
    s, most = np.float32(scale), np.float32(np.log(2.0 ** 31))      # the row sum of as many equal scores as there can be
    assert np.isfinite(s * np.float32(1.4426950408889634)) and np.isfinite(most / s)


def test_what_lies_beyond():
    """Two equal scores at a scale of 1e-39: lse / scale overflows, and with it
    every probability of the backward pass would be 0 instead of 1/2."""
    with np.errstate(over="ignore"):
        assert np.isinf(np.float32(np.log(2.0)) / np.float32(1e-39))


def test_default():
    """1 / sqrt(head_dim); heads of no value get as far as their refusal."""
    cu = torch.zeros(2, dtype=torch.int32)
    for dim, scale in ((64, 0.125), (0, 1.0)):
        q = torch.zeros(3, 2, dim, dtype=torch.bfloat16)
        assert _check(q, q, q, cu, None)[4] == scale
