"""SwiGLU over every BF16 gate, with the other factors up to the ends of the
range: finite where the definition is, and within what the header says."""
import pytest
import torch

import fine_grained_scaled_amd as fgs
from _model_refs import E, F64, U

pytestmark = pytest.mark.gpu

LARGEST = float(torch.finfo(torch.bfloat16).max)


def _gates():
    g = torch.arange(65536, dtype=torch.int32, device="cuda").to(torch.int16).view(torch.bfloat16)
    g = g[g.isfinite()]
    return g[:g.numel() // 8 * 8]


def _ulp(v):
    return torch.ldexp(torch.ones_like(v), torch.frexp(v.abs().clamp(min=2.0 ** -126))[1] - 8)


@pytest.mark.parametrize("u", [1.0, -1.5, 1e-38, 1e-30, 1e20, -1e30, 1e38, 1.8e38, LARGEST, -LARGEST])
def test_forward(u):
    g = _gates()
    x = torch.cat([g, torch.full_like(g, u)])[None]
    h = fgs.swiglu_fwd(x, checkpoint=False)[0][0].to(F64)
    assert torch.equal(h, fgs.swiglu_fwd(x)[0][0].to(F64))
    v, u = g.to(F64), x[0, -1].to(F64)
    want = v * torch.sigmoid(v) * u
    fits = want.abs() <= LARGEST
    small = want.abs() < 2.0 ** -116
    assert ((h - want).abs() <= _ulp(want))[fits & ~small].all()
    assert ((h - want).abs() <= torch.maximum(_ulp(want), want.abs()))[small].all()      # 0 at worst
    over = want.abs() >= LARGEST * (1 + 2.0 ** -7)
    assert torch.equal(h[over], torch.sign(want[over]) * torch.inf)


@pytest.mark.parametrize("d", [1.0, 1e-10, -1e-30, 1e10, 1e30, 1e38])
@pytest.mark.parametrize("u", [1.0, 1e-20, 1e20, -3e30, 1e38])
def test_backward(d, u):
    g = _gates()
    x = torch.cat([g, torch.full_like(g, u)])[None]
    dh = torch.full_like(g, d)[None]
    got = fgs.swiglu_bwd(dh, x)[0].to(F64)
    v, u, d = g.to(F64), x[0, -1].to(F64), dh[0, 0].to(F64)
    s = torch.sigmoid(v)
    # what the header leaves out: a factor that is no normal number any more
    normal = (torch.minimum(u.abs(), d.abs()) * torch.exp(torch.clamp(v, max=0) / 2) >= 2.0 ** -125) & (v > -174)
    steps = (v.abs() + 16) * 2 * E
    for name, value, want, size in (("dg", got[:len(g)], d * u * s * (1 + v * (1 - s)), (d * u).abs() * s * (1 + v.abs() * (1 - s))),
                                    ("du", got[len(g):], d * v * s, (d * v).abs() * s)):
        assert not value.isnan().any(), name
        fits = normal & (want.abs() <= LARGEST * (1 - 2.0 ** -7))
        # (du has no other factor than the gate: below 2^-126 it is rounded to the smallest steps)
        assert ((value - want).abs() <= (U * want.abs() + steps * size) * 1.01 + 1e-37)[fits].all(), name
