"""SwiGLU and its gradient against the definition in 64 bits, and what is kept in
8 bits against the library's quantizer."""
import pytest
import torch

import fine_grained_scaled_amd as fgs
from _model_refs import E, F64, U

pytestmark = pytest.mark.gpu


def _gate_up(T, I, seed=0, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(T, 2 * I, generator=g, device="cuda") * std
    x[:, ::37] *= 30
    return x.bfloat16()


def _halves(x):
    return x[:, :x.shape[1] // 2].to(F64), x[:, x.shape[1] // 2:].to(F64)


def _check_h(h, x):
    g, u = _halves(x)
    want = g * torch.sigmoid(g) * u
    # FP32 products, an exponent off by (|g| + 4) E, a reciprocal: a few steps, then BF16's rounding
    assert ((h.to(F64) - want).abs() <= (U + (g.abs() + 12) * 2 * E) * want.abs() * 1.01 + 1e-37).all()


def _gradients(g, u, dh):
    d, s = dh.to(F64), torch.sigmoid(g)
    dg, du = d * u * s * (1 + g * (1 - s)), d * g * s
    steps = (g.abs() + 16) * 2 * E
    size = d.abs() * u.abs() * s * (1 + g.abs() * (1 - s))       # 1 + g (1 - s) may cancel
    return torch.cat([dg, du], 1), torch.cat([U * dg.abs() + steps * size, (U + steps) * du.abs()], 1) * 1.01 + 1e-37


def _values(kept, I):
    """What the codes stand for."""
    T = kept.q.shape[0]
    codes = kept.q.view(torch.float8_e4m3fn).float()
    tiles = -(-I // 128)
    scale = kept.scales.t()
    per = lambda half: scale[:, half * tiles:(half + 1) * tiles].repeat_interleave(128, 1)[:, :I]
    return (codes * torch.cat([per(0), per(1)], 1)).to(F64) if T else codes.to(F64)


SIZES = [(1, 8), (300001, 8), (3, 9000), (7, 2048), (16, 128), (17, 136), (33, 1000), (300, 384), (128, 5464), (5, 120)]


@pytest.mark.parametrize("T, I", SIZES)
def test_forward(T, I):
    x = _gate_up(T, I, T)
    h, kept = fgs.swiglu_fwd(x)
    _check_h(h, x)
    plain, none = fgs.swiglu_fwd(x, checkpoint=False)
    assert none is None and torch.equal(plain, h)


@pytest.mark.parametrize("T, I", SIZES)
def test_kept_codes(T, I):
    x = _gate_up(T, I, T)
    _, kept = fgs.swiglu_fwd(x)
    tiles = -(-I // 128)
    for half in (0, 1):      # each half, its last tile filled up with zeros, through the library's quantizer
        padded = torch.zeros(T, 128 * tiles, device="cuda", dtype=torch.bfloat16)
        padded[:, :I] = x[:, half * I:(half + 1) * I]
        want = fgs.quantize_blockwise(padded, "tile")
        assert torch.equal(kept.q[:, half * I:(half + 1) * I], want.q[:, :I])
        assert torch.equal(kept.scales[half * tiles:(half + 1) * tiles], want.scales)
    if I % 128 == 0:
        want = fgs.quantize_blockwise(x, "tile")
        assert torch.equal(kept.q, want.q) and torch.equal(kept.scales, want.scales)


@pytest.mark.parametrize("T, I", SIZES)
@pytest.mark.parametrize("checkpoint", [True, False])
def test_backward(T, I, checkpoint):
    x = _gate_up(T, I, T)
    dh = (torch.randn(T, I, device="cuda") * 1e-2).bfloat16()
    if checkpoint:
        _, kept = fgs.swiglu_fwd(x)
        v = _values(kept, I)
        g, u = v[:, :I], v[:, I:]
    else:
        kept = x
        g, u = _halves(x)
    got = fgs.swiglu_bwd(dh, kept)
    want, bound = _gradients(g, u, dh)
    if checkpoint:       # the product of code and scale is rounded to FP32: the gradients at values off by E
        s = torch.sigmoid(g)
        d = dh.to(F64).abs()
        bound = bound + 4 * E * torch.cat([d * u.abs() * (1 + 2 * g.abs()) * s, d * g.abs() * (1 + g.abs()) * s], 1)
    assert ((got.to(F64) - want).abs() <= bound).all()


def test_special_values():
    """Zeros, tiny tiles, large values; NaN and Inf stay in their place in h, and in their tile in what is kept."""
    T, I = 16, 256
    x = _gate_up(T, I)
    x[0] = 0
    x[1] *= 2.0 ** -100
    x[2, :I], x[2, I:] = 100.0, 1e30
    x[3, :I] = -100.0
    h, kept = fgs.swiglu_fwd(x)
    _check_h(h, x)
    bad = x.clone()
    bad[5, 130], bad[6, I + 3] = float("nan"), float("inf")
    h2, kept2 = fgs.swiglu_fwd(bad)
    same = torch.ones(T, I, dtype=torch.bool, device="cuda")
    same[5, 130], same[6, 3] = False, False
    assert torch.equal(h2[same], h[same]) and h2[5, 130].isnan() and not h2[6, 3].isfinite()
    dh = torch.ones(T, I, device="cuda", dtype=torch.bfloat16)
    a, b = fgs.swiglu_bwd(dh, kept), fgs.swiglu_bwd(dh, kept2)
    hit = torch.zeros(T, 2 * I, dtype=torch.bool, device="cuda")
    hit[5, 128:256] = hit[5, I + 128:] = hit[6, :128] = hit[6, I:I + 128] = True
    assert torch.equal(a[~hit], b[~hit]) and b[hit].isnan().any()
    assert not a[0].any() and a.isfinite().all()


def test_strides():
    T, I = 40, 264
    x = _gate_up(T, I)
    wide = torch.zeros(T, 2 * I + 80, device="cuda", dtype=torch.bfloat16)
    wide[:, 16:16 + 2 * I] = x
    h, kept = fgs.swiglu_fwd(wide[:, 16:16 + 2 * I])
    want, want_kept = fgs.swiglu_fwd(x)
    assert torch.equal(h, want) and torch.equal(kept.q, want_kept.q) and torch.equal(kept.scales, want_kept.scales)
    dh = torch.randn(T, 2 * I, device="cuda").bfloat16()
    assert torch.equal(fgs.swiglu_bwd(dh[:, I:], kept), fgs.swiglu_bwd(dh[:, I:].contiguous(), kept))
    assert torch.equal(fgs.swiglu_bwd(dh[:, I:], wide[:, 16:16 + 2 * I]), fgs.swiglu_bwd(dh[:, I:].contiguous(), x))


def test_no_rows():
    x = _gate_up(0, 64)
    h, kept = fgs.swiglu_fwd(x)
    assert h.shape == (0, 64) and fgs.swiglu_bwd(h, kept).shape == (0, 128)


def test_differences():
    x = _gate_up(4, 64, std=0.7)
    dh = torch.randn(4, 64, device="cuda").bfloat16()
    got = fgs.swiglu_bwd(dh, x).to(F64)
    way = torch.randn(4, 128, device="cuda").to(F64)
    def total(step):
        v = x.to(F64) + step * way
        return (v[:, :64] * torch.sigmoid(v[:, :64]) * v[:, 64:] * dh.to(F64)).sum()
    slope = (total(1e-5) - total(-1e-5)) / 2e-5
    _, bound = _gradients(*_halves(x), dh)
    assert abs((got * way).sum() - slope) <= (bound * way.abs()).sum() + 1e-6


def test_autograd():
    x = _gate_up(50, 256).requires_grad_()
    dh = torch.randn(50, 256, device="cuda").bfloat16()
    fgs.swiglu(x).backward(dh)
    h, kept = fgs.swiglu_fwd(x.detach())
    assert torch.equal(x.grad, fgs.swiglu_bwd(dh, kept))
    x.grad = None
    fgs.swiglu(x, checkpoint=False).backward(dh)
    assert torch.equal(x.grad, fgs.swiglu_bwd(dh, x.detach()))
    x.grad = None
    fgs.swiglu(x).float().sum().backward()            # an expanded gradient
    assert torch.equal(x.grad, fgs.swiglu_bwd(torch.ones_like(dh), kept))


def test_what_is_kept_is_half():
    """The graph holds the codes and their scales, not gate_up."""
    saved = []
    with torch.autograd.graph.saved_tensors_hooks(lambda t: saved.append(t) or t, lambda t: t):
        x = _gate_up(256, 1024).requires_grad_()
        fgs.swiglu(x)
    assert sum(t.numel() * t.element_size() for t in saved) <= x.numel() * x.element_size() * (0.5 + 4 / 256)


def test_graph():
    T, I = 70, 392
    x, dh = _gate_up(T, I), torch.randn(T, I, device="cuda").bfloat16()
    fgs.swiglu_fwd(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        h, kept = fgs.swiglu_fwd(x)
        d = fgs.swiglu_bwd(dh, kept)
    for seed in range(3):
        x.copy_(_gate_up(T, I, seed + 4))
        graph.replay()
        torch.cuda.synchronize()
        want, want_kept = fgs.swiglu_fwd(x)
        assert torch.equal(h, want) and torch.equal(d, fgs.swiglu_bwd(dh, want_kept))
