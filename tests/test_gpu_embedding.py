"""Token embedding and its gradient against the definition in 64 bits: types,
odd sizes, tokens that fill most positions, tokens outside the vocabulary, sums
added to a gradient that is there."""
import pytest
import torch

import fine_grained_scaled_amd as fgs
from _model_refs import E, F64, U

pytestmark = pytest.mark.gpu

FP32, BF16 = torch.float32, torch.bfloat16


def _half(dtype):
    return U if dtype == BF16 else E


def _tokens(T, V, seed=0, kind="any", index=torch.int64):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = torch.randint(0, V, (T,), generator=g, device="cuda")
    if kind == "padded":
        t = torch.where(torch.rand(T, generator=g, device="cuda") < 0.8, V // 2, t)
    if kind == "one":
        t = torch.full((T,), V - 1, device="cuda")
    if kind == "outside":
        t = torch.where(torch.rand(T, generator=g, device="cuda") < 0.3, torch.tensor([-1, V, -2 ** 31, 2 ** 31 - 1], device="cuda")[t % 4], t)
    if kind == "few":
        t = t % 3
    return t.to(index)


@pytest.mark.parametrize("weight", [FP32, BF16])
@pytest.mark.parametrize("out", [FP32, BF16])
@pytest.mark.parametrize("T, V, W", [(1, 1, 8), (7, 100, 4096), (37, 1000, 8), (300, 33, 72), (1000, 500, 1000), (5, 9, 16392)])
def test_forward(weight, out, T, V, W):
    w = torch.randn(V, W, device="cuda").to(weight)
    for kind, index in (("any", torch.int64), ("outside", torch.int32)):
        t = _tokens(T, V, kind=kind, index=index)
        got = fgs.embedding_fwd(t, w, scale=0.3, out_dtype=out)
        inside = (t >= 0) & (t < V)
        want = torch.where(inside[:, None], w[torch.where(inside, t, 0).long()].to(F64) * 0.3, 0.0)
        # 0.3 is rounded to FP32, and so is the product, before the result is
        assert ((got.to(F64) - want).abs() <= (_half(out) + 2.1 * E) * want.abs()).all()
        assert got.dtype == out and got.shape == (T, W)


def test_forward_shapes_and_strides():
    t = _tokens(24, 50).view(2, 3, 4)
    with pytest.raises(fgs.FgsError):        # rows that are no multiple of 8 values apart
        fgs.embedding_fwd(t, torch.randn(50, 300, device="cuda")[:, 8:264])
    w = torch.randn(50, 304, device="cuda")
    assert torch.equal(fgs.embedding_fwd(t, w[:, 8:264]), w[:, 8:264][t])
    assert fgs.embedding_fwd(t[:0], w[:, :8]).shape == (0, 3, 4, 8)
    assert torch.equal(fgs.embedding_fwd(t[0, 0, 0], w[:, :8]), w[t[0, 0, 0], :8])


def _gradient(dout, t, V, scale):
    """(value, bound): a sum of n FP32 values is off by n E times the sum of their magnitudes, scale and its product by 2 E."""
    d = dout.to(F64)
    inside = (t >= 0) & (t < V)
    at, d = t[inside].long(), d[inside]
    value = torch.zeros(V, d.shape[1], dtype=F64, device="cuda").index_add_(0, at, d) * scale
    size = torch.zeros(V, d.shape[1], dtype=F64, device="cuda").index_add_(0, at, d.abs()) * abs(scale)
    count = torch.bincount(at, minlength=V).to(F64)[:, None]
    return value, (count + 3) * E * size


KINDS = ["any", "padded", "one", "outside", "few"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T, V, W", [(1, 1, 8), (15, 40, 64), (16, 40, 64), (17, 40, 520), (64, 7, 8), (1000, 3000, 264),
                                     (4096, 500, 128), (4097, 500, 128), (9000, 70000, 72), (20000, 1000, 2056)])
@pytest.mark.parametrize("dout_type, dtype", [(BF16, FP32), (FP32, BF16), (FP32, FP32), (BF16, BF16)])
def test_gradient(kind, T, V, W, dout_type, dtype):
    t = _tokens(T, V, seed=T, kind=kind, index=torch.int32 if W == 64 else torch.int64)
    dout = torch.randn(T, W, device="cuda").to(dout_type)
    got = fgs.embedding_bwd(dout, t, V, scale=1.7, dtype=dtype)
    value, bound = _gradient(dout, t, V, 1.7)
    assert got.dtype == dtype
    assert ((got.to(F64) - value).abs() <= bound + _half(dtype) * (value.abs() + bound)).all()
    assert torch.equal(got, fgs.embedding_bwd(dout, t, V, scale=1.7, dtype=dtype))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", [FP32, BF16])
@pytest.mark.parametrize("T", [0, 1, 700, 5000])
def test_added_to_a_gradient(kind, dtype, T):
    V, W = 900, 136
    t = _tokens(T, V, kind=kind)
    dout = torch.randn(T, W, device="cuda")
    old = torch.randn(V, W, device="cuda").to(dtype)
    out = old.clone()
    version = out._version
    assert fgs.embedding_bwd(dout, t, V, out=out) is out and out._version > version
    value, bound = _gradient(dout, t, V, 1.0)
    want = old.to(F64) + value
    assert ((out.to(F64) - want).abs() <= bound + 2 * E * (old.to(F64).abs() + value.abs()) + _half(dtype) * (want.abs() + bound)).all()
    idle = torch.ones(V, dtype=torch.bool, device="cuda")
    idle[t[(t >= 0) & (t < V)]] = False
    assert torch.equal(out[idle], old[idle])


def test_many_tokens():
    """More chunks than the waves that search them, and pieces of the greatest length."""
    T, V, W = 300001, 5000, 64
    for kind in ("any", "padded"):
        t = _tokens(T, V, kind=kind)
        dout = torch.randn(T, W, device="cuda").bfloat16()
        value, bound = _gradient(dout, t, V, 1.0)
        assert ((fgs.embedding_bwd(dout, t, V).to(F64) - value).abs() <= bound + E * value.abs()).all()


def test_rows_of_tokens_outside_reach_nothing():
    t = _tokens(5000, 300, kind="outside")
    dout = torch.randn(5000, 64, device="cuda")
    want = fgs.embedding_bwd(dout, t, 300)
    dout[(t < 0) | (t >= 300)] = float("nan")
    assert torch.equal(fgs.embedding_bwd(dout, t, 300), want)
    outside = torch.full((70,), -1, device="cuda")
    assert not fgs.embedding_bwd(dout[:70], outside, 300).any()


def test_gradient_strides_and_shapes():
    V, W = 40, 64
    t = _tokens(30, V).view(5, 6)
    wide = torch.randn(5, 6, 3 * W, device="cuda")
    dense = wide[..., W:2 * W].contiguous()
    want = fgs.embedding_bwd(dense.view(30, W), t.view(-1), V)
    assert torch.equal(fgs.embedding_bwd(wide[..., W:2 * W], t, V), want)
    assert torch.equal(fgs.embedding_bwd(wide.view(30, -1)[:, W:2 * W], t.view(-1), V), want)


def test_autograd():
    V, W = 300, 64
    t = _tokens(12, V).view(3, 4)
    for dtype in (FP32, BF16):
        w = torch.randn(V, W, device="cuda").to(dtype).requires_grad_()
        out = fgs.embedding(t, w, 2.0, FP32)
        g = torch.randn(3, 4, W, device="cuda")
        out.backward(g)
        assert w.grad.dtype == dtype and torch.equal(w.grad, fgs.embedding_bwd(g, t, V, 2.0, dtype))
        w.grad = None
        fgs.embedding(t, w).sum().backward()        # an expanded gradient, no strides
        counts = torch.bincount(t.flatten(), minlength=V).float()[:, None].expand(V, W)
        assert torch.equal(w.grad.float(), counts)


def test_differences():
    V, W = 20, 16
    t = _tokens(50, V, kind="few")
    g = torch.randn(50, W, device="cuda")
    dw = fgs.embedding_bwd(g, t, V, 0.5).to(F64)
    way = torch.randn(V, W, device="cuda").to(F64)
    total = lambda w: (0.5 * w[t] * g.to(F64)).sum()
    w = torch.randn(V, W, device="cuda").to(F64)
    slope = (total(w + way) - total(w - way)) / 2                     # linear: exact but for rounding
    assert abs((dw * way).sum() - slope) <= 60 * E * (way.abs() * _gradient(g.abs(), t, V, 0.5)[0]).sum()


def test_graph():
    V, W, T = 3000, 256, 5000
    t, dout = _tokens(T, V), torch.randn(T, W, device="cuda")
    kept = torch.zeros(V, W, device="cuda")
    fgs.embedding_bwd(dout, t, V)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fresh = fgs.embedding_bwd(dout, t, V)
        fgs.embedding_bwd(dout, t, V, out=kept)
    total = kept.clone()
    for seed, kind in enumerate(KINDS):
        t.copy_(_tokens(T, V, seed=seed, kind=kind))
        dout.normal_()
        fgs.embedding_bwd(dout, t, V, out=total)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(fresh, fgs.embedding_bwd(dout, t, V)) and torch.equal(kept, total)
