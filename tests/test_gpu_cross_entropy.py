"""The output head with softmax cross entropy against its definition in 64
bits: loss, lse and the gradients, at odd sizes, for masked tokens, strided
inputs and vocabularies in pieces."""
import pytest
import torch

import fine_grained_scaled_amd as fgs
from _model_refs import check, linear_cross_entropy

pytestmark = pytest.mark.gpu


def _inputs(T, V, K, seed=0, masked=0.0, index=torch.int64, known=4.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    w = (torch.randn(V, K, generator=g, device="cuda") * 1.5 * K ** -0.5).bfloat16()
    targets = torch.randint(0, V, (T,), generator=g, device="cuda")
    x = torch.randn(T, K, generator=g, device="cuda") + w[targets].float() * known * torch.rand(T, 1, generator=g, device="cuda")
    hidden = torch.rand(T, generator=g, device="cuda") < masked
    targets = torch.where(hidden, -100, targets).to(index)
    dloss = torch.rand(T, generator=g, device="cuda") * 2.0 / max(T, 1)
    return x.bfloat16(), w, targets, dloss


def _compare(x, w, targets, dloss, dlse=None):
    loss, lse = fgs.linear_cross_entropy_fwd(x, w, targets)
    dx, dw = fgs.linear_cross_entropy_bwd(dloss, x, w, targets, lse, dlse)
    want = linear_cross_entropy(x, w, targets, dloss, dlse)
    for name, got in (("loss", loss), ("lse", lse), ("dx", dx), ("dw", dw)):
        check(name, got, want[name])
    return loss, lse, dx, dw


@pytest.mark.parametrize("T", [1, 5, 64, 65, 256, 257, 700])
@pytest.mark.parametrize("V, K", [(1, 64), (7, 64), (128, 128), (129, 320), (1000, 576), (5003, 256)])
def test_sizes(T, V, K):
    _compare(*_inputs(T, V, K, seed=T + V))


@pytest.mark.parametrize("T, masked", [(40, 0.5), (300, 0.5), (300, 0.99), (300, 1.0), (2000, 0.9), (1, 1.0)])
@pytest.mark.parametrize("index", [torch.int32, torch.int64])
def test_masked(T, masked, index):
    _compare(*_inputs(T, 777, 128, seed=T, masked=masked, index=index))


@pytest.mark.parametrize("T, V, K", [(8200, 17001, 64), (16000, 9000, 128), (17, 600000, 64)])
def test_vocabulary_in_pieces(T, V, K):
    _compare(*_inputs(T, V, K, masked=0.3))


@pytest.mark.parametrize("T", [33, 400])
def test_gradient_of_lse(T):
    x, w, targets, dloss = _inputs(T, 1003, 192, masked=0.2)
    dlse = torch.randn(T, device="cuda") * 1e-3
    _compare(x, w, targets, dloss, dlse)
    _compare(x, w, targets, torch.zeros_like(dloss), dlse)


@pytest.mark.parametrize("T", [20, 333])
def test_strides(T):
    V, K = 515, 128
    x, w, targets, dloss = _inputs(T, V, K)
    wide_x, wide_w = torch.full((T, K + 72), 7.0, device="cuda").bfloat16(), torch.full((V, 3 * K), 7.0, device="cuda").bfloat16()
    wide_x[:, 8:8 + K], wide_w[:, K:2 * K] = x, w
    a = _compare(wide_x[:, 8:8 + K], wide_w[:, K:2 * K], targets, dloss)
    for one, other in zip(a, _compare(x, w, targets, dloss)):
        assert torch.equal(one, other)


@pytest.mark.parametrize("T", [50, 600])
def test_targets_outside_take_no_part(T):
    x, w, targets, dloss = _inputs(T, 300, 64)
    targets[::7], targets[3::7], targets[5::7] = -100, 300, 2 ** 40
    _compare(x, w, targets, dloss)
    out = (targets < 0) | (targets >= 300)
    clean = _compare(x, w, targets, dloss)
    x[out], dloss[out] = float("nan"), float("inf")
    for one, other in zip(clean, (lambda r: (*r, *fgs.linear_cross_entropy_bwd(dloss, x, w, targets, r[1])))(
            fgs.linear_cross_entropy_fwd(x, w, targets))):
        assert torch.equal(one, other)


def test_no_tokens():
    x, w, targets, dloss = _inputs(0, 300, 64)
    loss, lse = fgs.linear_cross_entropy_fwd(x, w, targets)
    dx, dw = fgs.linear_cross_entropy_bwd(dloss, x, w, targets, lse)
    assert loss.shape == lse.shape == (0,) and dx.shape == (0, 64) and not dw.any()


@pytest.mark.parametrize("size", [0.0, 1e-38, 1e-20, 1e20, 3e38])
def test_sizes_of_dloss(size):
    """The gradients scale with dloss over FP32's range, as far as BF16 goes."""
    x, w, targets, _ = _inputs(70, 200, 64)
    dloss = torch.full((70,), size, device="cuda")
    _, lse = fgs.linear_cross_entropy_fwd(x, w, targets)
    dx, dw = fgs.linear_cross_entropy_bwd(dloss, x, w, targets, lse)
    one = fgs.linear_cross_entropy_bwd(torch.ones_like(dloss), x, w, targets, lse)
    for got, unit in zip((dx, dw), one):
        want = unit.double() * float(dloss[0])
        fits = want.abs() < 3.3e38
        # both rounded to BF16, and what lies below its smallest value
        assert ((got.double() - want).abs()[fits] <= 2.02 * 2.0 ** -8 * want.abs()[fits] + 1e-38).all()


def test_large_logits():
    """Scores in the thousands: the statistics neither overflow nor vanish."""
    x, w, targets, dloss = _inputs(300, 500, 128)
    _compare((x.float() * 100).bfloat16(), (w.float() * 10).bfloat16(), targets, dloss)


def test_same_bits():
    x, w, targets, dloss = _inputs(3000, 3001, 256, masked=0.3)
    a = _compare(x, w, targets, dloss)
    for one, other in zip(a, _compare(x, w, targets, dloss)):
        assert torch.equal(one, other)


def test_non_finite_logits_reach_their_row_alone():
    x, w, targets, dloss = _inputs(300, 500, 128)
    loss, lse = fgs.linear_cross_entropy_fwd(x, w, targets)
    bad = x.clone()
    bad[17] = float("nan")
    got, got_lse = fgs.linear_cross_entropy_fwd(bad, w, targets)
    keep = torch.arange(300, device="cuda") != 17
    assert got[17].isnan() and got_lse[17].isnan()
    assert torch.equal(got[keep], loss[keep]) and torch.equal(got_lse[keep], lse[keep])
    dx, _ = fgs.linear_cross_entropy_bwd(dloss, x, w, targets, lse)
    got_dx, _ = fgs.linear_cross_entropy_bwd(dloss, bad, w, targets, got_lse)
    assert got_dx[17].isnan().all() and torch.equal(got_dx[keep], dx[keep])


def test_differences():
    """The gradients against differences of the loss in 64 bits."""
    x, w, targets, dloss = _inputs(9, 50, 64)
    _, lse = fgs.linear_cross_entropy_fwd(x, w, targets)
    dx, dw = fgs.linear_cross_entropy_bwd(dloss, x, w, targets, lse)
    g = torch.Generator(device="cuda").manual_seed(1)
    for t, grad, which in ((x, dx, 0), (w, dw, 1)):
        way = torch.randn(t.shape, generator=g, device="cuda").double()
        def total(step):
            a, b = x.double(), w.double()
            a, b = (a + step * way, b) if which == 0 else (a, b + step * way)
            return (torch.nn.functional.cross_entropy(a @ b.T, targets, reduction="none") * dloss.double()).sum()
        slope = float((total(1e-5) - total(-1e-5)) / 2e-5)
        # each product's gradient is off by two BF16 roundings at most
        bound = 2.1 * 2.0 ** -8 * float((linear_cross_entropy(x, w, targets, dloss)["dx" if which == 0 else "dw"][0].abs()
                                         * way.abs()).sum()) + 1e-8
        spread = linear_cross_entropy(x, w, targets, dloss)["dx" if which == 0 else "dw"][1]
        assert abs(float((grad.double() * way).sum()) - slope) <= max(bound, float((spread * way.abs()).sum()))


def test_autograd_and_master_weights():
    x, w, targets, _ = _inputs(200, 400, 128, masked=0.4)
    master = w.float().requires_grad_()
    leaf = x.clone().requires_grad_()
    loss, lse = fgs.linear_cross_entropy(leaf, master, targets, return_lse=True)
    (loss.sum() + 1e-3 * lse.square().sum()).backward()
    _, want_lse = fgs.linear_cross_entropy_fwd(x, w, targets)
    dx, dw = fgs.linear_cross_entropy_bwd(torch.ones_like(loss), x, w, targets, want_lse, 2e-3 * want_lse)
    assert torch.equal(leaf.grad, dx) and torch.equal(master.grad, dw.float())
    master.grad = None
    fgs.linear_cross_entropy(x, master, targets).mean().backward()
    assert master.grad.dtype == torch.float32


def test_graph():
    """Captured and replayed, with eager calls and other inputs between the replays."""
    T, V, K = 600, 1001, 128
    x, w, targets, dloss = _inputs(T, V, K, masked=0.3)
    def both():
        loss, lse = fgs.linear_cross_entropy_fwd(x, w, targets)
        return (loss, lse, *fgs.linear_cross_entropy_bwd(dloss, x, w, targets, lse))
    both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both()
    for seed in range(4):
        nx, nw, nt, nd = _inputs(T, V, K, seed=seed + 5, masked=0.2 * seed)
        x.copy_(nx), w.copy_(nw), targets.copy_(nt), dloss.copy_(nd)
        want = both()
        graph.replay()
        torch.cuda.synchronize()
        for one, other in zip(out, want):
            assert torch.equal(one, other)


def test_another_stream():
    x, w, targets, dloss = _inputs(300, 700, 128)
    want = _compare(x, w, targets, dloss)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        loss, lse = fgs.linear_cross_entropy_fwd(x, w, targets)
        dx, dw = fgs.linear_cross_entropy_bwd(dloss, x, w, targets, lse)
    side.synchronize()
    for one, other in zip(want, (loss, lse, dx, dw)):
        assert torch.equal(one, other)
