"""The global gradient norm and clipping against 64-bit sums.  The norm is an
FP32 rounding of an FP64 sum; an output is off by the factor's rounding, the
product's and, in BF16, the result's."""
import pytest
import torch

import fine_grained_scaled_amd as fgs
from _operator_refs import E, U, within

pytestmark = pytest.mark.gpu


def _grads(sizes, dtypes, std=1e-3, seed=0, offset=0):
    """Views of one buffer for each type, `offset` values into it."""
    g = torch.Generator().manual_seed(seed)
    got = []
    flats = {}
    for i, n in enumerate(sizes):
        flats.setdefault(dtypes[i % len(dtypes)], []).append((i, n))
    got = [None] * len(sizes)
    for kind, items in flats.items():
        flat = (torch.randn(offset + sum(n for _, n in items), generator=g) * std).to(kind).cuda()
        at = offset
        for i, n in items:
            got[i] = flat[at:at + n]
            at += n
    return got


def _check(grads, max_norm, out=None):
    before = [g.cpu() for g in grads]
    total = sum((g.double() ** 2).sum() for g in before) if before else torch.zeros((), dtype=torch.float64)
    norm = torch.as_tensor(total, dtype=torch.float64).sqrt()
    c = max_norm / norm if norm > max_norm else torch.ones((), dtype=torch.float64)
    got = fgs.clip_grad_norm(grads, max_norm, out=out)
    assert got.shape == () and got.dtype == torch.float32
    within("norm", got, (norm, 2 * E * norm))
    for i, (g, o) in enumerate(zip(before, grads if out is None else out)):
        want = g.double() * c
        if norm <= max_norm:
            assert torch.equal(o.cpu(), g)
        half, least = (U, 2.0 ** -134) if g.dtype == torch.bfloat16 else (E, 2.0 ** -149)
        within(f"out {i}", o, (want, want.abs() * (half + 4 * E) + least))
    if out is not None:
        assert all(torch.equal(a, b.cpu()) for a, b in zip(before, grads))


SIZES = [1, 0, 3, 17, 4096, 8193, 70001, 2, 5, 1023]


@pytest.mark.parametrize("dtypes", [[torch.float32], [torch.bfloat16], [torch.float32, torch.bfloat16]], ids=str)
@pytest.mark.parametrize("offset", [0, 1, 3])
@pytest.mark.parametrize("max_norm", [1e-3, 1e3])
def test_sizes_and_places(dtypes, offset, max_norm):
    _check(_grads(SIZES, dtypes, offset=offset), max_norm)


@pytest.mark.parametrize("shift", [0, 1, 2, 7])
def test_into_other_tensors_of_another_alignment(shift):
    kinds = [torch.float32, torch.bfloat16]
    grads = _grads(SIZES, kinds, seed=1, offset=1)
    out = [torch.full((n + shift,), 9.0, dtype=kinds[i % 2], device="cuda")[shift:] for i, n in enumerate(SIZES)]
    _check(grads, 0.01, out)
    _check(grads, torch.inf, out)


def test_writes_nothing_beside_its_tensors():
    flat = torch.full((1000,), 2.0, dtype=torch.bfloat16, device="cuda")
    _check([flat[3:500], flat[503:998]], 1.0)
    keep = torch.tensor([0, 1, 2, 500, 501, 502, 998, 999])
    assert (flat.cpu()[keep] == 2.0).all()


def test_more_tensors_than_a_launch_takes():
    _check(_grads([(i * 37) % 400 for i in range(300)], [torch.float32, torch.bfloat16], seed=2), 0.05)
    _check(_grads([0] * 130 + [5], [torch.float32], seed=2), 0.05)


def test_large():
    """Past 64 MiB in all, the larger chunks; one tensor among small ones."""
    _check(_grads([11, 40_000_003, 29, 1_000_000], [torch.float32, torch.float32, torch.bfloat16], seed=3), 1.0)


@pytest.mark.parametrize("gain", [1e-30, 1e30])
def test_values_whose_squares_leave_fp32(gain):
    _check(_grads([1000, 33], [torch.float32, torch.bfloat16], std=gain, seed=4), gain)


def test_zeros_nothing_and_zero_norm():
    _check([torch.zeros(100, device="cuda")], 1.0)
    _check([torch.zeros(100, device="cuda")], 0.0)
    _check(_grads([50], [torch.float32]), 0.0)
    assert float(fgs.clip_grad_norm([], 1.0)) == 0.0
    assert float(fgs.clip_grad_norm([torch.zeros(0, device="cuda")], 1.0)) == 0.0


def test_non_finite():
    g = _grads([100, 40], [torch.float32, torch.bfloat16], seed=5)
    g[1][3] = torch.inf
    norm = fgs.clip_grad_norm(g, 1.0)
    assert norm == torch.inf and not g[0].any()
    assert g[1][3].isnan() and not torch.cat([g[1][:3], g[1][4:]]).any()
    g = _grads([100, 40], [torch.float32, torch.bfloat16], seed=5)
    g[0][99] = torch.nan
    assert fgs.clip_grad_norm(g, 1.0).isnan() and g[0].isnan().all() and g[1].isnan().all()


def test_same_bits_and_graph_replays():
    g = _grads([200_000, 31, 4097], [torch.float32, torch.bfloat16], seed=6)
    out, ref = [torch.empty_like(x) for x in g], [torch.empty_like(x) for x in g]
    a = fgs.clip_grad_norm(g, 0.1, out=ref)
    b = fgs.clip_grad_norm(g, 0.1, out=out)
    assert torch.equal(a, b) and all(torch.equal(x, y) for x, y in zip(out, ref))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = fgs.clip_grad_norm(g, 0.1, out=out)
    for gain in (1.0, 3.0, 1e-3):
        g[0].mul_(gain)
        want = fgs.clip_grad_norm(g, 0.1, out=ref)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(norm, want) and all(torch.equal(x, y) for x, y in zip(out, ref))
