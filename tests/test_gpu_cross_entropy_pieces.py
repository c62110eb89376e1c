"""The output head's backward pass over several pieces of the vocabulary, within
bounds that a missing tile or piece exceeds."""
import os
import re

import pytest
import torch

import fine_grained_scaled_amd as fgs
from _head_refs import beyond, head, inputs

pytestmark = pytest.mark.gpu

SOURCE = os.path.join(os.path.dirname(os.path.abspath(fgs.__file__)), "csrc", "cross_entropy.hip")


def _pieces(T, V, rows):
    """Pieces of the vocabulary that hold words, of `rows` targets among T tokens."""
    text = open(SOURCE).read()
    values, least = re.search(r"PIECE_VALUES = \(int64_t\)1 << (\d+), PIECE_LEAST = (\d+);", text).groups()
    up = lambda n: -(-n // 256) * 256
    room = min(up(T) * up(V), max(1 << int(values), up(T) * int(least)))
    width = min(room // up(rows) // 256 * 256, up(V))
    return -(-V // width)


def _check(T, V, K, hidden=None, dlse=None, seed=0):
    x, w, targets, dloss = inputs(T, V, K, seed, "cuda")
    given = targets.clone()
    if hidden is not None:
        given[hidden] = -100
    keep = given >= 0
    loss, lse = fgs.linear_cross_entropy_fwd(x, w, given)
    dx, dw = fgs.linear_cross_entropy_bwd(dloss, x, w, given, lse, dlse)
    want = head(x[keep], w, targets[keep], dloss[keep], None if dlse is None else dlse[keep])
    for name, got in (("loss", loss[keep]), ("lse", lse[keep]), ("dx", dx[keep]), ("dw", dw)):
        assert not beyond(got, want[name]).any(), name
    assert not dx[~keep].any() and not loss[~keep].any() and not lse[~keep].any()
    again = fgs.linear_cross_entropy_bwd(dloss, x, w, given, lse, dlse)
    assert torch.equal(dx, again[0]) and torch.equal(dw, again[1])
    return int(keep.sum())


# two pieces with a narrow last one, three, a last tile of half the rows, the tile of up to 128 tokens
@pytest.mark.parametrize("T, V, K", [(8200, 17001, 64), (16000, 9000, 128), (8200, 40001, 64), (300, 300001, 64),
                                     (17, 600000, 64)])
def test_several_pieces(T, V, K):
    assert _pieces(T, V, T) > 1
    _check(T, V, K)


@pytest.mark.parametrize("T, V, K", [(8200, 40001, 64), (300, 300001, 64)])
def test_several_pieces_and_the_gradient_of_lse(T, V, K):
    assert _pieces(T, V, T) > 1
    dlse = torch.randn(T, generator=torch.Generator().manual_seed(1)).cuda() / T
    _check(T, V, K, dlse=dlse)


def test_several_pieces_of_fewer_than_planned():
    """A third of the rows masked: wider pieces than for all of them, and still more than one."""
    T, V, K = 8200, 40001, 64
    hidden = torch.rand(T, generator=torch.Generator().manual_seed(2)) < 0.3
    rows = _check(T, V, K, hidden.cuda())
    assert 1 < _pieces(T, V, rows) < _pieces(T, V, T)


def test_wide_heads():
    """Several tiles of dx and dw along the width, in several pieces."""
    T, V, K = 8200, 17001, 320
    assert _pieces(T, V, T) > 1
    _check(T, V, K)


@pytest.mark.parametrize("T, V, K", [(5, 1000, 64), (128, 5003, 256), (129, 5003, 256), (257, 1000, 576), (700, 129, 128)])
def test_one_piece(T, V, K):
    assert _pieces(T, V, T) == 1
    _check(T, V, K)


@pytest.mark.parametrize("T", [70, 300])
@pytest.mark.parametrize("size", [2.0 ** -126, 1e-38, 3e-39])
def test_gradients_of_the_smallest_dloss(T, size):
    """Down to FP32's subnormal numbers: the gradients are those of dloss 1 times it, to BF16's smallest step."""
    x, w, targets, _ = inputs(T, 200, 64, device="cuda")
    dloss = torch.full((T,), size, device="cuda")
    assert dloss.all()
    _, lse = fgs.linear_cross_entropy_fwd(x, w, targets)
    one = fgs.linear_cross_entropy_bwd(torch.ones_like(dloss), x, w, targets, lse)
    for got, unit in zip(fgs.linear_cross_entropy_bwd(dloss, x, w, targets, lse), one):
        want = unit.double() * float(dloss[0].double())
        # both are rounded to BF16 (the second one to steps of 2^-133 at least), after a product rounded to steps of 2^-149
        assert ((got.double() - want).abs() <= 2.02 * 2.0 ** -8 * want.abs() + 2.0 ** -133).all()
        some = want.abs() > 2.0 ** -132
        assert some.double().mean() > 0.2 and got[some].all()


@pytest.mark.parametrize("T", [3, 150])
def test_offsets_past_two_to_the_31(T):
    """w and dw of more than 2^31 values; x has 64 that are not zero, so that the scores' bounds stay small."""
    V, K = 140003, 16384
    g = torch.Generator(device="cuda").manual_seed(T)
    w = torch.empty(V, K, device="cuda", dtype=torch.bfloat16)
    for part in w.split(20000):
        part.copy_(torch.randn(part.shape, generator=g, device="cuda").abs() * 1.5 / 8)
    some = torch.cat([torch.randperm(K - 1, generator=g, device="cuda")[:63], torch.tensor([K - 1], device="cuda")])
    x = torch.zeros(T, K, device="cuda", dtype=torch.bfloat16)
    x[:, some] = torch.randn(T, 64, generator=g, device="cuda").abs().bfloat16()
    targets = torch.randint(V - 2000, V, (T,), generator=g, device="cuda")
    dloss = (0.5 + torch.rand(T, generator=g, device="cuda")) / T
    loss, lse = fgs.linear_cross_entropy_fwd(x, w, targets)
    dx, dw = fgs.linear_cross_entropy_bwd(dloss, x, w, targets, lse)
    for words in (slice(0, 300), slice(2 ** 31 // K - 300, 2 ** 31 // K + 300), slice(V - 2300, V)):
        want = head(x, w, targets, dloss, words=words)
        for name, got in (("loss", loss), ("lse", lse), ("dx", dx), ("dw", dw[words])):
            assert not beyond(got, want[name]).any(), name
    # whatever is not looked at: words that are no target have gradients of one sign in those columns, none elsewhere
    assert (dw[:V - 2000][:, some] >= 0).all() and int((dw != 0).any(0).sum()) <= 64
    torch.cuda.empty_cache()
