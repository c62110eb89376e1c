"""What the output head's bounds would notice: mistakes planted into the
definition's values exceed them (no GPU needed)."""
import pytest
import torch

from _head_refs import F64, beyond, head, inputs

SIZES = [(12, 60000, 64), (12, 600000, 64)]


@pytest.mark.parametrize("T, V, K", SIZES)
def test_a_missing_tile_of_words(T, V, K):
    x, w, targets, _ = inputs(T, V, K)
    want = head(x, w, targets)
    z = x.to(F64) @ w.to(F64).T
    z[:, 12800:12928] = -torch.inf
    lse = torch.logsumexp(z, 1)
    assert beyond(lse, want["lse"]).all() and not beyond(want["lse"][0].float(), want["lse"]).any()
    loss = lse - (want["lse"][0] - want["loss"][0])
    # (the target's own score is another one's error apart: 2e-4 of the sum is close to it at 600000 words)
    assert beyond(loss, want["loss"]).double().mean() > 0.5 and not beyond(want["loss"][0].float(), want["loss"]).any()


@pytest.mark.parametrize("T, V, K", SIZES)
@pytest.mark.parametrize("part", [0.5, 0.1])
def test_a_missing_piece_of_dx(T, V, K, part):
    """A piece of the vocabulary that is not added, or added twice."""
    x, w, targets, dloss = inputs(T, V, K)
    want = head(x, w, targets, dloss)
    first = int(V * (1 - part))
    z = x.to(F64) @ w.to(F64).T
    dz = torch.softmax(z, 1)
    dz[torch.arange(T), targets] -= 1
    piece = (dz * dloss.to(F64)[:, None])[:, first:] @ w[first:].to(F64)
    dx = want["dx"][0]
    assert beyond(dx - piece, want["dx"]).any(1).all() and beyond(dx + piece, want["dx"]).any(1).all()
    assert not beyond(dx.bfloat16(), want["dx"]).any()


@pytest.mark.parametrize("T, V, K", SIZES)
def test_scaled_dw(T, V, K):
    x, w, targets, dloss = inputs(T, V, K)
    want = head(x, w, targets, dloss)
    dw = want["dw"][0]
    assert beyond(dw * 1.05, want["dw"]).double().mean() > 0.99
    assert not beyond(dw.bfloat16(), want["dw"]).any()
    # a piece's rows of dw from the piece before it
    assert beyond(dw.roll(256, 0), want["dw"]).any(1).double().mean() > 0.99
