"""The output head where scores are large: loss, lse and gradients stay right for
every finite score.  The scores are whole numbers times a power of two that
FP32 holds exactly, so the definition's values are known."""
import math

import pytest
import torch

import fine_grained_scaled_amd as fgs
from _model_refs import E, U

pytestmark = pytest.mark.gpu

# T: the small tile, one large tile, a last tile of half the rows
TOKENS = [7, 200, 300]
V, K = 515, 64


def _apart(T, part, exponent, sign):
    """Row t scores sign part 2^exponent at its own word and one BF16 step (2^-7 of 2^exponent) less at every other."""
    x, w = torch.zeros(T, K, device="cuda"), torch.zeros(V, K, device="cuda")
    own = torch.arange(T, device="cuda") * 3 % K
    x[torch.arange(T), own] = 1.0
    top, gap = sign * part * 2.0 ** exponent, 2.0 ** (exponent - 7)
    w[:] = top - gap
    w[torch.arange(K), torch.arange(K)] = top
    assert torch.equal(w.bfloat16().float(), w)
    return x.bfloat16(), w.bfloat16(), own, top, gap


@pytest.mark.parametrize("T", TOKENS)
@pytest.mark.parametrize("exponent", [12, 16, 20, 24, 28, 31, 33, 36, 60, 100, 126])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("part", [1.3125, 1.375, 1.8125])
def test_one_score_above_the_others(T, exponent, sign, part):
    """The others are 2^5 and more below: together they have 514 e^-32 < 1e-11 of the probability, which FP32's 1 + .. loses,
    and lse is the largest score itself."""
    x, w, own, top, gap = _apart(T, part, exponent, sign)
    others = (V - 1) * math.exp(-min(gap, 700.0))
    loss, lse = fgs.linear_cross_entropy_fwd(x, w, own)
    assert loss.isfinite().all() and (loss.double().abs() <= others + 4 * E).all()
    assert torch.equal(lse.double(), torch.full_like(lse, top, dtype=torch.float64))
    # the target has all of the probability; p is off by a few E (an exponent of 0, a sum, a quotient)
    dx, dw = fgs.linear_cross_entropy_bwd(torch.ones(T, device="cuda"), x, w, own, lse)
    off = 16 * E + 2 * others
    assert dx.isfinite().all() and dw.isfinite().all()
    assert (dx.double().abs() <= 2.02 * off * abs(top) * (1 + 2.0 ** -6)).all()
    assert (dw.double().abs() <= 1.01 * off * T).all()
    # a target that has none of it: the loss is the distance, dz is 1 at the row's own word and -1 at the target
    other = own + K
    loss, lse = fgs.linear_cross_entropy_fwd(x, w, other)
    assert ((loss.double() - gap).abs() <= 4 * E * gap + others).all()
    dx, dw = fgs.linear_cross_entropy_bwd(torch.ones(T, device="cuda"), x, w, other, lse)
    count, k = torch.bincount(own, minlength=K).double(), torch.arange(K, device="cuda")
    for v, want in ((k, count), (k + K, -count)):
        assert ((dw[v, k].double() - want).abs() <= (2.02 * U + off) * count).all()


@pytest.mark.parametrize("T", TOKENS)
@pytest.mark.parametrize("top", [1.3125 * 2.0 ** 33, -1.375 * 2.0 ** 33, 1.8125 * 2.0 ** 90])
def test_all_scores_equal(T, top):
    """p = 1 / V in every word: loss log V, whatever the score (lse is the score itself, in FP32)."""
    x, w = torch.zeros(T, K, device="cuda"), torch.zeros(V, K, device="cuda")
    x[:, 0], w[:, 0] = 1.0, top
    targets = torch.arange(T, device="cuda") % V
    loss, lse = fgs.linear_cross_entropy_fwd(x.bfloat16(), w.bfloat16(), targets)
    assert ((loss.double() - math.log(V)).abs() <= 8 * E * math.log(V)).all()
    assert ((lse.double() - top).abs() <= 2 * E * abs(top)).all()


@pytest.mark.parametrize("T", TOKENS)
def test_scores_across_the_range(T):
    """Scores near both ends of FP32: finite, and the largest wins."""
    x, w = torch.zeros(T, K, device="cuda"), torch.zeros(V, K, device="cuda")
    x[:, 0] = 1.0
    w[:, 0] = -3.0e38
    w[V - 1, 0] = 3.0e38
    targets = torch.full((T,), V - 1, device="cuda")
    x, w = x.bfloat16(), w.bfloat16()
    loss, lse = fgs.linear_cross_entropy_fwd(x, w, targets)
    assert not loss.any() and torch.equal(lse, w[V - 1, 0].float().expand(T))
    dx, dw = fgs.linear_cross_entropy_bwd(torch.ones(T, device="cuda"), x, w, targets, lse)
    assert not dx.any() and not dw.any()
