"""The operators at a model's two ends and inside its MLP in 64 bits, written
out from their definitions, with error bounds for an implementation that keeps
scores, statistics and sums in 32 bits and rounds to BF16 where the header says
so.

U = 2^-8 is half a BF16 step relative to the value, E = 2^-24 half an FP32
step.  A sum of n FP32 terms is off by at most n E times the sum of their
magnitudes; the matrix units may cut where they do not round, so their sums
count twice."""
import torch

U = 2.0 ** -8
E = 2.0 ** -24
F64 = torch.float64


def linear_cross_entropy(x, w, targets, dloss=None, dlse=None):
    """dict of name -> (value, bound), float64 on the inputs' device."""
    x, w = x.to(F64), w.to(F64)
    (T, K), V = x.shape, w.shape[0]
    targets = targets.long()
    rows = torch.nonzero((targets >= 0) & (targets < V)).squeeze(1)
    zero = lambda *shape: (torch.zeros(*shape, dtype=F64, device=x.device), torch.zeros(*shape, dtype=F64, device=x.device))
    got = {"loss": zero(T), "lse": zero(T)}
    if dloss is not None:
        got.update(dx=zero(T, K), dw=zero(V, K))
    if len(rows) == 0:
        return got
    xr, at = x[rows], targets[rows][:, None]
    z = xr @ w.T
    ez = 2 * K * E * (xr.abs() @ w.abs().T)
    lse = torch.logsumexp(z, 1, keepdim=True)
    p = torch.exp(z - lse)
    # of the sum of exponents, relative: a term's own error weighs as the term does; exponents of arguments d are
    # off by 4 E (d + 1), and the sum of V terms by V E
    top = z.amax(1, keepdim=True)
    el = (p * (ez + 4 * E * (top - z + 1))).sum(1, keepdim=True) + (V + 64) * 2 * E
    zt, ezt = z.gather(1, at), ez.gather(1, at)
    elog = 4 * E * (lse.abs() + top.abs() + 2)
    got["lse"][0][rows], got["lse"][1][rows] = lse.squeeze(1), (el + elog).squeeze(1)
    got["loss"][0][rows] = (lse - zt).squeeze(1)
    got["loss"][1][rows] = (el + ezt + elog + 4 * E * zt.abs()).squeeze(1)
    if dloss is None:
        return got
    b = dloss.to(F64)[rows][:, None]
    e = dlse.to(F64)[rows][:, None] if dlse is not None else torch.zeros_like(b)
    ep = ez + got["lse"][1][rows][:, None] + 4 * E * (z.abs() + lse.abs() + (z - lse).abs() + 4)      # of p, relative
    dz = (b + e) * p
    edz = (b.abs() + e.abs()) * p * (ep + 8 * E) * 1.01
    dz.scatter_add_(1, at, -b)
    edz.scatter_add_(1, at, 8 * E * b.abs())
    edz = edz + U * (dz.abs() + edz)
    dx = dz @ w
    edx = edz @ w.abs() + 2 * (V + 16) * E * (dz.abs() @ w.abs())
    dw = dz.T @ xr
    edw = edz.T @ xr.abs() + 2 * (len(rows) + 16) * E * (dz.abs().T @ xr.abs())
    got["dx"][0][rows], got["dx"][1][rows] = dx, edx * 1.01 + U * (dx.abs() + edx)
    got["dw"][0][:], got["dw"][1][:] = dw, edw * 1.01 + U * (dw.abs() + edw)
    return got


def check(name, got, want):
    """Every value of `got` within its bound of the definition's."""
    value, bound = want
    assert got.shape == value.shape, name
    off = (got.to(F64) - value).abs()
    bad = ~(off <= bound + 1e-37)
    assert not bad.any(), f"{name}: {int(bad.sum())} values off, the worst {float((off / (bound + 1e-37)).max()):.3g} bounds"
