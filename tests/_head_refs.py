"""The output head with softmax cross entropy in 64 bits, with bounds for an
implementation whose sums are as short as tiles of 128 words or more make them.

U = 2^-8 is half a BF16 step relative to the value, E = 2^-24 half an FP32 step.

Scores: the sum of n exact products, 2 n E of their magnitudes (the matrix units
may cut where they do not round; n is K, less where x is zero).  Exponents: exp2 of a product of a difference
is off by 4 E (d + 1) at a distance d.

The sum of exponents: a lane adds 32 words at most (and a half's 32: 33 roundings),
four waves join their sums (a factor of 2 E, a product, a sum each: 4 E), then the
tiles in 64 chains of ceil(tiles / 64) links and 6 levels, where both sides
have a factor and a product (7 E).

dx: V words, 16 an instruction, each rounding (2 E) once; the parts and pieces
that are added after it are fewer than the instructions that they save, or 64.
dw: the same over the rows."""
import torch

U = 2.0 ** -8
E = 2.0 ** -24
F64 = torch.float64


def chain(V):
    """Roundings of a sum of exponents over V words."""
    tiles = -(-V // 128)
    return 33 + 4 * 4 + 7 * (-(-tiles // 64) + 6)


def head(x, w, targets, dloss=None, dlse=None, words=slice(None)):
    """dict of name -> (value, bound) of the rows, all with a target inside the vocabulary; dw of those words."""
    x, w, at = x.to(F64), w.to(F64), targets.long()[:, None]
    V = w.shape[0]
    z = x @ w.T
    ez = 2 * (x != 0).sum(1, keepdim=True) * E * (x.abs() @ w.abs().T)
    top = z.amax(1, keepdim=True)
    lse = torch.logsumexp(z, 1, keepdim=True)
    p = torch.exp(z - lse)
    zt, ezt = z.gather(1, at), ez.gather(1, at)
    el = (p * (ez + 4 * E * (top - z + 1))).sum(1, keepdim=True) + chain(V) * E
    el = el + 4 * E * ((lse - top).abs() + 1)              # the logarithm
    of_lse = el + 2 * E * lse.abs()
    got = {"lse": (lse.squeeze(1), of_lse.squeeze(1)),
           "loss": ((lse - zt).squeeze(1), (el + ezt + 2 * E * ((top - zt) + (lse - zt).abs())).squeeze(1))}
    if dloss is None:
        return got
    b = dloss.to(F64)[:, None]
    e = dlse.to(F64)[:, None] if dlse is not None else torch.zeros_like(b)
    ep = ez.add_(of_lse).add_((z - lse).abs_().add_(1).mul_(4 * E))        # of p, relative
    dz = p * (b + e)
    edz = p * (b.abs() + e.abs()) * (ep + 8 * E) * 1.01
    dz.scatter_add_(1, at, -b)
    edz.scatter_add_(1, at, 8 * E * b.abs())
    edz = edz + U * (dz.abs() + edz)
    size = dz.abs()
    dx, edx = dz @ w, edz @ w.abs() + 2 * (V / 16 + 64) * E * (size @ w.abs())
    dz, edz, size = dz[:, words], edz[:, words], size[:, words]
    dw, edw = dz.T @ x, edz.T @ x.abs() + 2 * (len(x) / 16 + 64) * E * (size.T @ x.abs())
    got["dx"] = dx, 1.01 * edx + U * (dx.abs() + edx)
    got["dw"] = dw, 1.01 * edw + U * (dw.abs() + edw)
    return got


def inputs(T, V, K, seed=0, device="cpu"):
    """Inputs whose sums over the vocabulary do not cancel: what a part of it misses shows."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, K, generator=g).abs().bfloat16()
    w = (torch.randn(V, K, generator=g).abs() * 1.5 * K ** -0.5).bfloat16()
    targets = torch.randint(0, V, (T,), generator=g)
    dloss = (0.5 + torch.rand(T, generator=g)) / T
    return tuple(t.to(device) for t in (x, w, targets, dloss))


def beyond(got, want):
    """Which values of `got` are further from the definition's than their bound."""
    value, bound = want
    assert got.shape == value.shape
    return ~((got.to(F64) - value).abs() <= bound)
