"""The first rows of a sequence, which attention's backward pass keeps more
exactly than the others: rows below 64 take delta from their own p and
dout . v, and hand ds to dq as value and remainder; rows below 32 hand p and
ds to dv and dk so.  Bounds that count those roundings alone, an imitation of
the kernels in FP32 that stays within them, the same with the exactness left
out in each place, which does not, and the kernels."""
import pytest
import torch

from _operator_refs import E, F64, U, attention, pack_offsets, within

FIRST, REST = 64, 32
R = U * U * 1.01          # value and remainder, both BF16, against the whole


def bounds(q, k, v, cu, scale, dout):
    """name -> (value, bound) of dq, dk, dv as attention() gives them, with
    what the first rows' roundings leave."""
    loose = attention(q, k, v, cu, scale, dout)
    q, k, v, dout = (t.to(F64) for t in (q, k, v, dout))
    H, D = q.shape[1:]
    G = H // k.shape[1]
    got = {n: (loose[n][0], torch.zeros_like(loose[n][0])) for n in ("dq", "dk", "dv")}
    for a, b in zip(cu[:-1].tolist(), cu[1:].tolist()):
        n = b - a
        if n <= 0:
            continue
        hidden = torch.ones(n, n, dtype=torch.bool).triu(1)
        row = torch.arange(n)[:, None]
        for h in range(H):
            qh, kh, vh, g = q[a:b, h], k[a:b, h // G], v[a:b, h // G], dout[a:b, h]
            z = (qh @ kh.T * scale).masked_fill(hidden, -torch.inf)
            p = torch.softmax(z, 1)
            mag = (qh.abs() @ kh.abs().T).masked_fill(hidden, 0.0).amax(1, keepdim=True)
            ez = scale * mag * (D + 8) * E
            ep = 2 * ez + (n + 16) * 2 * E + 2 * loose["lse"][1][h, a:b, None]     # of a probability, relative
            dp = g @ vh.T
            edp = (g.abs() @ vh.abs().T) * (D + 4) * E
            delta = (p * dp).sum(1, keepdim=True)
            own = ((ep + (n + 8) * E) * p * dp.abs() + p * edp).sum(1, keepdim=True) * 1.01
            rounded = (g.abs() * loose["out"][1][a:b, h]).sum(1, keepdim=True) * 1.01
            ds = p * (dp - delta)
            e = ep * ds.abs() * 1.01 + p * (edp + torch.where(row < FIRST, own, rounded)
                                            + (dp.abs() + delta.abs()) * 4 * E) * (1 + U)
            eds = e + torch.where(row < FIRST, R, U) * (ds.abs() + e)
            got["dq"][1][a:b, h] += scale * (eds @ kh.abs() + (2 * n + 4) * E * (ds.abs() @ kh.abs())) * 1.01
            few = torch.where(row < REST, R, U)
            eds, ep = e + few * (ds.abs() + e), (ep + few * (1 + ep)) * p
            got["dk"][1][a:b, h // G] += scale * (eds.T @ qh.abs() + (2 * n * G + 4) * E * (ds.T.abs() @ qh.abs())) * 1.01
            got["dv"][1][a:b, h // G] += (ep.T @ g.abs() + (2 * n * G + 4) * E * (p.T @ g.abs())) * 1.01
    return {name: (value, bound + U * (value.abs() + bound) + 1e-30) for name, (value, bound) in got.items()}


def imitation(q, k, v, cu, scale, dout, dq_rest=1, own_delta=True, dkv_rest=1):
    """The kernels' gradients in FP32 on the CPU, the remainders counted as
    often as said."""
    q, k, v, dout = (t.float() for t in (q, k, v, dout))
    bf = lambda t: t.to(torch.bfloat16).float()
    H, G = q.shape[1], q.shape[1] // k.shape[1]
    dq, dk, dv = (torch.zeros_like(t) for t in (q, k, v))
    for a, b in zip(cu[:-1].tolist(), cu[1:].tolist()):
        n = b - a
        if n <= 0:
            continue
        hidden = torch.ones(n, n, dtype=torch.bool).triu(1)
        row = torch.arange(n)[:, None]
        for h in range(H):
            qh, kh, vh, g = q[a:b, h], k[a:b, h // G], v[a:b, h // G], dout[a:b, h]
            z = (qh @ kh.T * scale).masked_fill(hidden, -torch.inf)
            lse = torch.logsumexp(z, 1, keepdim=True)
            p = torch.exp(z - lse)
            out = bf(bf(torch.exp(z - z.amax(1, keepdim=True))) @ vh / torch.exp(z - z.amax(1, keepdim=True)).sum(1, keepdim=True))
            dp = g @ vh.T
            delta = (g * out).sum(1, keepdim=True)
            if own_delta:
                delta = torch.where(row < FIRST, (p * dp).sum(1, keepdim=True), delta)
            ds = p * (dp - delta)
            rest = lambda t, rows, times: torch.where(row < rows, times * bf(t - bf(t)), 0.0)
            dq[a:b, h] = scale * ((bf(ds) + rest(ds, FIRST, dq_rest)) @ kh)
            dk[a:b, h // G] += scale * ((bf(ds) + rest(ds, REST, dkv_rest)).T @ qh)
            dv[a:b, h // G] += (bf(p) + rest(p, REST, dkv_rest)).T @ g
    return {n: t.to(torch.bfloat16) for n, t in (("dq", dq), ("dk", dk), ("dv", dv))}


def inputs(lengths, H, Hk, D, seed):
    g = torch.Generator().manual_seed(seed)
    x = [torch.randn(sum(lengths), h, D, generator=g).to(torch.bfloat16) for h in (H, Hk, Hk, H)]
    return x[0], x[1], x[2], pack_offsets(lengths), D ** -0.5, x[3]


CASES = [([1] * 9, 2, 2, 64), ([2, 1, 3], 4, 2, 128), ([32], 2, 2, 64), ([32, 31], 4, 1, 128), ([33], 2, 1, 64), ([64, 64], 2, 2, 128),
         ([65, 1], 2, 2, 64), ([200], 3, 3, 64)]


@pytest.mark.parametrize("lengths,H,Hk,D", CASES, ids=str)
def test_imitation(lengths, H, Hk, D):
    args = inputs(lengths, H, Hk, D, seed=len(lengths))
    want = bounds(*args)
    for name, got in imitation(*args).items():
        within(name, got, want[name])


# In dk and dv the roundings of rows past 32 hide those of the first.
PLANTED = [(what, name, *case) for case in CASES if max(case[0]) >= 31
           for what, name in [(dict(dq_rest=0), "dq"), (dict(dq_rest=2), "dq"), (dict(own_delta=False), "dq"),
                              (dict(dkv_rest=0), "dk"), (dict(dkv_rest=2), "dk"), (dict(dkv_rest=0), "dv"),
                              (dict(dkv_rest=2), "dv")] if name == "dq" or max(case[0]) <= REST + 1]


@pytest.mark.parametrize("what,name,lengths,H,Hk,D", PLANTED, ids=str)
def test_imitation_without_the_exactness(what, name, lengths, H, Hk, D):
    args = inputs(lengths, H, Hk, D, seed=len(lengths))
    with pytest.raises(AssertionError, match="outside their bound"):
        within(name, imitation(*args, **what)[name], bounds(*args)[name])


@pytest.mark.gpu
@pytest.mark.parametrize("lengths,H,Hk,D", CASES + [([1] * 70 + [64] * 3, 8, 2, 128), ([31, 0, 33, 63, 65, 127], 4, 2, 64)],
                         ids=str)
def test_kernels(lengths, H, Hk, D):
    import fine_grained_scaled_amd as fgs
    args = q, k, v, cu, scale, dout = inputs(lengths, H, Hk, D, seed=len(lengths))
    want = bounds(*args)
    on = [t.cuda() for t in (q, k, v)]
    out, lse = fgs.attention_fwd(*on, cu.cuda(), scale)
    for name, got in zip(("dq", "dk", "dv"), fgs.attention_bwd(dout.cuda(), *on, out, lse, cu.cuda(), scale)):
        within(name, got, want[name])
