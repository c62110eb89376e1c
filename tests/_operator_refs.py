"""The transformer operators in 64 bits on the CPU, written out from their
definitions, with error bounds for an implementation that keeps scores,
statistics and sums in 32 bits and rounds to BF16 where the header says so.

u = 2^-8 is half a BF16 step relative to the value, e = 2^-24 half an FP32
step.  A sum of n FP32 terms is off by at most n e times the sum of their
magnitudes."""
import math

import torch

U = 2.0 ** -8
E = 2.0 ** -24
F64 = torch.float64


def pack_offsets(lengths, before=0):
    return torch.tensor([before] + lengths, dtype=torch.int64).cumsum(0).to(torch.int32)


def attention(q, k, v, cu, scale, dout=None):
    """dict of name -> (value, bound), CPU tensors in, float64 out."""
    q, k, v = q.to(F64), k.to(F64), v.to(F64)
    T, H, D = q.shape
    G = H // k.shape[1]
    z0 = lambda like: (torch.zeros(like.shape, dtype=F64), torch.zeros(like.shape, dtype=F64))
    got = {"out": z0(q), "lse": (torch.full((H, T), -math.inf, dtype=F64), torch.zeros(H, T, dtype=F64))}
    if dout is not None:
        dout = dout.to(F64)
        got.update(dq=z0(q), dk=z0(k), dv=z0(v))
    for a, b in zip(cu[:-1].tolist(), cu[1:].tolist()):
        n = b - a
        if n <= 0:
            continue
        hidden = torch.ones(n, n, dtype=torch.bool).triu(1)
        for h in range(H):
            qh, kh, vh = q[a:b, h], k[a:b, h // G], v[a:b, h // G]
            z = (qh @ kh.T * scale).masked_fill(hidden, -math.inf)
            top = z.amax(1, keepdim=True)
            safe = torch.where(top == -math.inf, 0.0, top)
            l = torch.exp(z - safe).sum(1, keepdim=True)
            p = torch.exp(z - safe) / torch.where(l == 0, 1.0, l)
            out = p @ vh
            lse = (safe + l.log()).squeeze(1)
            # a score: D products summed in FP32, then scaled and shifted
            mag = (qh.abs() @ kh.abs().T).masked_fill(hidden, 0.0).amax(1, keepdim=True)
            ez = scale * mag * (D + 8) * E
            ep = 2 * ez + (n + 16) * 2 * E          # of a probability, relative
            sv = p @ vh.abs()
            eo = (U + ep) * sv * 1.01
            got["out"][0][a:b, h], got["out"][1][a:b, h] = out, eo + U * (out.abs() + eo) + 1e-30
            got["lse"][0][h, a:b] = lse
            finite = torch.where(lse.isfinite(), lse, 0.0).abs()
            got["lse"][1][h, a:b] = (ez + (n + 16) * 2 * E).squeeze(1) + 8 * E * (finite + safe.squeeze(1).abs() + 8)
            if dout is None:
                continue
            g = dout[a:b, h]
            delta = (g * out).sum(1, keepdim=True)
            ed = (g.abs() * got["out"][1][a:b, h]).sum(1, keepdim=True) * 1.01
            dp = g @ vh.T
            edp = (g.abs() @ vh.abs().T) * (D + 4) * E
            ep = ep + 2 * got["lse"][1][h, a:b, None]
            ds = p * (dp - delta)
            eds = (U + ep) * ds.abs() * 1.01 + p * (edp + ed + (dp.abs() + delta.abs()) * 4 * E) * (1 + U)

            def put(name, i, value, bound):
                got[name][0][a:b, i] += value
                got[name][1][a:b, i] += bound
            put("dv", h // G, p.T @ g, (U + ep.max() + n * E) * (p.T @ g.abs()) * 1.01)
            put("dq", h, scale * (ds @ kh), scale * (eds @ kh.abs() + n * E * (ds.abs() @ kh.abs())) * 1.01)
            put("dk", h // G, scale * (ds.T @ qh), scale * (eds.T @ qh.abs() + n * E * (ds.T.abs() @ qh.abs())) * 1.01)
    for name in ("dq", "dk", "dv"):                  # the one rounding of the result
        if name in got:
            value, bound = got[name]
            got[name] = (value, bound + U * (value.abs() + bound) + 1e-30)
    return got


def within(name, got, want):
    value, bound = want
    got = got.detach().cpu().to(F64)
    assert got.shape == value.shape, f"{name}: shape {tuple(got.shape)}"
    same = (got == value) | (got.isnan() & value.isnan())
    bad = ~(same | ((got - value).abs() <= bound))
    if bad.any():
        i = tuple(int(x) for x in bad.nonzero()[0])
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.numel()} outside their bound; first at {i}: "
                             f"{got[i].item()!r} for {value[i].item()!r} +- {bound[i].item()!r}")


# The FP32 row sums of the block boundary: a thread adds at most 32 terms,
# then 6 steps across the wave and at most 16 waves, so a sum is off by at most
# 64 E of its magnitudes and 1 / rms, its square root, by 40 E with the
# reciprocal square root's own error.
def _rows(t):
    return t.mean(1, keepdim=True)


def residual_norm(y, x, w_pre, w_post, gate, alpha, eps, kept):
    """r from the inputs; n from `kept`, the r that the implementation kept."""
    half = U if x.dtype == torch.bfloat16 else E
    y, x, w_pre, kept = y.to(F64), x.to(F64), w_pre.to(F64), kept.to(F64)
    g = torch.ones((), dtype=F64) if gate is None else gate.to(F64)
    z = y if w_post is None else y * (_rows(y * y) + eps).rsqrt() * w_post.to(F64)
    r = alpha * x + g * z
    tol = 52 * E * (g * z).abs() + 4 * E * (alpha * x).abs()
    n = kept * (_rows(kept * kept) + eps).rsqrt() * w_pre
    return {"r": (r, tol + half * (r.abs() + tol) + 1e-38), "n": (n, 50 * E * n.abs() + U * n.abs() * 1.001 + 1e-38)}


def residual_norm_grads(dr, dn, y, r, w_pre, w_post, gate, alpha, eps):
    half = U if r.dtype == torch.bfloat16 else E
    T = y.shape[0]
    dr, dn, y, f, w_pre = (t.to(F64) for t in (dr, dn, y, r, w_pre))
    g = torch.ones((), dtype=F64) if gate is None else gate.to(F64)
    rr = (_rows(f * f) + eps).rsqrt()
    fh, t = f * rr, dn * w_pre
    d = dr + rr * (t - fh * _rows(t * fh))
    ed = 170 * E * (dr.abs() + rr * (t.abs() + fh.abs() * _rows((t * fh).abs())))

    def rounded(value, tol, h):
        return value, tol + h * (value.abs() + tol) + 1e-38

    def summed(terms, tol):      # over the rows
        return terms.sum(0), tol.sum(0) + (T + 60) * E * terms.abs().sum(0) + 1e-38
    got = {"residual": rounded(alpha * d, abs(alpha) * ed, half), "w_pre": summed(dn * fh, torch.zeros_like(d))}
    if w_post is not None:
        ry = (_rows(y * y) + eps).rsqrt()
        yh = y * ry
        z = yh * w_post.to(F64)
    else:
        z = y
    if gate is not None:
        terms, tol = d * z, ed * z.abs() + 50 * E * (d * z).abs()
        got["gate"] = summed(terms, tol) if gate.dim() == 1 else rounded(terms, tol, U)
    dz, edz = d * g, (ed + 2 * E * d.abs()) * g.abs()
    if w_post is not None:
        got["w_post"] = summed(dz * yh, edz * yh.abs() + 50 * E * (dz * yh).abs())
        wp = w_post.to(F64)
        t = dz * wp
        et = edz * wp.abs() + 2 * E * t.abs()
        c = _rows(t * yh)
        ec = _rows(et * yh.abs()) + 170 * E * _rows((t * yh).abs())
        dz, edz = ry * (t - yh * c), ry * (et + 50 * E * t.abs() + yh.abs() * (ec + 50 * E * c.abs()))
    got["y"] = rounded(dz, edz, U)
    return got
