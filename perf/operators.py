"""The operators around the library's linear layers, as cases that can be
timed and checked: causal attention over packed sequences, the block boundary
(norm of the block's output, gate, residual scale, norm for the next block),
and the global gradient norm with clipping.

listed() and draw() give cases, prepare() makes a case's inputs on the GPU
from a seed, run() is one pass (in plain torch operations, or with own = True
through the library's entry points), work() the bytes and operations that the
pass cannot do without, exact() the definition in 64 bits.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# --------------------------------------------------------------------------
# the cases
# --------------------------------------------------------------------------

def listed():
    return [
        # one short prompt on a small model: nothing but latency
        dict(name="attention prompt 37", op="attention", way="forward", tokens=37, seqs=1, heads=8, kv_heads=2,
             dim=128, fused=False),
        # requests of a serving step, prompts of very different lengths in one pack
        dict(name="attention prompts 61", op="attention", way="forward", tokens=6143, seqs=61, heads=32, kv_heads=8,
             dim=128, fused=True),
        # one long document read in whole
        dict(name="attention prompt 16384", op="attention", way="forward", tokens=16384, seqs=1, heads=16, kv_heads=2,
             dim=128, fused=True),
        # a training step's micro-batch: documents packed to 8192 tokens
        dict(name="attention train packed", op="attention", way="train", tokens=8192, seqs=7, heads=32, kv_heads=8,
             dim=128, fused=True),
        # the same tokens as one document
        dict(name="attention train 8192", op="attention", way="train", tokens=8192, seqs=1, heads=32, kv_heads=8,
             dim=128, fused=True),
        # a small model's heads of 64, one key head per query head, ragged
        dict(name="attention train 64", op="attention", way="train", tokens=4099, seqs=9, heads=16, kv_heads=16,
             dim=64, fused=False),
        # one new token per request, every option on: latency
        dict(name="norm step 7", op="norm", way="forward", tokens=7, width=4096, residual="bf16", post=True,
             gate="channel", alpha=1.0),
        # the forward pass of a wide model's micro-batch, an FP32 residual stream
        dict(name="norm forward wide", op="norm", way="forward", tokens=8192, width=16384, residual="fp32", post=True,
             gate="channel", alpha=0.5),
        # a training step's backward pass, one gate for each channel
        dict(name="norm backward channel", op="norm", way="backward", tokens=8192, width=4096, residual="bf16",
             post=True, gate="channel", alpha=1.0),
        # an odd token count and a gate for each token and channel
        dict(name="norm backward token", op="norm", way="backward", tokens=4111, width=7168, residual="fp32",
             post=True, gate="token", alpha=0.7),
        # an adapter's few small gradients
        dict(name="clip small", op="clip", tensors=24, values=300007, dtype="fp32", max_norm=0.25),
        # a model's gradients: FP32 weight gradients and BF16 ones beside them, large and tiny, at odd places
        dict(name="clip model", op="clip", tensors=290, values=420000013, dtype="mixed", max_norm=1.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attention", "norm", "clip"])
    if op == "attention":
        way = rng.choice(["forward", "train"])
        kv = rng.choice([1, 2, 4, 8])
        heads = kv * rng.choice([1, 2, 3, 4, 5, 8])
        while heads > 32:
            heads = kv * rng.choice([1, 2, 3, 4])
        return dict(op=op, way=way, tokens=_log(rng, 1, 8192), seqs=_log(rng, 1, 64), heads=heads, kv_heads=kv,
                    dim=rng.choice([64, 128]), fused=rng.random() < 0.5)
    if op == "norm":
        width = 8 * _log(rng, 16, 2048)
        return dict(op=op, way=rng.choice(["forward", "backward"]), tokens=_log(rng, 1, min(16384, 2 ** 27 // width)),
                    width=width, residual=rng.choice(["bf16", "fp32"]), post=rng.random() < 0.7,
                    gate=rng.choice(["none", "channel", "token"]), alpha=rng.choice([1.0, 0.5, 0.7]))
    return dict(op=op, tensors=_log(rng, 1, 400), values=_log(rng, 1000, 400000000),
                dtype=rng.choice(["bf16", "fp32", "mixed"]), max_norm=rng.choice([0.01, 1.0, 1000.0]))


def _parts(total, parts, spread):
    """`total` cut into `parts` whole numbers whose sizes are spread over a
    factor of e^spread (some may be 0), the same for the same arguments."""
    rng = random.Random(total * 1009 + parts)
    w = [math.exp(rng.uniform(0.0, spread)) for _ in range(parts)]
    got = [int(total * x / sum(w)) for x in w]
    got[rng.randrange(parts)] += total - sum(got)
    return got


def _lengths(case):
    return _parts(case["tokens"], case["seqs"], 4.0)


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

def _inputs(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape, std=1.0, mean=0.0, dtype=torch.float32):
        x = torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)
        return x.mul_(std).add_(mean).to(dtype)

    s = dict(case)
    bf16 = torch.bfloat16
    if case["op"] == "attention":
        T, H, Hk, D = case["tokens"], case["heads"], case["kv_heads"], case["dim"]
        if case["fused"]:    # the output of one projection for q, k and v
            qkv = normal(T, H + 2 * Hk, D, dtype=bf16)
            s["q"], s["k"], s["v"] = qkv[:, :H], qkv[:, H:H + Hk], qkv[:, H + Hk:]
        else:
            s["q"], s["k"], s["v"] = (normal(T, h, D, dtype=bf16) for h in (H, Hk, Hk))
        lengths = _lengths(case)
        s["longest"] = max(lengths)
        s["cu"] = torch.tensor([0] + lengths, dtype=torch.int32).cumsum(0, dtype=torch.int32).cuda()
        if case["way"] == "train":
            s["do"] = normal(T, H, D, std=1e-2, dtype=bf16)
    elif case["op"] == "norm":
        T, W = case["tokens"], case["width"]
        res = DTYPES[case["residual"]]
        s["y"] = normal(T, W, std=0.5, dtype=bf16)
        s["w_post"] = normal(W, std=0.1, mean=1.0) if case["post"] else None
        s["w_pre"] = normal(W, std=0.1, mean=1.0)
        s["gate"] = {"none": None, "channel": (W,), "token": (T, W)}[case["gate"]]
        if s["gate"]:
            s["gate"] = normal(*s["gate"], std=0.3, mean=0.5, dtype=bf16 if case["gate"] == "token" else torch.float32)
        if case["way"] == "forward":
            s["x"] = normal(T, W, std=2.0, dtype=res)
        else:
            s["r"] = normal(T, W, std=2.0, dtype=res)        # what the forward pass kept: its new residual
            s["dr"] = normal(T, W, std=1e-2, dtype=res)
            s["dn"] = normal(T, W, std=1e-2, dtype=bf16)
    else:
        sizes = _parts(case["values"], case["tensors"], 9.0)
        kinds = {"bf16": [bf16], "fp32": [torch.float32], "mixed": [torch.float32, bf16]}[case["dtype"]]
        s["grads"], s["out"], s["flat"] = [], [], []
        for j, kind in enumerate(kinds):     # views of one buffer for each type, as a gradient bucket holds them
            mine = sizes[j::len(kinds)]
            flat = normal(sum(mine), std=1e-3, dtype=kind)
            to = torch.empty_like(flat)
            s["grads"] += list(flat.split(mine))
            s["out"] += list(to.split(mine))
            s["flat"].append(to)
    return s


def prepare(case, seed):
    return _inputs(case, seed)


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------

def run(s):
    if s["op"] == "attention":
        return _attention_own(s) if own else _attention_plain(s)
    if s["op"] == "norm":
        return _norm_own(s) if own else _norm_plain(s)
    return _clip_own(s) if own else _clip_plain(s)


def _attention_own(s):
    import fine_grained_scaled_amd as fgs
    out, lse = fgs.attention_fwd(s["q"], s["k"], s["v"], s["cu"])
    if s["way"] == "forward":
        return {"out": out, "lse": lse}
    dq, dk, dv = fgs.attention_bwd(s["do"], s["q"], s["k"], s["v"], out, lse, s["cu"])
    return {"out": out, "lse": lse, "dq": dq, "dk": dk, "dv": dv}


def _norm_own(s):
    import fine_grained_scaled_amd as fgs
    how = dict(w_post=s["w_post"], gate=s["gate"], alpha=s["alpha"], w_pre=s["w_pre"])
    if s["way"] == "forward":
        r, n = fgs.residual_norm_fwd(s["y"], s["x"], **how)
        return {"r": r, "n": n}
    g = fgs.residual_norm_bwd(s["dr"], s["dn"], s["y"], s["r"], **how)
    return {"dx": g.residual, "dy": g.y, "dgate": g.gate, "dw_post": g.w_post, "dw_pre": g.w_pre}


def _clip_own(s):
    import fine_grained_scaled_amd as fgs
    return {"norm": fgs.clip_grad_norm(s["grads"], s["max_norm"], out=s["out"]), "out": s["flat"]}


def _attention_plain(s):
    """softmax(q k^T / sqrt(dim)) v over the sequences padded to the longest,
    in 32 bits; the gradients by their formulas."""
    q, k, v, cu, L = s["q"], s["k"], s["v"], s["cu"].long(), s["longest"]
    T, H, D = q.shape
    G = H // k.shape[1]
    at = torch.arange(L, device=q.device)
    inside = at < (cu[1:] - cu[:-1])[:, None]                           # [sequences, L]
    place = (cu[:-1, None] + at).clamp(max=T - 1)
    token = torch.arange(T, device=q.device)
    seq = torch.searchsorted(cu[1:].contiguous(), token, right=True)
    pos = token - cu[seq]

    def padded(x, times=1):
        x = (x[place].float() * inside[:, :, None, None]).transpose(1, 2)
        return x.repeat_interleave(times, 1) if times > 1 else x.contiguous()   # [sequences, heads, L, dim]

    def packed(x):
        return x[seq, :, pos]

    def shared(x):   # the sum over the query heads that share a key head
        return x.unflatten(1, (-1, G)).sum(2)

    qp, kp, vp = padded(q), padded(k, G), padded(v, G)
    scale = D ** -0.5
    seen = (at[:, None] >= at)[None] & inside[:, None, :] & inside[:, :, None]
    seen = seen[:, None]
    z = torch.matmul(qp, kp.transpose(2, 3)).mul_(scale).masked_fill_(~seen, -math.inf)
    top = z.amax(3, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = z.sub_(top).exp_()
    total = p.sum(3, keepdim=True)
    p = p.div_(torch.where(total == 0, 1.0, total))
    o = torch.matmul(p, vp)
    got = {"out": packed(o).to(q.dtype), "lse": packed((top + total.log())).squeeze(2).t().contiguous()}
    if s["way"] == "forward":
        return got
    dop = padded(s["do"])
    dv = torch.matmul(p.transpose(2, 3), dop)
    ds = torch.matmul(dop, vp.transpose(2, 3)).sub_((dop * o).sum(3, keepdim=True)).mul_(p).mul_(scale)
    dq = torch.matmul(ds, kp)
    dk = torch.matmul(ds.transpose(2, 3), qp)
    return got | {"dq": packed(dq).to(q.dtype), "dk": packed(shared(dk)).to(q.dtype),
                  "dv": packed(shared(dv)).to(q.dtype)}


EPS = 1e-6


def _norm_plain(s):
    """r = alpha x + gate * (y / rms(y) * w_post); n = r / rms(r) * w_pre, r
    rounded to the residual's type before it is normed; the gradients by
    their formulas."""
    y, gate, alpha = s["y"].float(), s["gate"], s["alpha"]
    g = 1.0 if gate is None else gate.float()
    if s["post"]:
        ry = (y.square().mean(1, keepdim=True) + EPS).rsqrt()
        yh = y * ry
        z = yh * s["w_post"]
    else:
        z = y
    if s["way"] == "forward":
        r = (alpha * s["x"].float() + g * z).to(s["x"].dtype)
        f = r.float()
        return {"r": r, "n": (f * (f.square().mean(1, keepdim=True) + EPS).rsqrt() * s["w_pre"]).to(torch.bfloat16)}
    f, dn = s["r"].float(), s["dn"].float()
    rr = (f.square().mean(1, keepdim=True) + EPS).rsqrt()
    fh = f * rr
    t = dn * s["w_pre"]
    dr = s["dr"].float() + rr * (t - fh * (t * fh).mean(1, keepdim=True))
    got = {"dx": (alpha * dr).to(s["r"].dtype), "dw_pre": (dn * fh).sum(0), "dgate": None, "dw_post": None}
    if gate is not None:
        dg = dr * z
        got["dgate"] = dg.sum(0) if gate.dim() == 1 else dg.to(gate.dtype)
    dz = dr * g
    if s["post"]:
        got["dw_post"] = (dz * yh).sum(0)
        t = dz * s["w_post"]
        dz = ry * (t - yh * (t * yh).mean(1, keepdim=True))
    got["dy"] = dz.to(torch.bfloat16)
    return got


def _clip_plain(s):
    """norm = sqrt(sum of all squares); out = g * min(1, max_norm / norm)."""
    norm = torch.stack([g.double().square().sum() for g in s["grads"]]).sum().sqrt().float()
    c = (s["max_norm"] / norm).clamp(max=1.0)
    [o.copy_(g.float() * c) for g, o in zip(s["grads"], s["out"])]
    return {"norm": norm, "out": s["flat"]}


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------

def work(case):
    if case["op"] == "attention":
        T, H, Hk, D = case["tokens"], case["heads"], case["kv_heads"], case["dim"]
        pairs = sum(n * (n + 1) // 2 for n in _lengths(case))
        if case["way"] == "forward":     # q k^T and p v; q, k, v in, out and the row sums out
            return {"bytes": 2 * T * D * (2 * H + 2 * Hk) + 4 * T * H, "flops": 4 * D * H * pairs}
        # and the gradient's five products; the output's gradient in, three gradients out
        return {"bytes": 2 * T * D * (4 * H + 4 * Hk) + 4 * T * H, "flops": 14 * D * H * pairs}
    if case["op"] == "norm":
        T, W = case["tokens"], case["width"]
        res = 2 if case["residual"] == "bf16" else 4
        gate = {"none": 0, "channel": 4 * W, "token": 2 * T * W}[case["gate"]]
        weights = 4 * W * (2 if case["post"] else 1) + gate
        if case["way"] == "forward":
            return {"bytes": T * W * (2 + res + res + 2) + weights, "flops": 12 * T * W}
        return {"bytes": T * W * (2 + res + res + 2 + res + 2) + 2 * weights, "flops": 30 * T * W}
    size = {"bf16": 2, "fp32": 4, "mixed": 0}[case["dtype"]]
    sizes = _parts(case["values"], case["tensors"], 9.0)
    total = size * case["values"] if size else 4 * sum(sizes[0::2]) + 2 * sum(sizes[1::2])
    return {"bytes": 2 * total + 4, "flops": 3 * case["values"]}


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------

def exact(case, seed):
    s = _inputs(case, seed)
    f64 = torch.float64
    if case["op"] == "attention":
        H, D = s["q"].shape[1:]
        G = H // s["k"].shape[1]
        names = ["out"] + (["dq", "dk", "dv"] if case["way"] == "train" else [])
        got = {n: torch.zeros(s["k" if n in ("dk", "dv") else "q"].shape, dtype=f64, device="cuda") for n in names}
        got["lse"] = torch.empty(H, case["tokens"], dtype=f64, device="cuda")
        start = 0
        for n in _lengths(case):
            rows = slice(start, start + n)
            start += n
            if n == 0:
                continue
            hidden = torch.ones(n, n, dtype=torch.bool, device="cuda").triu(1)
            for h in range(H):
                q, k, v = s["q"][rows, h].to(f64), s["k"][rows, h // G].to(f64), s["v"][rows, h // G].to(f64)
                z = (q @ k.t() / math.sqrt(D)).masked_fill(hidden, -math.inf)
                lse = torch.logsumexp(z, 1)
                p = torch.exp(z - lse[:, None])
                o = p @ v
                got["lse"][h, rows], got["out"][rows, h] = lse, o
                if case["way"] == "train":
                    do = s["do"][rows, h].to(f64)
                    dz = p * (do @ v.t() - (do * o).sum(1)[:, None]) / math.sqrt(D)
                    got["dq"][rows, h] = dz @ k
                    got["dk"][rows, h // G] += dz.t() @ q
                    got["dv"][rows, h // G] += p.t() @ do
        return got
    if case["op"] == "norm":
        def rms(t):
            return torch.sqrt(torch.mean(t * t, 1, keepdim=True) + EPS)

        def norm_gradient(d, t, w):     # of d . (t / rms(t) * w): for t, and for w
            u = t / rms(t)
            return (d * w - u * torch.mean(d * w * u, 1, keepdim=True)) / rms(t), torch.sum(d * u, 0)

        y, w_pre = s["y"].to(f64), s["w_pre"].to(f64)
        gate = torch.ones((), dtype=f64, device="cuda") if s["gate"] is None else s["gate"].to(f64)
        w_post = s["w_post"].to(f64) if case["post"] else None
        z = y / rms(y) * w_post if case["post"] else y
        if case["way"] == "forward":
            r = case["alpha"] * s["x"].to(f64) + gate * z
            kept = r.to(s["x"].dtype).to(f64)       # the residual stream is kept in its type
            return {"r": r, "n": kept / rms(kept) * w_pre}
        through, dw_pre = norm_gradient(s["dn"].to(f64), s["r"].to(f64), w_pre)
        dr = s["dr"].to(f64) + through
        dgate = None
        if s["gate"] is not None:
            dgate = dr * z if s["gate"].dim() == 2 else torch.sum(dr * z, 0)
        dy, dw_post = norm_gradient(dr * gate, y, w_post) if case["post"] else (dr * gate, None)
        return {"dx": case["alpha"] * dr, "dy": dy, "dgate": dgate, "dw_post": dw_post, "dw_pre": dw_pre}
    total = torch.zeros((), dtype=f64, device="cuda")
    for g in s["grads"]:
        total += torch.dot(g.to(f64), g.to(f64))
    norm = torch.sqrt(total)
    factor = case["max_norm"] / norm if norm > case["max_norm"] else 1.0
    kinds = 2 if case["dtype"] == "mixed" else 1
    half = -(-case["tensors"] // 2) if kinds == 2 else case["tensors"]
    flats = [s["grads"][:half], s["grads"][half:]][:kinds]
    return {"norm": norm, "out": [torch.cat([g.to(f64) * factor for g in f]) if f else torch.zeros(0, dtype=f64, device="cuda")
                                  for f in flats]}
