"""The operators at the two ends of a language model and inside its MLP, as
cases that can be timed and checked: token embedding with its gradient, the
output head with softmax cross entropy over the vocabulary (the logits are
not kept) with its gradients, and SwiGLU with its input kept in 8 bits for
the backward pass.

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
IGNORED = -100


# --------------------------------------------------------------------------
# the cases
# --------------------------------------------------------------------------

def listed():
    return [
        # the likelihoods of a few tokens on a small model: latency, and one read of the head's weight
        dict(name="loss score 5", op="loss", way="forward", tokens=5, vocab=32003, width=512, masked=0.0,
             weights="mean"),
        # an evaluation batch of odd sizes
        dict(name="loss evaluate 4099", op="loss", way="forward", tokens=4099, vocab=50021, width=2048, masked=0.0,
             weights="mean"),
        # a small model's training step
        dict(name="loss train small", op="loss", way="train", tokens=1024, vocab=32000, width=512, masked=0.0,
             weights="mean"),
        # a training step's micro-batch, every token a target
        dict(name="loss train 8192", op="loss", way="train", tokens=8192, vocab=128000, width=4096, masked=0.0,
             weights="mean"),
        # fine-tuning: the prompts' tokens are no targets, an odd vocabulary, a weight for each token
        dict(name="loss train masked", op="loss", way="train", tokens=6143, vocab=100003, width=7168, masked=0.6,
             weights="token"),
        # one new token for each of a few requests: latency
        dict(name="embedding step 7", op="embedding", way="forward", tokens=7, vocab=128000, width=4096,
             weight="bf16", out="bf16", scale=1.0, padded=0.0),
        # the first layer of a micro-batch: FP32 master rows, scaled, into an FP32 residual stream
        dict(name="embedding forward", op="embedding", way="forward", tokens=16381, vocab=100003, width=7168,
             weight="fp32", out="fp32", scale=64.0, padded=0.0),
        # the gradient of a training step's micro-batch: a few thousand rows among many that stay zero
        dict(name="embedding gradient", op="embedding", way="backward", tokens=8192, vocab=128000, width=4096,
             weight="fp32", out="bf16", scale=1.0, padded=0.0),
        # batches padded to one length: most positions hold the same token
        dict(name="embedding gradient padded", op="embedding", way="backward", tokens=61440, vocab=32003, width=1024,
             weight="bf16", out="fp32", scale=32.0, padded=0.7),
        # the MLP of a few new tokens, nothing to keep: latency
        dict(name="swiglu step 7", op="swiglu", way="forward", tokens=7, inter=2048),
        # a training step's micro-batch, forward and backward over the kept codes
        dict(name="swiglu train", op="swiglu", way="train", tokens=8192, inter=14336),
        # odd tokens and a last tile that is not whole
        dict(name="swiglu train odd", op="swiglu", way="train", tokens=4111, inter=5464),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["loss", "embedding", "swiglu"])
    if op == "loss":
        width = 64 * _log(rng, 4, 112)
        vocab = _log(rng, 1000, 128000)
        tokens = _log(rng, 1, min(8192, 8192 * 128000 * 4096 // (width * vocab)))
        return dict(op=op, way=rng.choice(["forward", "train"]), tokens=tokens, vocab=vocab, width=width,
                    masked=rng.choice([0.0, 0.0, 0.3, 0.9]), weights=rng.choice(["mean", "mean", "token"]))
    if op == "embedding":
        width = 8 * _log(rng, 8, 1024)
        vocab = _log(rng, 1000, min(128000, 128000 * 4096 // width))
        return dict(op=op, way=rng.choice(["forward", "backward"]), tokens=_log(rng, 1, min(65536, 2 ** 27 // width)),
                    vocab=vocab, width=width, weight=rng.choice(["bf16", "fp32"]), out=rng.choice(["bf16", "fp32"]),
                    scale=rng.choice([1.0, 0.5, 45.25]), padded=rng.choice([0.0, 0.0, 0.5]))
    inter = 8 * _log(rng, 8, 2048)
    return dict(op=op, way=rng.choice(["forward", "train", "train"]), tokens=_log(rng, 1, min(16384, 2 ** 26 // inter)),
                inter=inter)


def _targets_masked(case):
    """Which tokens are no targets: the first `masked` of every document."""
    T, rng = case["tokens"], random.Random(case["tokens"] * 1009)
    masked, at = [False] * T, 0
    while at < T and case["masked"]:
        n = min(T - at, int(math.exp(rng.uniform(3.0, 7.0))))
        prompt = int(n * case["masked"])
        masked[at:at + prompt] = [True] * prompt
        at += n
    return masked


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

def _inputs(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape, std=1.0, mean=0.0, dtype=torch.float32):
        x = torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)
        return x.mul_(std).add_(mean).to(dtype)

    def uniform(*shape):
        return torch.rand(*shape, generator=gen, device="cuda")

    def words(count, vocab):
        """Tokens as text has them: the r-th most frequent one about 1 / r as often as the first."""
        rank = (uniform(count).double() * math.log(vocab)).exp_().long().sub_(1).clamp_(0, vocab - 1)
        step = next(s for s in range(7919, 8999) if math.gcd(s, vocab) == 1)      # frequent ones anywhere in the list
        return rank * step % vocab

    s = dict(case)
    bf16 = torch.bfloat16
    if case["op"] == "loss":
        T, V, K = case["tokens"], case["vocab"], case["width"]
        s["w"] = normal(V, K, std=1.5 * K ** -0.5, dtype=bf16)
        targets = words(T, V)
        # the last norm's output; the model knows some of the targets well and some not at all
        s["x"] = (normal(T, K) + s["w"][targets].float() * (6.0 * uniform(T, 1))).to(bf16)
        masked = torch.tensor(_targets_masked(case), device="cuda")
        s["targets"] = torch.where(masked, IGNORED, targets)
        if case["way"] == "train":
            share = 1.0 / max(1, T - sum(_targets_masked(case)))      # the mean over the targets
            s["dloss"] = torch.full((T,), share, device="cuda")
            if case["weights"] == "token":
                s["dloss"] *= 0.25 + uniform(T)
    elif case["op"] == "embedding":
        T, V, W = case["tokens"], case["vocab"], case["width"]
        s["tokens"] = words(T, V)
        if case["padded"]:
            s["tokens"] = torch.where(uniform(T) < case["padded"], 0, s["tokens"])
        if case["way"] == "forward":
            s["weight"] = normal(V, W, std=0.02, dtype=DTYPES[case["weight"]])
        else:
            s["dout"] = normal(T, W, std=1e-2, dtype=DTYPES[case["out"]])
    else:
        T, I = case["tokens"], case["inter"]
        s["gate_up"] = normal(T, 2 * I, dtype=bf16)
        s["gate_up"][:, ::977] *= 20         # a few channels stand out, as they do in trained models
        if case["way"] == "train":
            s["dh"] = normal(T, I, std=1e-2, dtype=bf16)
    return s


def prepare(case, seed):
    return _inputs(case, seed)


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------

def run(s):
    if s["op"] == "loss":
        return _loss_own(s) if own else _loss_plain(s)
    if s["op"] == "embedding":
        return _embedding_own(s) if own else _embedding_plain(s)
    return _swiglu_own(s) if own else _swiglu_plain(s)


def _loss_own(s):
    import fine_grained_scaled_amd as fgs
    loss, lse = fgs.linear_cross_entropy_fwd(s["x"], s["w"], s["targets"])
    if s["way"] == "forward":
        return {"loss": loss, "lse": lse}
    dx, dw = fgs.linear_cross_entropy_bwd(s["dloss"], s["x"], s["w"], s["targets"], lse)
    return {"loss": loss, "lse": lse, "dx": dx, "dw": dw}


def _embedding_own(s):
    import fine_grained_scaled_amd as fgs
    if s["way"] == "forward":
        return fgs.embedding_fwd(s["tokens"], s["weight"], scale=s["scale"], out_dtype=DTYPES[s["out"]])
    return fgs.embedding_bwd(s["dout"], s["tokens"], s["vocab"], scale=s["scale"], dtype=DTYPES[s["weight"]])


def _swiglu_own(s):
    import fine_grained_scaled_amd as fgs
    if s["way"] == "forward":
        return fgs.swiglu_fwd(s["gate_up"], checkpoint=False)[0]
    h, kept = fgs.swiglu_fwd(s["gate_up"])
    return {"h": h, "dgate_up": fgs.swiglu_bwd(s["dh"], kept)}


def _loss_plain(s):
    """z = x w^T, lse = log sum exp z, loss = lse - z[target]; dz = dloss (softmax(z) - onehot), dx = dz w,
    dw = dz^T x. Tokens without a target have loss and lse 0 and no gradient."""
    x, w, targets = s["x"].float(), s["w"].float(), s["targets"]
    some = targets >= 0
    at = torch.where(some, targets, 0)[:, None]
    z = x @ w.t()
    top = z.amax(1, keepdim=True)
    picked = z.gather(1, at)
    p = z.sub_(top).exp_()
    total = p.sum(1, keepdim=True)
    lse = top + total.log()
    got = {"loss": torch.where(some, (lse - picked).squeeze(1), 0.0), "lse": torch.where(some, lse.squeeze(1), 0.0)}
    if s["way"] == "forward":
        return got
    p.div_(total).scatter_add_(1, at, torch.full_like(total, -1.0))
    p.mul_(torch.where(some, s["dloss"], 0.0)[:, None])
    return got | {"dx": (p @ w).to(s["x"].dtype), "dw": (p.t() @ x).to(s["w"].dtype)}


def _embedding_plain(s):
    """out[t] = scale weight[tokens[t]]; dweight[v] = scale times the sum of dout[t] over the t with tokens[t] = v."""
    if s["way"] == "forward":
        return (s["weight"][s["tokens"]].float() * s["scale"]).to(DTYPES[s["out"]])
    dw = torch.zeros(s["vocab"], s["width"], device="cuda")
    return dw.index_add_(0, s["tokens"], s["dout"].float()).mul_(s["scale"]).to(DTYPES[s["weight"]])


def _kept(x):
    """x [T, I] as it is kept in 8 bits: tiles of 128 along the row, scale = amax / 448, E4M3 codes of x / scale;
    the quotient is formed in 64 bits and rounded to 32, which is the 32-bit division's result."""
    T, I = x.shape
    tiles = torch.nn.functional.pad(x, (0, -I % 128)).view(T, -1, 128)
    scale = (tiles.abs().amax(2, keepdim=True).double() / 448.0).float()
    scale = torch.where(scale == 0, 1.0, scale)
    codes = (tiles.double() / scale.double()).float().to(torch.float8_e4m3fn)
    return (codes.float() * scale).view(T, -1)[:, :I]


def _swiglu_plain(s):
    """h = g sigmoid(g) u; dg = dh u sigmoid(g) (1 + g (1 - sigmoid(g))), du = dh g sigmoid(g) at the kept g and u."""
    g, u = s["gate_up"].float().chunk(2, 1)
    h = (g * torch.sigmoid(g) * u).to(torch.bfloat16)
    if s["way"] == "forward":
        return h
    g, u, dh = _kept(g), _kept(u), s["dh"].float()
    sig = torch.sigmoid(g)
    dg = dh * u * sig * (1.0 + g * (1.0 - sig))
    return {"h": h, "dgate_up": torch.cat([dg, dh * g * sig], 1).to(torch.bfloat16)}


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------

def work(case):
    T = case["tokens"]
    if case["op"] == "loss":
        V, K = case["vocab"], case["width"]
        active = T - sum(_targets_masked(case))
        if case["way"] == "forward":      # x, w and targets in, loss and lse out; the product x w^T
            return {"bytes": 2 * (active + V) * K + 16 * T, "flops": 2 * active * V * K}
        # and the gradients' two products; dloss in, dx and dw out
        return {"bytes": 2 * (active + V) * K + 20 * T + 2 * (T + V) * K, "flops": 6 * active * V * K}
    if case["op"] == "embedding":
        V, W = case["vocab"], case["width"]
        weight, out = (2 if case[k] == "bf16" else 4 for k in ("weight", "out"))
        if case["way"] == "forward":
            return {"bytes": T * (8 + W * (weight + out)), "flops": T * W}
        return {"bytes": T * (8 + W * out) + V * W * weight, "flops": 2 * T * W}
    I = case["inter"]
    if case["way"] == "forward":
        return {"bytes": 6 * T * I, "flops": 6 * T * I}
    # the codes of both halves out and in again, their scales with them
    return {"bytes": T * I * (4 + 2 + 2 + 2 + 2 + 4) + 16 * T * -(-I // 128), "flops": 24 * T * I}


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------

def _e4m3(v):
    """v (64 bits, at most 448) rounded to the nearest E4M3 value, ties to even."""
    exponent = torch.frexp(v)[1].clamp(min=-5) - 1
    step = torch.ldexp(torch.ones_like(v), exponent - 3)
    return torch.round(v / step) * step


def exact(case, seed):
    s = _inputs(case, seed)
    f64 = torch.float64
    T = case["tokens"]
    if case["op"] == "loss":
        w = s["w"].to(f64)
        got = {"loss": torch.zeros(T, dtype=f64, device="cuda"), "lse": torch.zeros(T, dtype=f64, device="cuda")}
        if case["way"] == "train":
            got["dx"] = torch.zeros(T, case["width"], dtype=f64, device="cuda")
            got["dw"] = torch.zeros_like(w)
        rows = torch.nonzero(s["targets"] >= 0).squeeze(1)
        for r in rows.split(1024):
            x, target = s["x"][r].to(f64), s["targets"][r]
            z = torch.matmul(x, w.t())
            lse = torch.logsumexp(z, 1)
            mine = torch.arange(len(r), device="cuda")
            got["lse"][r] = lse
            got["loss"][r] = lse - z[mine, target]
            if case["way"] == "train":
                dz = torch.exp(z - lse[:, None])
                dz[mine, target] -= 1.0
                dz *= s["dloss"][r].to(f64)[:, None]
                got["dx"][r] = torch.matmul(dz, w)
                got["dw"] += torch.matmul(dz.t(), x)
        return got
    if case["op"] == "embedding":
        if case["way"] == "forward":
            return torch.index_select(s["weight"], 0, s["tokens"]).to(f64) * case["scale"]
        order = torch.argsort(s["tokens"], stable=True)
        ids, counts = torch.unique_consecutive(s["tokens"][order], return_counts=True)
        sums = torch.segment_reduce(s["dout"][order].to(f64), "sum", lengths=counts, axis=0)
        got = torch.zeros(case["vocab"], case["width"], dtype=f64, device="cuda")
        got[ids] = sums * case["scale"]
        return got
    I = case["inter"]

    def swish(t):
        return t / (1.0 + torch.exp(-t))

    gate, up = s["gate_up"][:, :I].to(f64), s["gate_up"][:, I:].to(f64)
    h = swish(gate) * up
    if case["way"] == "forward":
        return h
    for half in (gate, up):      # in place: the values that the codes stand for
        for tile in half.split(128, 1):
            scale = (tile.abs().max(1, keepdim=True).values / 448.0).float().to(f64)     # kept in 32 bits
            scale[scale == 0.0] = 1.0
            tile.copy_(_e4m3((tile / scale).float().to(f64)) * scale)      # codes of the 32-bit quotient
    dh = s["dh"].to(f64)
    z = torch.exp(-gate)
    slope = (1.0 + z + gate * z) / (1.0 + z) ** 2
    return {"h": h, "dgate_up": torch.cat([dh * up * slope, dh * swish(gate)], 1)}
