"""Embedding, SwiGLU with its input kept in 8 bits and the output head together:
the example's training loop, and a small model's gradients, each operator's
against its definition at the values that it met in the run."""
import math
import os
import sys

import pytest
import torch

import fine_grained_scaled_amd as fgs
from _model_refs import E, F64, U, check, linear_cross_entropy

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "examples"))


def test_example_runs():
    import train_lm
    losses, norms = train_lm.train(steps=3, tokens=256, vocab=515, width=256, heads=4, kv_heads=2, hidden=256, layers=1,
                                   say=lambda _: None)
    assert all(math.isfinite(v) for v in losses + norms) and min(norms) > 0


def test_example_gradients():
    """The tied weight's gradient is the output head's plus the embedding's, and reruns give the same bits."""
    import train_lm
    torch.manual_seed(0)
    device = torch.device("cuda")
    model = train_lm.Model(515, 256, 4, 2, 256, 1, device)
    ids, targets, cu = train_lm.batch(515, 256, torch.Generator().manual_seed(0), device)
    grads = []
    for _ in range(2):
        model.zero_grad()
        each, embedded = model(ids, targets, cu)
        each.sum().backward()
        head = model.weight.grad.clone()
        model.add_embedding_gradient(embedded, ids)
        grads.append([p.grad.clone() for p in model.parameters()])
        d = embedded.grad.to(F64)
        add = torch.zeros(515, 256, dtype=F64, device=device).index_add_(0, ids, d) * model.scale
        size = torch.zeros(515, 256, dtype=F64, device=device).index_add_(0, ids, d.abs()) * model.scale
        count = torch.bincount(ids, minlength=515).to(F64)[:, None]
        got = model.weight.grad.to(F64)
        assert ((got - head.to(F64) - add).abs() <= (count + 4) * E * (size + head.to(F64).abs())).all()
        assert add.abs().sum() > 0 and head.abs().sum() > 0
    for a, b in zip(*grads):
        assert torch.equal(a, b)


def test_operators_together():
    T, V, K, I = 300, 701, 128, 392
    g = torch.Generator(device="cuda").manual_seed(3)
    weight = (torch.randn(V, K, generator=g, device="cuda") * K ** -0.5).requires_grad_()
    up = torch.randn(K, 2 * I, generator=g, device="cuda") * K ** -0.5
    down = torch.randn(I, K, generator=g, device="cuda") * I ** -0.5
    tokens = torch.randint(0, V, (T,), generator=g, device="cuda")
    targets = torch.where(torch.rand(T, generator=g, device="cuda") < 0.3, -100, torch.randint(0, V, (T,), generator=g, device="cuda"))
    met = {}

    def keep(name, t):
        met[name] = t.detach()
        t.register_hook(lambda d: met.__setitem__("d" + name, d.clone()))
        return t

    x = keep("x", fgs.embedding(tokens, weight, 11.25, torch.bfloat16))
    gate_up = keep("gate_up", (x.float() @ up).bfloat16())
    h = keep("h", fgs.swiglu(gate_up))
    y = keep("y", (h.float() @ down).bfloat16())
    loss = keep("loss", fgs.linear_cross_entropy(y, weight, targets))
    (loss.sum() / T).backward()

    want = linear_cross_entropy(met["y"], weight.detach().bfloat16(), targets, met["dloss"])
    check("loss", loss.detach(), want["loss"])
    check("dy", met["dy"], want["dx"])
    # the values that SwiGLU's codes stand for
    _, kept = fgs.swiglu_fwd(met["gate_up"])
    assert torch.equal(met["dgate_up"], fgs.swiglu_bwd(met["dh"], kept))
    tiles = -(-I // 128)
    scale = torch.cat([kept.scales.t()[:, i * tiles:(i + 1) * tiles].repeat_interleave(128, 1)[:, :I] for i in (0, 1)], 1)
    v = (kept.q.view(torch.float8_e4m3fn).float() * scale).to(F64)
    a, u, d = v[:, :I], v[:, I:], met["dh"].to(F64)
    s = torch.sigmoid(a)
    slope, size = 1 + a * (1 - s), 1 + a.abs() * (1 - s)
    steps = (2 * a.abs() + 24) * 2 * E
    check("dgate_up", met["dgate_up"], (torch.cat([d * u * s * slope, d * a * s], 1),
          torch.cat([U * (d * u * s * slope).abs() + steps * d.abs() * u.abs() * s * size, (U + steps) * (d * a * s).abs()], 1) * 1.01 + 1e-37))
    # the weight's gradient: both ends'
    dx = met["dx"].to(F64)
    add = torch.zeros(V, K, dtype=F64, device="cuda").index_add_(0, tokens, dx) * 11.25
    size = torch.zeros(V, K, dtype=F64, device="cuda").index_add_(0, tokens, dx.abs()) * 11.25
    count = torch.bincount(tokens, minlength=V).to(F64)[:, None]
    value, bound = want["dw"]
    check("dweight", weight.grad, (value + add, bound + (count + 4) * E * (size + value.abs() + bound)))
