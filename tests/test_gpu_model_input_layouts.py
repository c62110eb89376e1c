"""The autograd forms on inputs that are no dense tensors: shifted token ids, a
slice of a wider projection, transposed weights."""
import pytest
import torch

import fine_grained_scaled_amd as fgs

pytestmark = pytest.mark.gpu


def _elsewhere(t):
    """The same values transposed in memory, at an unaligned place, with rows 5 values wider, and one row for all where they
    are alike."""
    flat = torch.zeros(t.numel() + 8, dtype=t.dtype, device=t.device)
    wide = torch.zeros(t.shape[0], t.shape[1] + 5, dtype=t.dtype, device=t.device)
    wide[:, 2:-3] = t
    return t.t().contiguous().t(), flat[3:3 + t.numel()].view(t.shape).copy_(t), wide[:, 2:-3]


@pytest.mark.parametrize("index", [torch.int32, torch.int64])
def test_shifted_tokens(index):
    """ids[:, :-1] in, ids[:, 1:] as targets: views of one batch."""
    B, S, V, K = 3, 41, 90, 64
    ids = torch.randint(0, V, (B, S), device="cuda").to(index)
    weight = torch.randn(V, K, device="cuda").requires_grad_()
    g = torch.randn(B, S - 1, K, device="cuda")
    tokens = ids[:, :-1]
    assert not tokens.is_contiguous()
    out = fgs.embedding(tokens, weight, 2.0)
    assert torch.equal(out, fgs.embedding_fwd(tokens.contiguous(), weight.detach(), 2.0))
    got, = torch.autograd.grad(out, weight, g)
    assert torch.equal(got, fgs.embedding_bwd(g, tokens.contiguous(), V, 2.0))
    x = torch.randn(B, K, device="cuda").bfloat16().requires_grad_()
    column = ids[:, 5]                       # every document's sixth token
    loss = fgs.linear_cross_entropy(x, weight, column)
    assert torch.equal(loss, fgs.linear_cross_entropy(x, weight, column.contiguous()))
    for one, other in zip(torch.autograd.grad(loss.sum(), (x, weight)),
                          torch.autograd.grad(fgs.linear_cross_entropy(x, weight, column.contiguous()).sum(), (x, weight))):
        assert torch.equal(one, other)


@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
def test_embedding_weight(kind):
    tokens = torch.randint(0, 50, (70,), device="cuda")
    weight = torch.randn(50, 64, device="cuda").to(kind)
    want = fgs.embedding_fwd(tokens, weight, 0.5)
    g = torch.randn(70, 64, device="cuda").to(kind)
    for w in _elsewhere(weight) + (weight[:1].expand(50, 64),):
        w = w.detach().requires_grad_()
        out = fgs.embedding(tokens, w, 0.5)
        assert torch.equal(out, want if w.stride(0) else want.new_tensor(0.5) * weight[:1].expand(70, 64))
        grad, = torch.autograd.grad(out, w, g)
        assert torch.equal(grad, fgs.embedding_bwd(g, tokens, 50, 0.5, kind))


@pytest.mark.parametrize("checkpoint", [True, False])
def test_swiglu_input(checkpoint):
    x = torch.randn(40, 2 * 136, device="cuda").bfloat16()
    dh = torch.randn(40, 136, device="cuda").bfloat16()
    leaf = x.clone().requires_grad_()
    want = fgs.swiglu(leaf, checkpoint)
    want_grad, = torch.autograd.grad(want, leaf, dh)
    for v in _elsewhere(x):
        v = v.detach().requires_grad_()
        h = fgs.swiglu(v, checkpoint)
        assert torch.equal(h, want) and torch.equal(torch.autograd.grad(h, v, dh)[0], want_grad)


def test_refusals_name_what_is_wrong():
    x, w = torch.zeros(8, 64, device="cuda").bfloat16(), torch.zeros(9, 64, device="cuda").bfloat16()
    t = torch.zeros(8, dtype=torch.int64, device="cuda")
    for bad in ((x[0], w, t[:1]), (x[None], w, t), (x, w[0], t)):
        with pytest.raises((TypeError, ValueError)):
            fgs.linear_cross_entropy(*bad)
    with pytest.raises((TypeError, ValueError)):
        fgs.embedding(t, w[0])
    with pytest.raises((TypeError, ValueError)):
        fgs.swiglu(x[0])
