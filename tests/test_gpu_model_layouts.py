"""The operators at a model's ends and SwiGLU on inputs and gradients in other
layouts, and two calls at once."""
import pytest
import torch

import fine_grained_scaled_amd as fgs

pytestmark = pytest.mark.gpu


def _layouts(t):
    """The same values elsewhere: transposed in memory, at an unaligned place, with wide rows."""
    flat = torch.zeros(t.numel() + 8, dtype=t.dtype, device=t.device)
    moved = flat[3:3 + t.numel()].view(t.shape).copy_(t)
    wide = torch.zeros(t.shape[0], t.shape[1] + 5, dtype=t.dtype, device=t.device)
    wide[:, 2:-3] = t
    return t.t().contiguous().t(), moved, wide[:, 2:-3]


def test_output_head():
    T, V, K = 70, 301, 128
    x, w = torch.randn(T, K, device="cuda").bfloat16(), (torch.randn(V, K, device="cuda") / 11).bfloat16()
    targets = torch.randint(0, V, (T,), device="cuda")

    def run(x, w, dloss):
        x, w = x.detach().requires_grad_(), w.detach().requires_grad_()
        loss = fgs.linear_cross_entropy(x, w, targets)
        return loss.detach(), *torch.autograd.grad(loss, (x, w), dloss)

    dloss = torch.rand(T, device="cuda")
    want = run(x, w, dloss)
    for a, b in zip(_layouts(x), _layouts(w)):
        for one, other in zip(run(a, b, dloss.repeat_interleave(3)[::3]), want):
            assert torch.equal(one, other)
    for one, other in zip(run(x, w, torch.ones((), device="cuda").expand(T)), run(x, w, torch.ones(T, device="cuda"))):
        assert torch.equal(one, other)


def test_embedding():
    T, V, W = 90, 50, 64
    tokens = torch.randint(0, V, (T,), device="cuda", dtype=torch.int32)
    for kind in (torch.float32, torch.bfloat16):
        weight = torch.randn(V, W, device="cuda").requires_grad_()
        out = fgs.embedding(tokens, weight, 0.5, kind)
        dout = torch.randn(T, W, device="cuda").to(kind)
        want, = torch.autograd.grad(out, weight, dout, retain_graph=True)
        for d in _layouts(dout):
            assert torch.equal(torch.autograd.grad(out, weight, d, retain_graph=True)[0], want)
        assert torch.equal(want, fgs.embedding_bwd(dout, tokens.long(), V, 0.5))


@pytest.mark.parametrize("checkpoint", [True, False])
def test_swiglu(checkpoint):
    x = torch.randn(40, 2 * 136, device="cuda").bfloat16().requires_grad_()
    h = fgs.swiglu(x, checkpoint)
    dh = torch.randn(40, 136, device="cuda").bfloat16()
    want, = torch.autograd.grad(h, x, dh, retain_graph=True)
    for d in _layouts(dh):
        assert torch.equal(torch.autograd.grad(h, x, d, retain_graph=True)[0], want)


def test_two_calls_at_once():
    """Calls on two streams share nothing."""
    sides = [torch.cuda.Stream() for _ in range(2)]
    inputs, want = [], []
    for i, (T, V, K) in enumerate([(600, 3001, 256), (90, 5003, 320)]):
        g = torch.Generator(device="cuda").manual_seed(i)
        x, w = torch.randn(T, K, generator=g, device="cuda").bfloat16(), (torch.randn(V, K, generator=g, device="cuda") / 16).bfloat16()
        inputs.append((x, w, torch.randint(0, V, (T,), generator=g, device="cuda"), torch.rand(T, generator=g, device="cuda")))

    def run(x, w, targets, dloss):
        loss, lse = fgs.linear_cross_entropy_fwd(x, w, targets)
        dx, dw = fgs.linear_cross_entropy_bwd(dloss, x, w, targets, lse)
        h, kept = fgs.swiglu_fwd(x)
        return loss, lse, dx, dw, fgs.embedding_bwd(dx, targets, w.shape[0]), h, fgs.swiglu_bwd(h, kept)

    want = [run(*a) for a in inputs]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for side, a in zip(sides, inputs):
            with torch.cuda.stream(side):
                got.append(run(*a))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            for one, other in zip(a, b):
                assert torch.equal(one, other)


def test_own_workspaces():
    """A caller's workspace, with what an earlier call left in it."""
    T, V, K = 300, 1001, 128
    x, w = torch.randn(T, K, device="cuda").bfloat16(), (torch.randn(V, K, device="cuda") / 11).bfloat16()
    targets = torch.randint(0, V, (T,), device="cuda")
    dloss = torch.rand(T, device="cuda")
    loss, lse = fgs.linear_cross_entropy_fwd(x, w, targets)
    dx, dw = fgs.linear_cross_entropy_bwd(dloss, x, w, targets, lse)
    de = fgs.embedding_bwd(dx, targets, V)
    room = torch.full((1 << 28,), 0xFF, dtype=torch.uint8, device="cuda")
    for _ in range(2):
        a, b = fgs.linear_cross_entropy_fwd(x, w, targets, workspace=room)
        assert torch.equal(a, loss) and torch.equal(b, lse)
        a, b = fgs.linear_cross_entropy_bwd(dloss, x, w, targets, lse, workspace=room)
        assert torch.equal(a, dx) and torch.equal(b, dw)
        assert torch.equal(fgs.embedding_bwd(dx, targets, V, workspace=room), de)
    with pytest.raises(fgs.FgsError):
        fgs.linear_cross_entropy_fwd(x, w, targets, workspace=room[:100])
