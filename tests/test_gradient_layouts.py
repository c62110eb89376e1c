"""Gradients reach a backward pass in whatever layout the rest of the graph
gives them: each is read as it is or copied, and none is refused."""
import pytest
import torch

import fine_grained_scaled_amd as fgs
from fine_grained_scaled_amd.ops import _readable


def _ok(t, least):
    return t.stride(-1) == 1 and t.data_ptr() % 16 == 0 and all(s % 8 == 0 and s >= least for s in t.stride()[:-1])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=str)
def test_readable(dtype):
    flat = torch.arange(4096, dtype=torch.float32).to(dtype)
    assert flat.data_ptr() % 16 == 0
    as_they_are = [flat[:1024].view(16, 64), flat.view(32, 128)[:, 64:], flat.view(8, 4, 128)[:, 1:3, :64]]
    for t in as_they_are:
        assert _readable(t, 64) is t
    copied = [flat[1:1025].view(16, 64), flat[3:1027].view(2, 8, 64), flat.view(64, 64).t(), flat[:64].expand(16, 64),
              flat[:2040].view(30, 68)[:, :64], flat[:16].view(16, 1).expand(16, 64)]
    for t in copied:
        got = _readable(t, 64)
        assert _ok(got, 64) and torch.equal(got, t)
    heads = flat.view(32, 2, 64)[:, :1].expand(-1, 4, -1)
    assert _readable(heads, 0) is heads


def _apart(x):
    """x's values through torch.cat behind one other value: the gradient comes
    back contiguous, one value off its alignment."""
    return torch.cat([x.new_zeros(1), x.flatten()])


@pytest.mark.gpu
@pytest.mark.parametrize("residual", [torch.float32, torch.bfloat16], ids=str)
def test_boundary_after_cat(residual):
    g = torch.Generator().manual_seed(0)
    y, x = torch.randn(5, 64, generator=g).to(torch.bfloat16).cuda(), torch.randn(5, 64, generator=g).to(residual).cuda()
    w = torch.ones(64, device="cuda")
    a = torch.randn(2, 320, generator=g).cuda()

    def grads(through):
        on = [t.detach().clone().requires_grad_() for t in (y, x, w)]
        r, n = fgs.residual_norm(on[0], on[1], w_pre=on[2])
        ((through(r).float() * a[0]).sum() + (through(n).float() * a[1]).sum()).backward()
        return [t.grad for t in on]
    for got, want in zip(grads(lambda t: _apart(t)[1:]), grads(torch.flatten)):
        assert torch.equal(got, want)


@pytest.mark.gpu
def test_attention_after_cat():
    g = torch.Generator().manual_seed(1)
    q, k, v = (torch.randn(40, h, 64, generator=g).to(torch.bfloat16).cuda() for h in (4, 2, 2))
    a = torch.randn(40 * 4 * 64, generator=g).to(torch.bfloat16).cuda()
    cu = torch.tensor([0, 9, 40], dtype=torch.int32, device="cuda")

    def grads(through):
        on = [t.detach().clone().requires_grad_() for t in (q, k, v)]
        (through(fgs.attention(*on, cu)) * a).sum().backward()
        return [t.grad for t in on]
    for got, want in zip(grads(lambda t: _apart(t)[1:]), grads(torch.flatten)):
        assert torch.equal(got, want)
