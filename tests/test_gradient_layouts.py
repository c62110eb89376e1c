"""Gradients reach a backward pass in whatever layout the rest of the graph
gives them: each is read as it is or copied, and none is refused."""
import ctypes

import pytest
import torch

import fine_grained_scaled_amd as fgs
from fine_grained_scaled_amd import _lib
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


def test_strides_of_single_rows_and_heads():
    """The stride of a dimension of one entry means nothing: a transposed
    column is a row with a stride of 1, and contiguous() leaves it so.  Calls
    that are not refused for a stride end at a NULL lse or n, before any HIP
    call."""
    row = torch.zeros(64, 1, dtype=torch.bfloat16).t()
    assert row.stride() == (1, 1) and row.contiguous().stride() == (1, 1)
    lib, at, null = _lib.load(), ctypes.c_void_p(0x10000), ctypes.c_void_p(0)

    def norm(rows, ld):
        assert lib.fgs_residual_norm_fwd(at, ld, at, ld, 0, rows, 64, null, at, ld, 2, 1.0, at, 1e-6, at, null, null) < 0
        return lib.fgs_last_error()
    assert b"n is NULL" in norm(1, 1) and b"n is NULL" in norm(1, 68) and b"n is NULL" in norm(2, 64)
    assert b"row stride" in norm(2, 1) and b"multiple of 8" in norm(2, 68)

    def attention(tokens, heads, token, head):
        view = lambda: (ctypes.c_int64 * 3)(0x10000, token, head)
        assert lib.fgs_attention_fwd(view(), view(), view(), at, 1, tokens, heads, heads, 64, 0.125, view(), null, null) < 0
        return lib.fgs_last_error()
    for taken in ((1, 4, 3, 64), (9, 1, 64, 1), (1, 1, -1, 5), (9, 4, 256, 64)):
        assert b"lse" in attention(*taken)
    for refused in ((2, 4, 3, 64), (9, 2, 256, 1), (9, 1, -64, 5)):
        assert b"stride" in attention(*refused)


@pytest.mark.gpu
def test_a_single_row_of_any_stride():
    g = torch.Generator().manual_seed(2)
    y, x = (torch.randn(64, 1, generator=g).to(torch.bfloat16).cuda().t() for _ in range(2))
    assert y.stride(0) == 1
    w = torch.ones(64, device="cuda")
    for got, want in zip(fgs.residual_norm_fwd(y, x, w_pre=w),
                         fgs.residual_norm_fwd(*(t.clone(memory_format=torch.contiguous_format) for t in (y, x)), w_pre=w)):
        assert torch.equal(got, want)
    q, k = torch.randn(1, 4, 64, generator=g).to(torch.bfloat16).cuda(), torch.randn(4, 1, 64, generator=g).to(torch.bfloat16).cuda()
    cu = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    v = k[2:3]
    odd = [t.as_strided(t.shape, (3, 64, 1)) for t in (q, v, v)]
    assert torch.equal(fgs.attention_fwd(*odd, cu)[0], fgs.attention_fwd(q, v, v, cu)[0])
