"""Clipping writes its tensors as torch's own operations in place do: a graph
that saved one of them notices."""
import pytest
import torch

import fine_grained_scaled_amd as fgs

pytestmark = pytest.mark.gpu


def test_version_counters():
    grads = [torch.ones(5, device="cuda"), torch.ones(70, device="cuda", dtype=torch.bfloat16)]
    fgs.clip_grad_norm(grads, 0.5)
    assert [g._version for g in grads] == [1, 1]
    out = [torch.empty_like(g) for g in grads]
    fgs.clip_grad_norm(grads, 0.25, out=out)
    assert [g._version for g in grads] == [1, 1] and [o._version for o in out] == [1, 1]
    fgs.clip_grad_norm([], 0.25)


def test_second_backward_through_a_clipped_gradient():
    x = torch.ones(8, device="cuda", requires_grad=True)
    grad, = torch.autograd.grad(x.pow(3).sum(), x, create_graph=True)
    again = (grad * grad).sum()                      # saves the gradient
    fgs.clip_grad_norm([grad.detach()], 1e-3)        # shares the counter
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        again.backward()
