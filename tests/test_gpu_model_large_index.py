"""The operators at a model's ends and SwiGLU where element offsets pass 2^31."""
import pytest
import torch

import fine_grained_scaled_amd as fgs
from _model_refs import check, linear_cross_entropy

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def memory_back():
    yield
    torch.cuda.empty_cache()


def test_embedding():
    V, W = 40000, 65536
    w = torch.empty(V, W, device="cuda", dtype=torch.bfloat16)
    w[-3:] = torch.randn(3, W, device="cuda").bfloat16()
    w[:2] = torch.randn(2, W, device="cuda").bfloat16()
    tokens = torch.tensor([V - 1, 0, V - 2, 1, V - 1], device="cuda")
    assert torch.equal(fgs.embedding_fwd(tokens, w), w[tokens])
    del w
    dout = torch.randn(5, W, device="cuda").bfloat16()
    dw = fgs.embedding_bwd(dout, tokens, V)
    assert torch.equal(dw[V - 1], dout[0].float() + dout[4].float()) and torch.equal(dw[V - 2], dout[2].float())
    assert torch.equal(dw[0], dout[1].float()) and torch.equal(dw[1], dout[3].float())
    assert not dw[2:V - 2].any()
    fgs.embedding_bwd(dout[:1], tokens[:1], V, out=dw)
    assert torch.equal(dw[V - 1], (dout[0].float() + dout[4].float()) + dout[0].float()) and not dw[2:V - 2].any()


@pytest.mark.parametrize("T", [3, 150])
def test_output_head(T):
    V, K = 140003, 16384
    g = torch.Generator(device="cuda").manual_seed(T)
    w = torch.empty(V, K, device="cuda", dtype=torch.bfloat16)
    for part in w.split(20000):
        part.copy_(torch.randn(part.shape, generator=g, device="cuda") / 128)
    x = torch.randn(T, K, generator=g, device="cuda").bfloat16()
    targets = torch.randint(V - 2000, V, (T,), generator=g, device="cuda")
    dloss = torch.rand(T, generator=g, device="cuda")
    loss, lse = fgs.linear_cross_entropy_fwd(x, w, targets)
    dx, dw = fgs.linear_cross_entropy_bwd(dloss, x, w, targets, lse)
    want = linear_cross_entropy(x, w, targets, dloss)
    for name, got in (("loss", loss), ("lse", lse), ("dx", dx)):
        check(name, got, want[name])
    for a in range(0, V, 20000):
        check("dw", dw[a:a + 20000], tuple(t[a:a + 20000] for t in want["dw"]))


def test_swiglu():
    T, I = 20000, 65536
    x = torch.zeros(T, 2 * I, device="cuda", dtype=torch.bfloat16)
    x[-5:] = torch.randn(5, 2 * I, device="cuda").bfloat16()
    dh = torch.zeros(T, I, device="cuda", dtype=torch.bfloat16)
    dh[-5:] = torch.randn(5, I, device="cuda").bfloat16()
    h, kept = fgs.swiglu_fwd(x)
    d = fgs.swiglu_bwd(dh, kept)
    want, want_kept = fgs.swiglu_fwd(x[-5:])
    assert torch.equal(h[-5:], want) and torch.equal(kept.q[-5:], want_kept.q)
    assert torch.equal(kept.scales[:, -5:], want_kept.scales) and torch.equal(d[-5:], fgs.swiglu_bwd(dh[-5:], want_kept))
    assert not h[:-5].any() and not d[:-5].any()
