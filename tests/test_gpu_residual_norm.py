"""The block boundary (norm, gate, scaled residual, norm), forward and
backward, against its definition in 64 bits (tests/_operator_refs.py)."""
import pytest
import torch

import fine_grained_scaled_amd as fgs
from fine_grained_scaled_amd import _lib
from _operator_refs import residual_norm, residual_norm_grads, within

pytestmark = pytest.mark.gpu
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _inputs(rows, width, residual, post, gate, seed=0):
    g = torch.Generator().manual_seed(seed)

    def normal(*shape, std=1.0, mean=0.0, dtype=torch.float32):
        return (torch.randn(*shape, generator=g) * std + mean).to(dtype)
    res = DTYPES[residual]
    s = dict(y=normal(rows, width, std=0.5, dtype=torch.bfloat16), x=normal(rows, width, std=2.0, dtype=res),
             dr=normal(rows, width, dtype=res), dn=normal(rows, width, dtype=torch.bfloat16))
    how = dict(w_pre=normal(width, std=0.1, mean=1.0), w_post=normal(width, std=0.1, mean=1.0) if post else None,
               gate=None if gate == "none" else normal(width, std=0.3, mean=0.5) if gate == "channel"
               else normal(rows, width, std=0.3, mean=0.5, dtype=torch.bfloat16))
    return s, how


def _on(t):
    return None if t is None else t.cuda()


def _check(s, how, alpha=0.7, eps=1e-6, move=_on):
    dev = {k: move(t) for k, t in s.items()}
    dhow = {k: _on(t) for k, t in how.items()} | dict(alpha=alpha, eps=eps)
    r, n = fgs.residual_norm_fwd(dev["y"], dev["x"], **dhow)
    got = fgs.residual_norm_bwd(dev["dr"], dev["dn"], dev["y"], r, **dhow)
    torch.cuda.synchronize()
    want = residual_norm(s["y"], s["x"], how["w_pre"], how["w_post"], how["gate"], alpha, eps, r.cpu())
    within("r", r, want["r"])
    within("n", n, want["n"])
    assert r.dtype == s["x"].dtype
    want = residual_norm_grads(s["dr"], s["dn"], s["y"], r.cpu(), how["w_pre"], how["w_post"], how["gate"], alpha, eps)
    for name in ("residual", "y", "gate", "w_post", "w_pre"):
        have = getattr(got, name)
        assert (have is None) == (name not in want), name
        if have is not None:
            within(name, have, want[name])


@pytest.mark.parametrize("gate", ["none", "channel", "token"])
@pytest.mark.parametrize("post", [True, False], ids=["post", "bare"])
@pytest.mark.parametrize("residual", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,width", [(5, 136), (33, 1032), (7, 4104)])
def test_options(rows, width, residual, post, gate):
    _check(*_inputs(rows, width, residual, post, gate, seed=rows))


# one vector, the wave's width, a thread's 1, 2 and 4 vectors and their edges
@pytest.mark.parametrize("width", [8, 64, 504, 512, 520, 1024, 2048, 7168, 8192, 8200, 16376, 16384])
@pytest.mark.parametrize("rows", [1, 3])
def test_widths(rows, width):
    _check(*_inputs(rows, width, "bf16", True, "channel", seed=width))


@pytest.mark.parametrize("rows,width", [(1100, 64), (2500, 128), (1537, 520), (700, 8192)])
def test_more_rows_than_workgroups(rows, width):
    _check(*_inputs(rows, width, "fp32", True, "channel", seed=rows))


@pytest.mark.parametrize("rows,width,residual,post,gate", [
    (300, 8200, "fp32", True, "token"), (261, 16384, "fp32", True, "channel"), (300, 16384, "bf16", True, "channel"),
    (270, 12296, "fp32", False, "channel"), (270, 12296, "bf16", False, "none"), (513, 8208, "fp32", True, "none")])
def test_wide_rows_more_than_workgroups(rows, width, residual, post, gate):
    """Rows of two vectors a thread, several to a workgroup."""
    _check(*_inputs(rows, width, residual, post, gate, seed=rows))


# rows held at once by one workgroup, and the first counts that are not
@pytest.mark.parametrize("rows,width", [(16, 64), (17, 64), (2, 4096), (3, 4096), (512, 136), (4097, 8)])
def test_rows_at_once(rows, width):
    _check(*_inputs(rows, width, "bf16", True, "channel", seed=rows))


@pytest.mark.parametrize("rows", [3, 40])
def test_sums_written_to_any_place(rows):
    """The gradients of weights and channel gate need no alignment beyond
    their values'."""
    s, how = _inputs(rows, 64, "fp32", True, "channel", seed=7)
    dev = {k: t.cuda() for k, t in (s | how).items()}
    want = fgs.residual_norm_bwd(dev["dr"], dev["dn"], dev["y"], dev["x"], w_pre=dev["w_pre"], w_post=dev["w_post"],
                                 gate=dev["gate"])
    lib = _lib.load()
    sums = torch.full((3, 68), 9.0, device="cuda")
    dx, dy = torch.empty_like(dev["x"]), torch.empty_like(dev["y"])
    ws = torch.empty(lib.fgs_residual_norm_workspace_bytes(rows, 64), dtype=torch.uint8, device="cuda")
    at = lambda t: t.data_ptr()
    _lib.check(lib.fgs_residual_norm_bwd(
        at(dev["dr"]), 64, at(dev["dn"]), 64, at(dev["y"]), 64, at(dev["x"]), 64, _lib.OUT_FP32, rows, 64,
        at(dev["w_post"]), at(dev["gate"]), 0, _lib.GATE_CHANNEL, 1.0, at(dev["w_pre"]), 1e-6, at(dx), at(dy),
        at(sums[0, 1:]), at(sums[1, 1:]), at(sums[2, 1:]), at(ws), ws.numel(),
        torch.cuda.current_stream().cuda_stream))
    for got, name in zip(sums, ("gate", "w_post", "w_pre")):
        assert torch.equal(got[1:65], getattr(want, name)) and (got[[0, 65, 66, 67]] == 9.0).all()
    assert torch.equal(dx, want.residual) and torch.equal(dy, want.y)


def test_row_strides():
    s, how = _inputs(21, 264, "bf16", True, "token", seed=3)

    def wide(t):
        x = torch.zeros(t.shape[0], t.shape[1] + 40, dtype=t.dtype, device="cuda")
        x[:, 8:-32] = t.cuda()
        return x[:, 8:-32]
    _check(s, how, move=wide)


def test_rows_of_zeros_and_extremes():
    """eps keeps a row of zeros finite; a row of large values and one of tiny
    ones stay finite as long as their squares do."""
    s, how = _inputs(6, 512, "fp32", True, "channel", seed=4)
    s["y"][0] = 0
    s["x"][0] = 0
    s["y"][1] *= 2.0 ** 50
    s["y"][2] *= 2.0 ** -50
    s["x"][3] *= 2.0 ** 50
    _check(s, how)
    s["y"][4, 7] = torch.nan
    dhow = {k: _on(t) for k, t in how.items()}
    r, n = fgs.residual_norm_fwd(s["y"].cuda(), s["x"].cuda(), **dhow)
    bad = ~n.isfinite().all(1)
    assert bad.tolist() == [False, False, False, False, True, False]
    assert not n[0].any() and not r[0].any()


def test_no_rows():
    s, how = _inputs(0, 64, "bf16", True, "channel")
    dhow = {k: _on(t) for k, t in how.items()}
    r, n = fgs.residual_norm_fwd(s["y"].cuda(), s["x"].cuda(), **dhow)
    assert r.shape == n.shape == (0, 64)
    g = fgs.residual_norm_bwd(s["dr"].cuda(), s["dn"].cuda(), s["y"].cuda(), r, **dhow)
    assert not g.w_pre.any() and not g.w_post.any() and not g.gate.any()


def test_same_bits_and_graph_replays():
    s, how = _inputs(900, 1024, "bf16", True, "channel", seed=5)
    dev = {k: _on(t) for k, t in s.items()}
    dhow = {k: _on(t) for k, t in how.items()}

    def step():
        r, n = fgs.residual_norm_fwd(dev["y"], dev["x"], **dhow)
        return (r, n, *fgs.residual_norm_bwd(dev["dr"], dev["dn"], dev["y"], r, **dhow))
    want = step()
    assert all(torch.equal(a, b) for a, b in zip(want, step()))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for gain in (1.0, 2.0, 0.25):
        dev["y"].mul_(gain)
        want = step()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("gate", ["none", "channel", "token"])
def test_autograd_against_differences(gate):
    """The gradient of sum(r * a) + sum(n * b) along random directions, by
    central differences in 64 bits."""
    s, how = _inputs(9, 72, "fp32", True, gate, seed=6)
    leaves = {"y": s["y"], "x": s["x"], **{k: t for k, t in how.items() if t is not None}}
    on = {k: t.cuda().requires_grad_() for k, t in leaves.items()}
    r, n = fgs.residual_norm(on["y"], on["x"], w_pre=on["w_pre"], w_post=on["w_post"], gate=on.get("gate"), alpha=0.7)
    ((r * s["dr"].cuda()).sum() + (n.float() * s["dn"].cuda().float()).sum()).backward()
    bounds = residual_norm_grads(s["dr"], s["dn"], s["y"], r.detach().cpu(), how["w_pre"], how["w_post"], how["gate"],
                                 0.7, 1e-6)

    def f(v):
        z = v["y"] * ((v["y"] ** 2).mean(1, keepdim=True) + 1e-6).rsqrt() * v["w_post"]
        rr = 0.7 * v["x"] + v.get("gate", 1.0) * z
        nn = rr * ((rr ** 2).mean(1, keepdim=True) + 1e-6).rsqrt() * v["w_pre"]
        return (rr * s["dr"].double()).sum() + (nn * s["dn"].double()).sum()
    gen = torch.Generator().manual_seed(2)
    for name, leaf in on.items():
        at = {k: t.double() for k, t in leaves.items()}
        d = torch.randn(at[name].shape, generator=gen, dtype=torch.float64)
        h = 1e-6
        up, down = f(at | {name: at[name] + h * d}), f(at | {name: at[name] - h * d})
        tol = (bounds["residual" if name == "x" else name][1] * d.abs()).sum() + 1e-6
        assert abs((leaf.grad.cpu().double() * d).sum() - (up - down) / (2 * h)) <= tol, name
