"""Causal attention over packed sequences, forward and backward, against its
definition in 64 bits (tests/_operator_refs.py, whose bounds follow from the
roundings that include/fgs.h names)."""
import pytest
import torch

import fine_grained_scaled_amd as fgs
from _operator_refs import attention, pack_offsets, within

pytestmark = pytest.mark.gpu


def _inputs(lengths, H, Hk, D, seed=0, fused=False, before=0, after=0, gain=1.0):
    g = torch.Generator().manual_seed(seed)
    T = before + sum(lengths) + after
    x = torch.randn(T, H + 2 * Hk, D, generator=g)
    x[:, :H] *= gain
    x = x.to(torch.bfloat16)
    dout = torch.randn(T, H, D, generator=g).to(torch.bfloat16)
    q, k, v = x[:, :H], x[:, H:H + Hk], x[:, H + Hk:]
    if fused:
        dev = x.cuda()
        on = dev[:, :H], dev[:, H:H + Hk], dev[:, H + Hk:]
    else:
        on = tuple(t.contiguous().cuda() for t in (q, k, v))
    return (q, k, v), on, dout, pack_offsets(lengths, before)


def _check(lengths, H, Hk, D, scale=None, **how):
    host, on, dout, cu = _inputs(lengths, H, Hk, D, **how)
    want = attention(*host, cu, D ** -0.5 if scale is None else scale, dout)
    cu = cu.cuda()
    out, lse = fgs.attention_fwd(*on, cu, softmax_scale=scale)
    dq, dk, dv = fgs.attention_bwd(dout.cuda(), *on, out, lse, cu, softmax_scale=scale)
    torch.cuda.synchronize()
    for name, got in (("out", out), ("lse", lse), ("dv", dv), ("dq", dq), ("dk", dk)):
        within(name, got, want[name])


# lengths around the tiles of 32, 64 and 128 rows, and sequences of none
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lengths", [[1], [2, 1, 0, 3], [31, 33], [64], [65, 63], [127, 0, 128, 129], [300], [17] * 70, [3] * 254, [2] * 255],
                         ids=str)
def test_lengths(lengths, D):
    _check(lengths, 4, 2, D, seed=len(lengths))


@pytest.mark.parametrize("H,Hk", [(1, 1), (3, 1), (4, 1), (6, 2), (5, 5), (8, 1), (16, 8), (32, 8), (8, 8)])
def test_heads(H, Hk):
    _check([45, 150], H, Hk, 128, seed=H, fused=True)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("gain,scale", [(8.0, None), (30.0, None), (1.0, 0.5), (1.0, 1e-3)])
def test_scores_large_and_small(gain, scale, D):
    """Scores of hundreds move the running maximum again and again."""
    _check([200, 40], 2, 2, D, seed=3, gain=gain, scale=scale)


@pytest.mark.parametrize("lengths,H,Hk,D", [([1500, 60], 2, 1, 128), ([1300], 4, 1, 64), ([70, 1, 1100, 0, 131], 3, 3, 64),
                                            ([1280, 1280], 8, 2, 128)], ids=str)
def test_long_sequences_share_their_key_tiles(lengths, H, Hk, D):
    """Few heads and a long sequence: several workgroups a key tile, whose
    sums meet in the workspace; the same bits again, and in a replayed graph."""
    _check(lengths, H, Hk, D, seed=sum(lengths), before=5, after=130)
    _, on, dout, cu = _inputs(lengths, H, Hk, D, seed=1)
    cu, dout = cu.cuda(), dout.cuda()
    out, lse = fgs.attention_fwd(*on, cu)
    first = fgs.attention_bwd(dout, *on, out, lse, cu)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = fgs.attention_bwd(dout, *on, out, lse, cu)
    for _ in range(4):
        again = fgs.attention_bwd(dout, *on, out, lse, cu)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) and torch.equal(a, c) for a, b, c in zip(first, again, got))


def test_tokens_of_no_sequence():
    host, on, dout, cu = _inputs([40, 0, 70], 4, 2, 128, seed=5, before=37, after=50)
    _check([40, 0, 70], 4, 2, 128, seed=5, before=37, after=50)
    out, lse = fgs.attention_fwd(*on, cu.cuda())
    grads = fgs.attention_bwd(dout.cuda(), *on, out, lse, cu.cuda())
    for t in (out, *grads):
        assert not t[:37].any() and not t[147:].any()
    assert (lse[:, :37] == -torch.inf).all() and (lse[:, 147:] == -torch.inf).all()


def test_no_sequence_and_no_token():
    on = [torch.zeros(0, h, 64, dtype=torch.bfloat16, device="cuda") for h in (4, 2, 2)]
    cu = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = fgs.attention_fwd(*on, cu)
    assert out.shape == (0, 4, 64) and lse.shape == (4, 0)
    assert [tuple(t.shape) for t in fgs.attention_bwd(out, *on, out, lse, cu)] == [(0, 4, 64), (0, 2, 64), (0, 2, 64)]
    on = [torch.ones(9, h, 64, dtype=torch.bfloat16, device="cuda") for h in (4, 2, 2)]
    out, lse = fgs.attention_fwd(*on, cu)
    assert not out.any() and (lse == -torch.inf).all()


def test_strides_and_broadcast_heads():
    """Heads outermost, keys shared by every head as an expanded view, a row
    pitch that is no multiple of the heads."""
    host, _, dout, cu = _inputs([90, 33], 4, 4, 64, seed=7)
    q = host[0].transpose(0, 1).contiguous().cuda().transpose(0, 1)
    k = host[1][:, :1].cuda().expand(-1, 4, -1)
    wide = torch.zeros(123, 5, 64, dtype=torch.bfloat16, device="cuda")
    wide[:, :4] = host[2].cuda()
    v = wide[:, :4]
    want = attention(host[0], host[1][:, :1].expand(-1, 4, -1), host[2], cu, 0.125, dout)
    out, lse = fgs.attention_fwd(q, k, v, cu.cuda())
    got = fgs.attention_bwd(dout.cuda(), q, k, v, out, lse, cu.cuda())
    for name, t in zip(("out", "lse", "dq", "dk", "dv"), (out, lse, *got)):
        within(name, t, want[name])


def test_non_finite_values_stay_where_the_mask_puts_them():
    """A row depends on the tokens it sees: NaN and Inf in later tokens, in
    other sequences and in tokens of none do not reach it."""
    lengths = [70, 150, 20]
    host, _, dout, cu = _inputs(lengths, 4, 2, 128, seed=9, after=13)
    q, k, v = (t.clone() for t in host)
    clean = attention(q, k, v, cu, 128 ** -0.5)
    at = 70 + 100                                   # token 100 of the second sequence
    v[at, 0, 5] = torch.inf
    v[at + 20, 1, 9] = torch.nan
    k[at + 30, 0, 3] = torch.nan
    q[at + 40, 2] = torch.nan
    v[240:] = torch.nan
    k[240:] = torch.inf
    on = [t.cuda() for t in (q, k, v)]
    out, lse = fgs.attention_fwd(*on, cu.cuda())
    for rows in (slice(0, at), slice(220, 253)):
        within("out", out[rows], [t[rows] for t in clean["out"]])
        within("lse", lse[:, rows], [t[:, rows] for t in clean["lse"]])
    got, ref = out.cpu().to(torch.float64), torch.zeros(253, 4, 128, dtype=torch.float64)
    # the rows after them, key by key, hidden keys left out
    for t in range(at, 220):
        for h in range(4):
            s = slice(70, t + 1)
            z = (k[s, h // 2].double() @ q[t, h].double()) * 128 ** -0.5
            p = torch.softmax(z, 0)
            ref[t, h] = p @ v[s, h // 2].double()
    bad = got[at:220].isfinite() != ref[at:220].isfinite()
    assert not bad.any(), f"{int(bad.sum())} values finite on one side only"
    ok = ref[at:220].isfinite()
    assert ((got[at:220] - ref[at:220]).abs()[ok] <= clean["out"][1][at:220][ok]).all()
    # the backward pass keeps them in their sequence
    dq, dk, dv = fgs.attention_bwd(dout.cuda(), *on, out, lse, cu.cuda())
    for t in (dq, dk, dv):
        assert t[:70].isfinite().all() and t[220:].isfinite().all()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lengths,at,H,Hk", [([70, 150, 20], 170, 4, 2), ([40, 60], 50, 3, 3), ([30, 1300], 1201, 2, 1)],
                         ids=str)
@pytest.mark.parametrize("where", ["dout", "q", "k", "v"])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_gradients_of_rows_that_see_nothing_non_finite(where, value, lengths, at, H, Hk, D):
    """One NaN or Inf in token `at`: the gradients that the formulas keep
    apart from it are those without it."""
    host, _, dout, cu = _inputs(lengths, H, Hk, D, seed=23)
    want = attention(*host, cu, D ** -0.5, dout)
    x = dict(q=host[0].clone(), k=host[1].clone(), v=host[2].clone(), dout=dout.clone())
    x[where][at, 0, 7] = value
    q, k, v = (x[n].cuda() for n in "qkv")
    out, lse = fgs.attention_fwd(q, k, v, cu.cuda())
    got = dict(zip(("dq", "dk", "dv"), fgs.attention_bwd(x["dout"].cuda(), q, k, v, out, lse, cu.cuda())))
    begin, end = next((a, b) for a, b in zip(cu[:-1].tolist(), cu[1:].tolist()) if a <= at < b)
    every = torch.arange(sum(lengths))
    other = (every < begin) | (every >= end)
    if where in ("q", "dout"):      # rows other than `at`; keys that `at` does not see
        keep = dict(dq=every != at, dk=other | (every > at), dv=other | (every > at))
    else:                           # rows that do not see `at`; keys of other sequences
        keep = dict(dq=other | (every < at), dk=other, dv=other)
    for name, rows in keep.items():
        within(name, got[name][rows.cuda()], [t[rows] for t in want[name]])


def test_rows_without_a_finite_score():
    """Keys of -Inf give a first row scores of -Inf only: out 0, lse -Inf."""
    host, _, _, cu = _inputs([40], 2, 1, 64, seed=11)
    q, k, v = (t.clone() for t in host)
    q[:, :, 0] = 1.0
    k[0] = 0.0
    k[0, 0, 0] = -torch.inf
    q[:, :, 1:] = q[:, :, 1:].nan_to_num()
    out, lse = fgs.attention_fwd(q.cuda(), k.cuda(), v.cuda(), cu.cuda())
    assert not out[0].any() and (lse[:, 0] == -torch.inf).all()
    assert out[1:].isfinite().all() and lse[:, 1:].isfinite().all()
    # row 1 sees one finite score: its own value
    assert torch.equal(out[1].cpu(), v[1].expand(2, -1))


def test_same_bits_again():
    _, on, dout, cu = _inputs([500, 77, 300], 8, 2, 128, seed=13)
    cu, dout = cu.cuda(), dout.cuda()
    first = None
    for _ in range(3):
        out, lse = fgs.attention_fwd(*on, cu)
        now = (out, lse, *fgs.attention_bwd(dout, *on, out, lse, cu))
        first = first or now
        assert all(torch.equal(a, b) for a, b in zip(first, now))


def test_offsets_past_32_bits():
    """A pack whose last rows lie more than 2^32 bytes into the tensors."""
    T, H, D = 70000, 1, 64
    wide = torch.empty(T, 1, 34000, dtype=torch.bfloat16, device="cuda")      # 4.76e9 bytes
    host, _, dout, _ = _inputs([130], H, H, D, seed=15)
    rows = slice(T - 130, T)
    views = []
    for i in range(3):
        x = wide[:, :, i * D:(i + 1) * D]
        x[rows] = host[i].cuda()
        views.append(x)
    cu = torch.tensor([T - 130, T], dtype=torch.int32)
    want = attention(*host, torch.tensor([0, 130]), D ** -0.5, dout)
    out, lse = fgs.attention_fwd(*views, cu.cuda())
    full = torch.zeros(T, H, D, dtype=torch.bfloat16, device="cuda")
    full[rows] = dout.cuda()
    dq, dk, dv = fgs.attention_bwd(full, *views, out, lse, cu.cuda())
    for name, t in (("out", out[rows]), ("lse", lse[:, rows]), ("dq", dq[rows]), ("dk", dk[rows]), ("dv", dv[rows])):
        within(name, t, want[name])
    assert not out[:T - 130].any() and not dk[:T - 130].any()


def test_autograd_against_differences():
    """The gradient of sum(out * w) along a random direction, by central
    differences of the 64-bit definition."""
    host, on, w, cu = _inputs([50, 29], 4, 2, 64, seed=17)
    leaves = [t.detach().clone().requires_grad_() for t in on]
    (fgs.attention(*leaves, cu.cuda()) * w.cuda()).float().sum().backward()
    g = torch.Generator().manual_seed(1)
    for i, leaf in enumerate(leaves):
        d = torch.randn(host[i].shape, generator=g, dtype=torch.float64)
        at = [t.to(torch.float64) for t in host]

        def f(x):
            args = list(at)
            args[i] = x
            return (attention(*args, cu, 0.125)["out"][0] * w.double()).sum()
        h = 1e-5
        want = (f(at[i] + h * d) - f(at[i] - h * d)) / (2 * h)
        bounds = attention(*host, cu, 0.125, w)[("dq", "dk", "dv")[i]][1]
        tol = (bounds * d.abs()).sum() + 1e-6
        assert abs((leaf.grad.cpu().double() * d).sum() - want) <= tol


def test_other_stream_and_graph_replays():
    _, on, dout, cu = _inputs([190, 66], 8, 2, 128, seed=19)
    cu, dout = cu.cuda(), dout.cuda()

    def step():
        out, lse = fgs.attention_fwd(*on, cu)
        return (out, lse, *fgs.attention_bwd(dout, *on, out, lse, cu))
    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for gain in (1.0, 0.5, 2.0):
        on[0].mul_(gain)
        want = step()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))
