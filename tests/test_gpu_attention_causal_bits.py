"""A row of attention depends on the tokens that it sees alone, to the bit:
later tokens, and the other sequences of its pack, may hold anything finite."""
import pytest
import torch

import fine_grained_scaled_amd as fgs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H,Hk", [(2, 2), (4, 1), (2, 1)])
@pytest.mark.parametrize("gain", [1.0, 8.0, 40.0])
def test_later_tokens_change_no_bit(gain, H, Hk, D):
    """Scores of hundreds, of rows that grow at different tiles, make the
    kernel move the value that its exponents are taken from."""
    g = torch.Generator().manual_seed(D + H)
    T, keep = 400, 307
    q, k, v = (torch.randn(T, h, D, generator=g) for h in (H, Hk, Hk))
    q *= gain * torch.rand(T, H, 1, generator=g)
    on = [t.to(torch.bfloat16).cuda() for t in (q, k, v)]
    cu = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    out, lse = fgs.attention_fwd(*on, cu)
    for other in (0.0, 5.0):
        changed = [t.clone() for t in on]
        for t in changed:
            t[keep:] = other * torch.randn(T - keep, t.shape[1], D, generator=g).to(torch.bfloat16).cuda()
        got, got_lse = fgs.attention_fwd(*changed, cu)
        assert torch.equal(got[:keep], out[:keep]) and torch.equal(got_lse[:, :keep], lse[:, :keep])
    # the prefix by itself, behind another sequence
    front = [torch.cat([5.0 * t[:50], t[:keep]]) for t in on]
    got, got_lse = fgs.attention_fwd(*front, torch.tensor([0, 50, 50 + keep], dtype=torch.int32, device="cuda"))
    assert torch.equal(got[50:], out[:keep]) and torch.equal(got_lse[:, 50:], lse[:, :keep])
