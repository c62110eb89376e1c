"""What SwiGLU keeps, as an operand of a product: gate_up itself where the
halves' tiles are the rows' tiles, refused where a half ends inside one."""
import pytest
import torch

import fine_grained_scaled_amd as fgs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("I", [128, 384])
def test_whole_tiles_are_an_operand(I):
    x = torch.randn(256, 2 * I, device="cuda").bfloat16()
    w = fgs.quantize_blockwise(torch.randn(128, 2 * I, device="cuda").bfloat16(), "block").rowwise()
    _, kept = fgs.swiglu_fwd(x)
    want = fgs.gemm_block_scaled(fgs.quantize_blockwise(x, "tile").rowwise(), w)
    assert torch.equal(fgs.gemm_block_scaled(kept.rowwise(), w), want)


@pytest.mark.parametrize("I", [8, 64, 192, 200, 448])
def test_halves_that_end_inside_a_tile_are_none(I):
    """192: 2 x 192 columns are three tiles of whole rows, and the halves have two each."""
    x = torch.randn(40, 2 * I, device="cuda").bfloat16()
    h, kept = fgs.swiglu_fwd(x)
    with pytest.raises(ValueError):
        kept.rowwise()
    dh = torch.randn(40, I, device="cuda").bfloat16()
    # a caller's own codes and scales, in the same layout
    again = fgs.Quantized(kept.q, kept.scales, None, None, fgs.SCALE_TILE_1x128)
    assert torch.equal(fgs.swiglu_bwd(dh, kept), fgs.swiglu_bwd(dh, again))
