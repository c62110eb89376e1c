"""The example's training loop: FP8 linear layers, attention over a pack, the
block boundary and clipping together."""
import math
import os
import sys

import pytest

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "examples"))


def test_loss_falls():
    import train_block
    losses, norms = train_block.train(steps=6, tokens=256, say=lambda _: None)
    assert all(math.isfinite(v) for v in losses + norms) and min(norms) > 0
    assert losses[-1] < losses[0]
