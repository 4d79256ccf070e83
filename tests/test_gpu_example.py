"""examples/moe_block.py end to end: training lowers the loss with clipped
gradients, and the few-token serving path gives the training path's outputs."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_block_trains_and_serves():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import moe_block

    r = moe_block.main()
    assert r["losses"][-1] < 0.9 * r["losses"][0]
    assert r["norms"][0] > 1.0 and r["clipped"] <= 1.0 + 1e-5  # clipping is at work
    # fp32 on both sides: sums of 256 and 512 terms of order one
    assert all(v < 1e-4 for v in r["served"].values()), r["served"]
