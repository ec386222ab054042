"""Refusals of the Python binding's adapter and gradient calls (no GPU: each is found before a tensor's place is looked at)."""
import pytest
import torch

import weight_quantized_mlp_amd as wq


@pytest.mark.parametrize("fmt,w", [(wq.WQ_FMT_FP8W, torch.zeros((0, 64), dtype=torch.uint8)),
                                   (wq.WQ_FMT_NVFP4, torch.zeros((0, 1, 36), dtype=torch.uint8))])
def test_a_projection_without_outputs(fmt, w):
    for M in (0, 4):
        with pytest.raises(ValueError, match="at least one column"):
            wq.qlinear_backward(fmt, torch.zeros((M, 0)), w, torch.zeros(0))
