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


def test_a_result_type_that_contradicts_a_given_tensor():
    """A type asked for by name is never ignored in favour of another tensor's."""
    F32, BF16 = torch.float32, torch.bfloat16
    x, dy = torch.zeros((4, 64), dtype=BF16), torch.zeros((4, 48))
    a, b = torch.zeros((2, 8, 64)), torch.zeros((2, 48, 8))
    args = (dy, x, a, b, torch.zeros(2), torch.zeros(4, dtype=torch.int32))
    half, full = torch.zeros((4, 64), dtype=BF16), torch.zeros((4, 64))
    for kw in (dict(dx=half, dx_dtype=F32), dict(dx0=half, dx_dtype=F32), dict(dx0=full, dx_dtype=BF16), dict(dx0=half, dx=full)):
        with pytest.raises(TypeError, match="dx_dtype"):
            wq.lora_backward(*args, **kw)
    with pytest.raises(TypeError, match="dtype"):
        wq.qlinear_backward(wq.WQ_FMT_FP8W, dy, torch.zeros((48, 64), dtype=torch.uint8), torch.zeros(48), dtype=BF16, out=full)
    # agreeing ones pass on to the next check, of the tensors' place
    for kw in (dict(dx=half, dx_dtype=BF16), dict(dx0=half, dx=half), dict(dx0=full), dict(dx_dtype=F32), {}):
        with pytest.raises(ValueError):
            wq.lora_backward(*args, **kw)
