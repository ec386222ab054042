"""The norms around a block at the edges of what their header allows: in place with parts absent, and calls without rows."""
import pytest
import torch

import weight_quantized_mlp_amd as wq
from adapter_common import DEV, randn

F32, BF16 = torch.float32, torch.bfloat16
gpu = pytest.mark.gpu


@gpu
@pytest.mark.parametrize("ht", [F32, BF16])
@pytest.mark.parametrize("H", [320, 5120, 12000, 16392])          # one, two and four chunks per thread, rows read again
@pytest.mark.parametrize("post,gate,pre", [(False, False, True), (True, False, False), (False, True, True), (True, True, True)])
def test_in_place_with_absent_parts(H, ht, post, gate, pre):
    """h_out = h and dh_in = dh give the bits of separate outputs, whichever parts are there."""
    M = 300
    h, y = randn(1, (M, H), ht)[0], randn(2, (M, H), BF16)[0]
    kw = dict(post=randn(3, (H,))[0] if post else None, gate=randn(4, (3, H))[0] if gate else None, alpha=0.7,
              pre=randn(5, (H,))[0] if pre else None)
    ho, x = wq.block_norm_run(h, y, **kw)
    into = h.clone()
    a, b = wq.block_norm_run(into, y, h_out=into, **kw)
    assert a is into and torch.equal(a, ho) and (not pre or torch.equal(b, x))
    dh, dx = randn(6, (M, H), ht)[0], randn(7, (M, H), ht)[0] if pre else None
    apart = wq.block_norm_backward(ho, y, dh, dx, **kw)
    for p, q in zip(wq.block_norm_backward(ho, y, dh, dx, dh_in=dh, **kw), apart):
        assert q is None or torch.equal(p, q)
