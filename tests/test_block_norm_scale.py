"""block_norm_run and block_norm_backward on rows of very large and very small values, and rows of zeros under a tiny eps.

The bounds are those of test_block_norm.py: with u = 2^-24, a row sum, what it is multiplied into and a second sum over that are off
by at most chain(H) u of their magnitudes, a sum over M rows by M u more.  They hold at every size whose squares, and whose products
with the gradients, lie in float32's normal range: here 1e-28 (1e-14 squared) to 1.6e37 (16392 elements of 3e16 squared), and 1e-14 to
3e16 with gradients near 1.  Reciprocals of the norm's root then lie between 3e-17 and 1e15, du between 1e-17 and 1e15.
"""
import numpy as np
import pytest
import torch

import oracle
import weight_quantized_mlp_amd as wq
from adapter_common import DEV, host, randn
from test_block_norm import chain, near

F32, BF16 = torch.float32, torch.bfloat16
pytestmark = pytest.mark.gpu

# (eps, scales of h's rows, scales of y's rows); 0: a row of zeros
ROWS = [(1e-6, [1e15, 1e16, 1e13, 1.0, 1e-3, 0.0], [1.0] * 6), (1e-6, [1.0] * 6, [1e15, 1e16, 1e13, 1.0, 1e-3, 0.0]),
        (0.0, [1e-14, 1e-13, 1e15, 1.0], [1.0] * 4), (0.0, [1.0] * 4, [1e-14, 1e-13, 1e15, 1.0]),
        (1e-30, [0.0, 1e-14, 1.0], [1.0, 1.0, 0.0]), (1e-26, [0.0, 1e15, 1e-13], [1e-13, 0.0, 1e15])]


def scaled(seed, H, scales, dtype):
    t, _ = randn(seed, (len(scales), H))
    t = (t * torch.tensor(scales, device=DEV, dtype=F32)[:, None]).to(dtype)
    return t, t.double().cpu().numpy()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("H", [320, 7000, 16392])          # rows held as one and as two chunks per thread, and rows read again
@pytest.mark.parametrize("which", range(len(ROWS)))
def test_gradients_of_scaled_rows(which, H, dtype):
    eps, hs, ys = ROWS[which]
    M, alpha, offset = len(hs), 0.7, 1.0
    print("[block norm scale]", which, H, dtype, flush=True)
    h, hd = scaled(1, H, hs, dtype)
    y, yd = scaled(2, H, ys, dtype)
    (post, postd), (pre, pred), (gate, gated) = randn(3, (H,), F32, 0.5), randn(4, (H,), F32, 0.5), randn(5, (1, H))
    dx, dxd = randn(6, (M, H), dtype)
    eps32 = float(np.float32(eps))
    for dh, dhd in ((None, None), randn(7, (M, H), dtype)):
        got = wq.block_norm_backward(h, y, dh, dx, post=post, gate=gate, alpha=alpha, pre=pre, eps=eps, offset=offset)
        ref = oracle.block_norm_backward_ref(hd, yd, dhd, dxd, postd, gated, alpha, pred, eps32, offset)
        A = np.abs
        r = 1 / np.sqrt(np.mean(hd * hd, axis=1, keepdims=True) + eps32)
        dn = A(dxd * (offset + pred))
        du = (0 if dhd is None else A(dhd)) + r * dn + r ** 3 * A(hd) * np.mean(dn * A(hd), axis=1, keepdims=True)
        ry, w = 1 / np.sqrt(np.mean(yd * yd, axis=1, keepdims=True) + eps32), A(offset + postd)
        dp = alpha * A(gated) * du
        mags = [du, ry * dp * w + ry ** 3 * A(yd) * np.mean(dp * w * A(yd), axis=1, keepdims=True),
                np.sum(dp * A(yd) * ry, axis=0), np.sum(alpha * du * A(yd) * ry * w, axis=0, keepdims=True), np.sum(A(dxd * hd * r), axis=0)]
        for i, name in enumerate(("dh", "dy", "dpost", "dgate", "dpre")):
            near(got[i], ref[i], mags[i], dtype if i < 2 else F32, 2 * chain(H) + (M if i >= 2 else 0), name)


@pytest.mark.parametrize("H", [320, 7000, 16392])
@pytest.mark.parametrize("which", range(len(ROWS)))
def test_forward_of_scaled_rows(which, H):
    eps, hs, ys = ROWS[which]
    (h, hd), (y, yd) = scaled(1, H, hs, F32), scaled(2, H, ys, F32)
    (post, postd), (pre, pred), (gate, gated) = randn(3, (H,), F32, 0.5), randn(4, (H,), F32, 0.5), randn(5, (1, H))
    eps32 = float(np.float32(eps))
    ho, x = wq.block_norm_run(h, y, post=post, gate=gate, alpha=0.7, pre=pre, eps=eps, offset=1.0)
    ref, _ = oracle.block_norm_ref(hd, yd, postd, gated, 0.7, None, eps32, 1.0)
    near(ho, ref, np.abs(hd) + np.abs(ref - hd), F32, chain(H), "h_out")
    refx = oracle.norm_ref(host(ho).astype(np.float64), pred, eps32, 1.0)
    near(x, refx, np.abs(refx), F32, chain(H), "x")
