"""The block calls on activations past 4 GiB: the rows around the boundary and the last ones, against the same rows elsewhere."""
import numpy as np
import pytest
import torch

import weight_quantized_mlp_amd as wq
from adapter_common import DEV, U
from awq_common import awq_weights

F32, BF16 = torch.float32, torch.bfloat16
pytestmark = pytest.mark.gpu
M, WIDE = 127013, 17408                                           # 4.42 GB as bfloat16
EDGE = (1 << 32) // (2 * WIDE)                                    # the row in which byte 2^32 lies
ROWS = torch.tensor([0, EDGE - 1, EDGE, EDGE + 1, M - 2, M - 1])


@pytest.fixture(scope="module")
def wide():
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.empty((M, WIDE), dtype=BF16, device=DEV)
    for r in range(0, M, 16384):
        x[r:r + 16384] = torch.randn((min(16384, M - r), WIDE), generator=g, device=DEV, dtype=F32)
    yield x
    del x
    torch.cuda.empty_cache()


def test_linear(wide):
    """Bound as in the linear's own tests: 2 (K + 8) u of the sum of magnitudes, 2^-39 of the row's largest."""
    N = 40
    bank, w = awq_weights(1, 1, N, WIDE, 3)
    y = wq.awq_linear_run(wide, bank, N)
    x = wide[ROWS.to(DEV)].double().cpu().numpy()
    got = y[ROWS.to(DEV)].double().cpu().numpy()
    tol = 2 * (WIDE + 8) * U * (np.abs(x) @ np.abs(w[0]).T) + 2.0 ** -39 * np.abs(x).max(axis=1, keepdims=True) * np.abs(w[0]).sum(axis=1)[None]
    assert np.all(np.abs(got - x @ w[0].T) <= tol)


@pytest.mark.parametrize("dxt", [BF16, F32])
def test_linear_backward(dxt):
    """dx past 4 and 8 GiB: 32 rows of dy over and over give the same 32 rows of dx over and over."""
    N = 64
    bank, _ = awq_weights(2, 1, N, WIDE, 4)
    dy = torch.randn((32, N), device=DEV).to(BF16).repeat((M + 31) // 32, 1)[:M].contiguous()
    dx = wq.awq_linear_backward(dy, bank, WIDE, 4, dtype=dxt)
    for r in (0, (EDGE // 2) // 32 * 32, EDGE // 32 * 32, M // 32 * 32 - 32):
        assert torch.equal(dx[r:r + 32], dx[:32]), r
    alone = wq.awq_linear_backward(dy[:32].float(), bank, WIDE, 4, dtype=F32)
    err = (dx[:32].float() - alone).norm() / alone.norm()
    assert err <= (2.0 ** -8 if dxt == BF16 else 2.0 ** -16)


def test_norms(wide):
    rows = ROWS.to(DEV)
    y = wide.flip(0)
    post, pre, gate = (torch.randn((WIDE,), device=DEV).to(BF16) for _ in range(3))
    kw = dict(post=post, gate=gate, alpha=0.5, pre=pre, offset=1.0)
    h, x = wq.block_norm_run(wide, y, **kw)
    h0, x0 = wq.block_norm_run(wide[rows].contiguous(), y[rows].contiguous(), **kw)
    assert torch.equal(h[rows], h0) and torch.equal(x[rows], x0)
    need = (True, True, False, False, False)
    dh, dy, *_ = wq.block_norm_backward(h, y, wide, x, need=need, **kw)
    dh0, dy0, *_ = wq.block_norm_backward(h0, y[rows].contiguous(), wide[rows].contiguous(), x0, need=need, **kw)
    assert torch.equal(dh[rows], dh0) and torch.equal(dy[rows], dy0)
