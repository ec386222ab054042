"""awq_linear_backward, the gradient through a frozen AWQ projection, against float64 on the dequantised weights.

Bounds as for the other formats' gradient: u = 2^-24; dy enters as float16 terms that are off by 2^-11 of the element (float32 dy into
a bfloat16 dx), by 2^-22 (float32 into float32) or not at all (bfloat16 dy), or by half of float16's smallest step, 2^-25 where the row's
largest is at least 2^14; the float32 sum of N products by 2 (N + 8) u of the sum of magnitudes; dx is rounded once.
"""
import numpy as np
import pytest
import torch

import weight_quantized_mlp_amd as wq
from adapter_common import DEV, U, host, norm_bound, randn
from awq_common import awq_weights

F32, BF16 = torch.float32, torch.bfloat16
pytestmark = pytest.mark.gpu
_cache = {}


def weights(N, K, layout):
    if (N, K, layout) not in _cache:
        bank, w = awq_weights(N + K, 1, N, K, layout)
        _cache[N, K, layout] = (bank, w[0])
    return _cache[N, K, layout]


def check(got, dyd, dq, dyt, dxt):
    N = dyd.shape[1]
    got, ref, size = host(got).astype(np.float64), dyd @ dq, np.abs(dyd) @ np.abs(dq)
    each = 0 if dyt == BF16 else (2.0 ** -11 if dxt == BF16 else 2.0 ** -22)
    floor = 2.0 ** -39 * np.abs(dyd).max(axis=1, keepdims=True) * np.abs(dq).sum(axis=0, keepdims=True)
    bound = (each + 2 * (N + 8) * U) * size + floor + (torch.finfo(dxt).eps / 2 if dxt == BF16 else 0) * np.abs(ref)
    assert np.all(np.abs(got - ref) <= bound), np.max(np.abs(got - ref) / np.maximum(bound, 1e-300))
    err = np.linalg.norm(got - ref) / max(np.linalg.norm(ref), 1e-300)
    # normwise: a float16 rounding of random signs is 2^-11 / sqrt(3) at most, times 4; bfloat16 results their own rounding
    assert err <= norm_bound(N) + (2.0 ** -9 / np.sqrt(3) + 2.0 ** -8 if dxt == BF16 else 0), err


# rows that fill no, one and several tiles; N within and past a step of 64; K of one group, tiles that end inside a record, split plans
SHAPES = [(1, 1, 32), (1, 512, 256), (3, 67, 320), (8, 1000, 544), (16, 130, 192), (33, 5120, 128), (64, 257, 1056),
          (129, 67, 320), (130, 512, 640), (257, 384, 2144), (300, 1537, 448), (700, 96, 96), (513, 4097, 288)]


@pytest.mark.parametrize("dyt,dxt", [(F32, F32), (BF16, BF16), (F32, BF16), (BF16, F32)])
@pytest.mark.parametrize("layout", [3, 4])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_gradient(M, N, K, layout, dyt, dxt):
    print("[awq_linear_backward]", M, N, K, layout, dyt, dxt, flush=True)
    bank, dq = weights(N, K, layout)
    dy, dyd = randn(M + N, (M, N), dyt, 1e-3)
    dy[M // 2] *= 1024                                                 # rows of unlike magnitudes
    dyd[M // 2] *= 1024
    guard = torch.full((M * K + 64,), 7.0, device=DEV, dtype=dxt)
    got = wq.awq_linear_backward(dy, bank, K, layout, out=guard[: M * K].view(M, K))
    assert (guard[M * K:] == 7.0).all()
    check(got, dyd, dq, dyt, dxt)


@pytest.mark.parametrize("M", [1, 40, 200])
@pytest.mark.parametrize("layout", [3, 4])
def test_one_hot_reads_the_weights(layout, M):
    """dy = e_n: dx is row n of dq(W), exactly."""
    N, K = 150, 352
    bank, dq = weights(N, K, layout)
    at = np.random.default_rng(M).integers(0, N, M)
    at[:2] = (0, N - 1)[:M] if M > 1 else (N - 1,)
    dy = torch.zeros((M, N), device=DEV)
    dy[torch.arange(M), torch.from_numpy(at)] = 1.0
    assert np.array_equal(host(wq.awq_linear_backward(dy, bank, K, layout)), dq[at].astype(np.float32))


@pytest.mark.parametrize("dyt", [F32, BF16])
def test_masked_rows_and_bad_values(dyt):
    """Zero rows give zeros; NaN and infinities stay in their row, as float32 products would have them."""
    M, N, K = 70, 131, 160
    bank, dq = weights(N, K, 3)
    dy, dyd = randn(1, (M, N), dyt)
    dy[5] = 0
    clean = wq.awq_linear_backward(dy, bank, K, dtype=F32)
    assert (clean[5] == 0).all()
    bad = dy.clone()
    bad[7, 130], bad[9, 64] = float("inf"), float("nan")
    got = wq.awq_linear_backward(bad, bank, K, dtype=F32)
    rest = [m for m in range(M) if m not in (7, 9)]
    assert torch.equal(got[rest], clean[rest]) and torch.isnan(got[9]).all()
    with np.errstate(invalid="ignore"):
        np.testing.assert_array_equal(host(got[7]), (np.sign(dq[130]) * np.inf).astype(np.float32))


@pytest.mark.parametrize("M,N,K", [(40, 1100, 256), (300, 200, 512)])
def test_is_the_gradient_of_the_forward_call(M, N, K):
    """Differences of sum(c * awq_linear_run(x)) along a direction: the map is linear, so one difference is exact up to float32."""
    bank, dq = weights(N, K, 3)
    c, cd = randn(1, (M, N))
    d, dd = randn(2, (M, K))
    dx = host(wq.awq_linear_backward(c, bank, K)).astype(np.float64)
    y = host(wq.awq_linear_run(d, bank, N)).astype(np.float64)
    assert abs(np.sum(dx * dd) - np.sum(y * cd)) <= norm_bound(N, K) * np.linalg.norm(dx) * np.linalg.norm(dd)


def test_a_replayed_graph_reads_new_values():
    M, N, K = 129, 2000, 320
    bank, _ = weights(N, K, 4)
    dy, _ = randn(1, (M, N), BF16)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        wq.awq_linear_backward(dy, bank, K, 4)
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dx = wq.awq_linear_backward(dy, bank, K, 4)
    for i in range(3):
        dy.copy_(randn(20 + i, (M, N), BF16)[0])
        want = wq.awq_linear_backward(dy, bank, K, 4)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(dx, want)


def test_empty_and_refused_calls():
    bank, _ = weights(48, 64, 3)
    assert wq.awq_linear_backward(torch.empty((0, 48), device=DEV), bank, 64).shape == (0, 64)
    dy, _ = randn(1, (4, 48), F32)
    with pytest.raises(TypeError):
        wq.awq_linear_backward(dy.half(), bank, 64)
    with pytest.raises(TypeError):
        wq.awq_linear_backward(dy, bank, 64, dtype=torch.float16)
    with pytest.raises(TypeError):
        wq.awq_linear_backward(dy, bank, 64, dtype=BF16, out=torch.empty((4, 64), device=DEV))
    with pytest.raises(ValueError):
        wq.awq_linear_backward(dy, bank, 96)
    with pytest.raises(wq.WQError):
        wq.awq_linear_backward(dy, bank, 64, workspace=torch.empty(64, dtype=torch.uint8, device=DEV))
