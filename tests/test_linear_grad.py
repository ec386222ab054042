"""qlinear_backward, the gradient through a frozen quantised projection, against the float64 oracle."""
import numpy as np
import pytest
import torch

import oracle
import synth
import weight_quantized_mlp_amd as wq
from adapter_common import DEV, U, host, norm_bound, randn, rel2

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
FP8, NV = wq.WQ_FMT_FP8W, wq.WQ_FMT_NVFP4
_cache = {}


def weights(fmt, N, K):
    """(w, scale, global scale, float64 dequantised [N, K])."""
    if (fmt, N, K) not in _cache:
        if fmt == FP8:
            w = np.random.default_rng(N + K).standard_normal((N, K)).astype(np.float32) * 0.02
            s = (10.0 ** np.random.default_rng(N).uniform(-3, -1, N)).astype(np.float32)
            codes = synth.to_e4m3_codes(w / (np.abs(w).max(axis=1, keepdims=True) / 448))
            _cache[fmt, N, K] = (torch.from_numpy(codes).to(DEV), torch.from_numpy(s).to(DEV), 1.0,
                                 oracle.e4m3_to_f64(codes) * s.astype(np.float64)[:, None])
        else:
            wp, ws, gs = synth.nvfp4_tensor(N, K, 23, 1)
            blk = oracle.block64_pack(wp, ws)
            _cache[fmt, N, K] = (torch.from_numpy(blk).to(DEV), None, float(gs), oracle.nvfp4_dequant(blk, gs).astype(np.float64))
    return _cache[fmt, N, K]


SHAPES = [(1, 1, 64), (1, 512, 256), (3, 67, 320), (8, 1000, 512), (16, 130, 192), (33, 5120, 128), (64, 257, 1024),
          (129, 67, 320), (130, 512, 640), (257, 384, 2112), (300, 1537, 448), (700, 96, 64)]


@pytest.mark.parametrize("dyt,dxt", [(F32, F32), (BF16, BF16), (F32, BF16), (BF16, F32)])
@pytest.mark.parametrize("fmt", [FP8, NV], ids=["fp8", "nvfp4"])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_gradient(M, N, K, fmt, dyt, dxt):
    print("[qlinear_backward]", M, N, K, fmt, dyt, dxt, flush=True)
    if fmt == FP8 and M == 3:
        K += 16                                                        # not a multiple of 64
    w, s, gs, dq = weights(fmt, N, K)
    dy, dyd = randn(M + N, (M, N), dyt, 1e-3)
    dy[M // 2] *= 1024                                                 # rows of unlike magnitudes
    dyd[M // 2] *= 1024
    got = wq.qlinear_backward(fmt, dy, w, s, gs, dtype=dxt)
    ref = dyd @ dq
    size = np.abs(dyd) @ np.abs(dq)
    assert got.dtype == dxt and tuple(got.shape) == (M, K)
    # dy's elements: one float16 rounding (bfloat16 dx: 2^-11 at most) or two terms (float32 dx: 2^-22), FP8 scales one
    # float32 rounding; subnormal float16 terms 2^-25 of a largest element of at least 2^14
    each = (2.0 ** -11 if dxt == BF16 else 2.0 ** -22) + 4 * U
    floor = 2.0 ** -25 * 2.0 ** -14 * np.abs(dyd if fmt == NV else dyd * host(s)[None, :]).max(axis=1, keepdims=True) * \
        np.abs(dq if fmt == NV else dq / host(s).astype(np.float64)[:, None]).sum(axis=0, keepdims=True)
    bound = (each + 2 * (N + 8) * U) * size + floor + torch.finfo(dxt).eps / 2 * np.abs(ref)
    assert np.all(np.abs(host(got) - ref) <= bound)
    row = np.linalg.norm(host(got) - ref, axis=1) / np.maximum(np.linalg.norm(ref, axis=1), 1e-300)
    # normwise, a float16 rounding of random signs is 2^-11 / sqrt(3) at most; times 4
    assert row.max() <= norm_bound(N) + (2.0 ** -9 / np.sqrt(3) + torch.finfo(dxt).eps / 2 if dxt == BF16 else 2.0 ** -20)


@pytest.mark.parametrize("fmt", [FP8, NV], ids=["fp8", "nvfp4"])
@pytest.mark.parametrize("M", [1, 40, 200])
def test_one_hot_reads_the_weights(fmt, M):
    """dy = e_n: dx is row n of dq(W), exactly (FP8: one rounding of the scaled code)."""
    N, K = 150, 320
    w, s, gs, dq = weights(fmt, N, K)
    at = np.random.default_rng(M).integers(0, N, M)
    at[:2] = (0, N - 1)[:M] if M > 1 else (N - 1,)
    dy = torch.zeros((M, N), device=DEV)
    dy[torch.arange(M), torch.from_numpy(at)] = 1.0
    got = host(wq.qlinear_backward(fmt, dy, w, s, gs))
    # float32 dx: the scale (FP8) enters as two float16 terms, 2^-22 of it
    assert np.all(np.abs(got - dq[at]) <= (2.0 ** -22 + 2 * U) * np.abs(dq[at]))


@pytest.mark.parametrize("fmt", [FP8, NV], ids=["fp8", "nvfp4"])
def test_zero_rows_and_masked_tokens(fmt):
    w, s, gs, dq = weights(fmt, 130, 192)
    assert wq.qlinear_backward(fmt, torch.empty((0, 130), device=DEV), w, s, gs).shape == (0, 192)
    dy, dyd = randn(4, (70, 130), F32)
    dy[::3] = 0
    got = host(wq.qlinear_backward(fmt, dy, w, s, gs))
    assert not got[::3].any() and np.isfinite(got).all()
    dy[5] = float("nan")
    dy[6, 0] = float("inf")
    bad = host(wq.qlinear_backward(fmt, dy, w, s, gs))
    keep = np.delete(np.arange(70), (5, 6))
    assert np.array_equal(bad[keep], got[keep])                        # a row's NaN stays in its row
    assert np.isnan(bad[5]).all() and not np.isfinite(bad[6]).all()
    for value in (3e38, 1e-38, 1e-44):                                 # extreme rows keep their own scale
        dy2 = torch.zeros((2, 130), device=DEV)
        dy2[0, 3] = value
        one = host(wq.qlinear_backward(fmt, dy2, w, s, gs)).astype(np.float64)
        want = float(dy2[0, 3]) * dq[3]
        fine = np.abs(want) < 3e38
        assert np.all(np.abs(one[0] - want)[fine] <= 2.0 ** -20 * np.abs(want)[fine] + 2.0 ** -149 * 1100) and not one[1].any()


def test_matches_the_forward_transpose():
    """<dy, qlinear(x)> = <qlinear_backward(dy), x>."""
    N, K, M = 320, 448, 140
    for fmt in (FP8, NV):
        w, s, gs, dq = weights(fmt, N, K)
        x, xd = randn(1, (M, K), F32)
        dy, dyd = randn(2, (M, N), F32)
        y = host(wq.qlinear_run(fmt, x, w, s, gs)).astype(np.float64)
        dx = host(wq.qlinear_backward(fmt, dy, w, s, gs)).astype(np.float64)
        # the forward rounds x to float16 (2^-11), 2-norms of the two factors
        assert abs(np.sum(dyd * y) - np.sum(dx * xd)) <= 2.0 ** -9 * np.linalg.norm(dyd) * np.linalg.norm(y)


def test_graph_replays_and_streams():
    w, s, gs, _ = weights(NV, 257, 1024)
    dy, _ = randn(6, (140, 257), F32)
    out = torch.empty((140, 1024), device=DEV)
    ws = torch.empty(max(1, wq.qlinear_backward_workspace_bytes(NV, 140, 257, 1024, F32)), dtype=torch.uint8, device=DEV)
    run = lambda: wq.qlinear_backward(NV, dy, w, s, gs, out=out, workspace=ws)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        run()
    for _ in range(3):
        dy.normal_()
        run()
        torch.cuda.synchronize()
        want = host(out).copy()
        out.fill_(float("nan"))
        ws.fill_(0xFF)
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(host(out), want)
    with torch.cuda.stream(st):
        again = wq.qlinear_backward(NV, dy, w, s, gs)
    torch.cuda.synchronize()
    assert np.array_equal(host(again), want)


def test_rows_past_4_GiB():
    M, N, K = 63000, 17408, 64                 # dy: 4.4 GB
    w, s, gs, dq = weights(FP8, N, K)
    dy = torch.randn((M, N), device=DEV, generator=torch.Generator(DEV).manual_seed(3))
    rows = [0, 1, 61679, 61680, 61681, 61682, M - 1]
    got = host(wq.qlinear_backward(FP8, dy, w, s, gs)[rows])
    assert rel2(got, dy[rows].double().cpu().numpy() @ dq) <= norm_bound(N)
