"""qlinear_backward on rows of a wide range: infinities among finite values, and small elements beside a large one."""
import numpy as np
import pytest
import torch

import oracle
import synth
import weight_quantized_mlp_amd as wq
from adapter_common import DEV, U, host

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
FP8, NV = wq.WQ_FMT_FP8W, wq.WQ_FMT_NVFP4


def weights(fmt, N, K, scale=1.0):
    """(w, scale, global scale, float64 dequantised [N, K]) with zeros among the codes."""
    if fmt == FP8:
        r = np.random.default_rng(N)
        codes = synth.to_e4m3_codes((r.standard_normal((N, K)) * 20).astype(np.float32))
        codes[r.random((N, K)) < 0.25] = 0
        s = np.full(N, scale, dtype=np.float32)
        return torch.from_numpy(codes).to(DEV), torch.from_numpy(s).to(DEV), 1.0, oracle.e4m3_to_f64(codes) * scale
    wp, ws, gs = synth.nvfp4_tensor(N, K, 31, 1)
    blk = oracle.block64_pack(wp, ws)
    return torch.from_numpy(blk).to(DEV), None, float(gs), oracle.nvfp4_dequant(blk, gs).astype(np.float64)


@pytest.mark.parametrize("M", [5, 200])
@pytest.mark.parametrize("dxt", [F32, BF16])
@pytest.mark.parametrize("fmt", [FP8, NV], ids=["fp8", "nvfp4"])
def test_an_infinity_keeps_its_sign_beside_large_values(fmt, dxt, M):
    """inf times a weight is an infinity of the weight's sign, and NaN times zero weights; finite neighbours of any size
    change nothing, though they lie past float16's range."""
    N, K = 150, 320
    w, s, gs, dq = weights(fmt, N, K)
    assert (dq == 0).any()
    dy = torch.randn((M, N), device=DEV, generator=torch.Generator(DEV).manual_seed(M)) * 1e6
    dy[0, 7] = float("inf")
    dy[1, 149] = float("-inf")
    dy[2, 3], dy[2, 4] = float("inf"), float("-inf")
    got = host(wq.qlinear_backward(fmt, dy, w, s, gs, dtype=dxt))
    with np.errstate(invalid="ignore"):
        for m, sign, n in ((0, 1, 7), (1, -1, 149)):
            want = sign * np.inf * dq[n]
            assert np.array_equal(np.isnan(got[m]), np.isnan(want)) and np.array_equal(got[m][dq[n] != 0], want[dq[n] != 0])
        want = np.inf * dq[3] - np.inf * dq[4]
    assert np.array_equal(got[2], want.astype(np.float32), equal_nan=True)
    assert np.isfinite(got[3:]).all()


@pytest.mark.parametrize("M", [5, 200])
@pytest.mark.parametrize("dxt", [F32, BF16])
@pytest.mark.parametrize("fmt", [FP8, NV], ids=["fp8", "nvfp4"])
def test_small_elements_beside_a_large_one(fmt, dxt, M):
    """A large element in every row, the others 2^-14 to 2^-40 of it.  Where the large one meets a zero weight dx is made
    of the small ones alone, and is as exact as they were taken: within 2^-22 (bfloat16 dx: 2^-11) of each, or 2^-51
    (2^-39) of the row's largest."""
    N, K = 150, 320
    w, s, gs, dq = weights(fmt, N, K)
    r = np.random.default_rng(M)
    for bits in (14, 20, 28, 40):
        dyn = (r.standard_normal((M, N)) * 2.0 ** -bits).astype(np.float32)
        at = r.integers(0, N, M)
        dyn[np.arange(M), at] = np.where(r.random(M) < 0.5, -1.0, 1.0)
        got = host(wq.qlinear_backward(fmt, torch.from_numpy(dyn).to(DEV), w, s, gs, dtype=dxt)).astype(np.float64)
        dyd = dyn.astype(np.float64)
        ref, size = dyd @ dq, np.abs(dyd) @ np.abs(dq)
        each, floor = (2.0 ** -22, 2.0 ** -51) if dxt == F32 else (2.0 ** -11, 2.0 ** -39)
        # the elements as they are taken (FP8: and scaled; NVFP4: 1 / global scale and its product), the sums, dx's rounding
        bound = (each + 4 * U + 2 * (N + 8) * U) * size + floor * np.abs(dyd).max(1, keepdims=True) * np.abs(dq).sum(0) + \
            torch.finfo(dxt).eps / 2 * np.abs(ref)
        assert np.all(np.abs(got - ref) <= bound), bits
        zero = dq[at] == 0
        assert zero.any() and np.all(size[zero] < 1.5 * N * 2.0 ** -bits * np.abs(dq).max())    # those columns see no large one
