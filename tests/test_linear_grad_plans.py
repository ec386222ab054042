"""qlinear_backward on every tile height and on whole, split and mixed plans of the GEMM, against float64."""
import numpy as np
import pytest
import torch

import oracle
import synth
import weight_quantized_mlp_amd as wq
from adapter_common import DEV, U, norm_bound
from adapter_dispatch import grad_plan

F32, BF16 = torch.float32, torch.bfloat16
FP8, NV = wq.WQ_FMT_FP8W, wq.WQ_FMT_NVFP4

# M, N, K, dx, (activation blocks of 32 rows per tile, plan): bfloat16 dx has tiles of 32 mb rows, float32 dx of 16 mb
PLANS = [
    (38, 67, 192, BF16, 1, "whole"), (30, 201, 192, BF16, 1, "split"),
    (3326, 68, 1152, BF16, 2, "whole"), (1844, 2099, 576, BF16, 2, "split"), (3109, 330, 5248, BF16, 2, "mixed"),
    (4199, 70, 1856, BF16, 4, "whole"), (2218, 5375, 1088, BF16, 4, "split"), (1372, 354, 11840, BF16, 4, "mixed"),
    (30, 67, 192, F32, 2, "whole"), (32, 209, 192, F32, 2, "split"), (474, 282, 17664, F32, 2, "mixed"),
    (5568, 65, 576, F32, 4, "whole"), (1833, 2951, 576, F32, 4, "split"), (1195, 249, 6912, F32, 4, "mixed"),
]


def kind(full, tail):
    return "whole" if tail == 0 else "mixed" if full else "split"


@pytest.mark.parametrize("M,N,K,dxt,mb,plan", PLANS)
def test_the_shapes_reach_their_plans(M, N, K, dxt, mb, plan):
    got, full, tail, parts = grad_plan(M, N, K, 2 if dxt == F32 else 1)
    assert (got, kind(full, tail)) == (mb, plan) and (parts > 1) == (tail > 0)


def weights(fmt, N, K):
    """(w, scale, global scale, float64 dequantised [N, K] on the GPU)."""
    r = np.random.default_rng(N + K)
    if fmt == FP8:
        w = torch.from_numpy(r.integers(0, 256, (N, K)).astype(np.uint8))
        w[(w & 0x7F) == 0x7F] = 0x31                                    # no NaN codes
        s = torch.from_numpy((10.0 ** r.uniform(-4, -2, N)).astype(np.float32))
        return w.to(DEV), s.to(DEV), 1.0, (w.view(torch.float8_e4m3fn).double() * s.double()[:, None]).to(DEV)
    wp, ws, gs = synth.nvfp4_tensor(N, K, 29, 1)
    blk = oracle.block64_pack(wp, ws)
    return torch.from_numpy(blk).to(DEV), None, float(gs), torch.from_numpy(oracle.nvfp4_dequant(blk, gs)).to(DEV).double()


def check(fmt, M, N, K, dyt, dxt, seed=0):
    w, s, gs, dq = weights(fmt, N, K)
    g = torch.Generator(DEV).manual_seed(seed + M)
    dy = (torch.randn((M, N), device=DEV, generator=g) * 1e-3).to(dyt)
    dy[M // 2] *= 1024
    dy[M // 3] = 0
    got = wq.qlinear_backward(fmt, dy, w, s, gs, dtype=dxt)
    assert got.dtype == dxt and tuple(got.shape) == (M, K)
    dyd = dy.double()
    ref, size = dyd @ dq, dyd.abs() @ dq.abs()
    err = (got.double() - ref).abs()
    # dy's elements: one float16 rounding (2^-11 at most) or two terms (2^-22), FP8 scales one float32 rounding; subnormal
    # float16 values, 2^-25 where the row's largest is 2^14 or more; the sum of N products; dx's own rounding
    each = (2.0 ** -11 if dxt == BF16 else 2.0 ** -22) + 4 * U
    sc = s.double() if fmt == FP8 else torch.ones(N, device=DEV, dtype=torch.float64)
    floor = 2.0 ** -39 * (dyd * sc).abs().amax(1, keepdim=True) * (dq / sc[:, None]).abs().sum(0, keepdim=True)
    bound = (each + 2 * (N + 8) * U) * size + floor + torch.finfo(dxt).eps / 2 * ref.abs()
    assert bool((err <= bound).all())
    row = err.norm(dim=1) / ref.norm(dim=1).clamp_min(1e-300)
    # normwise, a float16 rounding of random signs is 2^-11 / sqrt(3) at most; times 4
    assert float(row.max()) <= norm_bound(N) + (2.0 ** -9 / np.sqrt(3) + torch.finfo(dxt).eps / 2 if dxt == BF16 else 2.0 ** -20)
    assert not bool(got[M // 3].any())


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", [FP8, NV], ids=["fp8", "nvfp4"])
@pytest.mark.parametrize("M,N,K,dxt,mb,plan", PLANS)
def test_plans(M, N, K, dxt, mb, plan, fmt):
    for dyt in (F32, BF16):
        print("[qlinear_backward]", M, N, K, fmt, dyt, dxt, mb, plan, flush=True)
        check(fmt, M, N, K, dyt, dxt)


@pytest.mark.gpu
@pytest.mark.parametrize("dyt,dxt", [(F32, F32), (BF16, BF16), (F32, BF16), (BF16, F32)])
@pytest.mark.parametrize("fmt", [FP8, NV], ids=["fp8", "nvfp4"])
@pytest.mark.parametrize("N", [6145, 18432, 18433, 26003])
def test_rows_longer_than_the_registers_hold(N, fmt, dyt, dxt):
    """dy rows on both sides of what a workgroup keeps in registers (6144 and 18432 elements)."""
    print("[qlinear_backward] N", N, fmt, dyt, dxt, flush=True)
    check(fmt, 37, N, 128, dyt, dxt)
