"""A SwiGLU MLP with adapters on gate, up and down, forward and backward, built from the single calls (the fused MLP calls
take no adapters): qlinear_run + lora_run per projection, the activation and its gradient in torch, qlinear_backward and
lora_backward chained through dx0.  Every step is compared with float64 on that step's own inputs."""
import numpy as np
import pytest
import torch

import oracle
import synth
import weight_quantized_mlp_amd as wq
from adapter_common import DEV, U, host, norm_bound, randn, rel2
from adapter_dispatch import few_rows, one_launch
from test_lora import ids_for

F32, BF16 = torch.float32, torch.bfloat16
E = 4
SIZES = [(300, 256, 512, 64), (19, 512, 256, 16)]                       # rows, hidden, intermediate, rank: tiles, row kernels


def test_the_sizes_reach_both_kinds_of_kernel():
    tiled = [not few_rows(M, H, I, R, 2) and not one_launch(M, H, I, R) and not one_launch(M, I, H, R) for M, H, I, R in SIZES]
    assert tiled == [True, False]


def projection(fmt, N, K, seed):
    """(w, scale, global scale) and the float64 dequantised [N, K]."""
    if fmt == wq.WQ_FMT_FP8W:
        w0 = np.random.default_rng(seed).standard_normal((N, K)).astype(np.float32) * 0.05
        s = (np.abs(w0).max(axis=1) / 448).astype(np.float32)
        codes = synth.to_e4m3_codes(w0 / s[:, None])
        return (torch.from_numpy(codes).to(DEV), torch.from_numpy(s).to(DEV), 1.0), oracle.fp8w_dequant(codes, s).astype(np.float64)
    wp, ws, gs = synth.nvfp4_tensor(N, K, 50 + seed, 1)
    blk = oracle.block64_pack(wp, ws)
    return (torch.from_numpy(blk).to(DEV), None, float(gs)), oracle.nvfp4_dequant(blk, gs).astype(np.float64)


class Linear:
    """One frozen projection and its adapters; a float64 twin checks every call."""

    def __init__(self, fmt, N, K, R, seed):
        self.fmt, (self.w, self.dq) = fmt, projection(fmt, N, K, seed)
        self.a, self.ad = randn(seed, (E, R, K), BF16, K ** -0.5)
        self.b, self.bd = randn(seed + 100, (E, N, R), BF16, 0.2)
        self.sc = np.linspace(0.5, 2.0, E).astype(np.float32)
        self.scale, self.R = torch.from_numpy(self.sc).to(DEV), R

    def forward(self, x, ids):
        y = wq.qlinear_run(self.fmt, x, *self.w)
        base = host(y).astype(np.float64)
        # the projection takes x as float16 (2^-11 of each element)
        assert rel2(base, host(x).astype(np.float64) @ self.dq.T) <= 2.0 ** -9
        wq.lora_run(x, self.a, self.b, self.scale, ids, y, out=y)
        ref = oracle.lora_ref(host(x), self.ad, self.bd, self.sc, ids.cpu().numpy(), base)
        part = np.linalg.norm(ref - base) / np.linalg.norm(ref)
        assert rel2(host(y), ref) <= norm_bound(x.shape[1], self.R) * part + 2 * U
        return y

    def backward(self, dy, x, ids, dx0=None):
        """dx is dx0 + the projection's and the adapters' parts."""
        dx = wq.qlinear_backward(self.fmt, dy, *self.w, dtype=F32)
        if dx0 is not None:
            dx += dx0
        before = host(dx).astype(np.float64)
        dx, da, db = wq.lora_backward(dy, x, self.a, self.b, self.scale, ids, dx, dx)
        dyd, N = host(dy).astype(np.float64), dy.shape[1]
        M, K = x.shape
        want = dyd @ self.dq + (0 if dx0 is None else host(dx0))
        assert rel2(before, want) <= norm_bound(N) + 2.0 ** -20
        rx, ra, rb = oracle.lora_backward_ref(dyd, host(x), self.ad, self.bd, self.sc, ids.cpu().numpy(), before)
        assert rel2(host(dx), rx) <= norm_bound(N, self.R) + 2 * U
        assert rel2(host(da), ra) <= norm_bound(N, M) and rel2(host(db), rb) <= norm_bound(K, M)
        return dx, da, db


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["runs", "random"])
@pytest.mark.parametrize("fmt", [wq.WQ_FMT_FP8W, wq.WQ_FMT_NVFP4], ids=["fp8", "nvfp4"])
@pytest.mark.parametrize("M,H,I,R", SIZES)
def test_mlp_with_adapters(M, H, I, R, fmt, kind):
    print("[adapter mlp]", M, H, I, R, fmt, kind, flush=True)
    gate, up, down = Linear(fmt, I, H, R, 1), Linear(fmt, I, H, R, 2), Linear(fmt, H, I, R, 3)
    x, _ = randn(7, (M, H), BF16)
    ids = torch.from_numpy(ids_for(kind, M, E, 3)).to(DEV)
    g, u = gate.forward(x, ids), up.forward(x, ids)
    s = torch.sigmoid(g)
    act = g * s * u
    out = down.forward(act, ids)
    dout = out / M                                                      # the gradient of |out|^2 / 2M
    dact, _, _ = down.backward(dout, act, ids)
    dx, _, _ = gate.backward(dact * u * (s + g * s * (1 - s)), x, ids)
    dx, _, _ = up.backward(dact * g * s, x, ids, dx)
    assert torch.isfinite(dx).all()

    # the whole chain against differences of the loss, in float64 on the dequantised weights
    def loss(xd):
        def lin(p, z):
            return oracle.lora_ref(z, p.ad, p.bd, p.sc, ids.cpu().numpy(), z @ p.dq.T)
        gd = lin(gate, xd)
        return np.sum(lin(down, gd / (1 + np.exp(-gd)) * lin(up, xd)) ** 2) / (2 * M)
    xd, dxd = host(x).astype(np.float64), host(dx).astype(np.float64)
    norm = np.linalg.norm(dxd)
    other = np.random.default_rng(0).standard_normal((M, H))
    for d in (dxd / norm, other / np.linalg.norm(other)):
        slope = (loss(xd + 1e-4 * d) - loss(xd - 1e-4 * d)) / 2e-4
        # float16 roundings of at most 2^-11 of each projection's input, three in a row and once more in each factor of the
        # gradient, each grown a few times by the layers: 2% covers ten of them at four times, and a part left out is more
        assert abs(np.sum(dxd * d) - slope) <= 0.02 * norm
