"""Adapters on a frozen quantised projection, trained as a program would: forward (qlinear_run + lora_run), the loss's
gradient, backward (qlinear_backward + lora_backward) and adamw_run on the adapters, whose bfloat16 copies the next
forward reads.  Every step's gradients are compared with the float64 oracle's at the same weights."""
import numpy as np
import pytest
import torch

import oracle
import synth
import weight_quantized_mlp_amd as wq
from adapter_common import DEV, host, norm_bound, randn, rel2, runs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("fmt", [wq.WQ_FMT_FP8W, wq.WQ_FMT_NVFP4], ids=["fp8", "nvfp4"])
def test_training_steps(fmt, bits):
    M, K, N, E, R = 150, 256, 192, 3, 16
    if fmt == wq.WQ_FMT_FP8W:
        w0 = np.random.default_rng(0).standard_normal((N, K)).astype(np.float32) * 0.05
        s = (np.abs(w0).max(axis=1) / 448).astype(np.float32)
        codes = synth.to_e4m3_codes(w0 / s[:, None])
        dq = oracle.fp8w_dequant(codes, s).astype(np.float64)
        W = (torch.from_numpy(codes).to(DEV), torch.from_numpy(s).to(DEV), 1.0)
    else:
        wp, ws, gs = synth.nvfp4_tensor(N, K, 41, 1)
        blk = oracle.block64_pack(wp, ws)
        dq = oracle.nvfp4_dequant(blk, gs).astype(np.float64)
        W = (torch.from_numpy(blk).to(DEV), None, float(gs))
    x, xd = randn(1, (M, K), torch.bfloat16)
    target, td = randn(2, (M, N))
    ids_h = runs(3, M, E, 6)
    ids_h[:3] = (0, 1, 2)
    ids = torch.from_numpy(ids_h).to(DEV)
    sc_h = np.array([2.0, 1.0, 0.5], dtype=np.float32)
    sc = torch.from_numpy(sc_h).to(DEV)
    a, b = randn(4, (E, R, K), std=K ** -0.5)[0], torch.zeros((E, N, R), device=DEV)
    a16, b16 = a.to(torch.bfloat16), b.to(torch.bfloat16)
    da, db = torch.empty_like(a), torch.empty_like(b)
    state = lambda dt: [torch.zeros(t.shape, dtype=dt, device=DEV) for t in (a, b)]
    if bits == 8:
        m, v = ([t.view(d) for t in state(torch.uint8)] for d in (torch.float8_e4m3fn, torch.float8_e5m2))
        scales = [[torch.ones((t.numel() + 255) // 256, device=DEV) for t in (a, b)] for _ in range(2)]
    else:
        m, v, scales = state(torch.float32), state(torch.float32), (None, None)
    table = wq.adamw_table([a, b], [da, db], m, v, [a16, b16], *scales)
    step, lr = torch.zeros(1, dtype=torch.int64, device=DEV), torch.full((1,), 1e-2, device=DEV)
    for t in range(4):
        ad, bd = a16.double().cpu().numpy(), b16.double().cpu().numpy()
        y = wq.qlinear_run(fmt, x, *W)
        base = host(y).astype(np.float64)
        wq.lora_run(x, a16, b16, sc, ids, y, out=y)
        assert rel2(host(y), oracle.lora_ref(xd, ad, bd, sc_h, ids_h, base)) <= norm_bound(K, R)
        dy = (y - target) / M                                           # the gradient of |y - target|^2 / 2M
        dyd = host(dy).astype(np.float64)
        dx = wq.qlinear_backward(fmt, dy, *W)
        wq.lora_backward(dy, x, a16, b16, sc, ids, dx, dx, da, db)
        rx, ra, rb = oracle.lora_backward_ref(dyd, xd, ad, bd, sc_h, ids_h, dyd @ dq)
        assert rel2(host(dx), rx) <= norm_bound(N, N, R) + 2.0 ** -20
        assert rel2(host(da), ra) <= norm_bound(N, M) and rel2(host(db), rb) <= norm_bound(K, M)
        assert t > 0 or not host(da).any()                              # b = 0 at the start: only b learns
        before = a.clone(), b.clone()
        step += 1
        wq.adamw_run(table, step, lr, seed=t)
        assert torch.equal(a16, a.to(torch.bfloat16)) and torch.equal(b16, b.to(torch.bfloat16))
        assert not torch.equal(b, before[1]) and torch.isfinite(a).all() and torch.isfinite(b).all()
