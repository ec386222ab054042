"""8-bit states, with and without keep_v, of blocks in which one element's gradients are far larger than the others'.

m's codes reach to 2^-18 of a block's largest, v's to 2^-32, which is 2^-16 in gradient.  An element between the two keeps
an m; with keep_v its v does not become zero either, and the step not a division by the newest gradient alone.

However its gradients run, an element with float32 states never moves by more than lr (1 - beta1) / sqrt((1 - beta2)
(1 - beta1^2 / beta2)) = 7.27 lr (m and v are sums of g and g^2 with weights (1 - beta1) beta1^i and (1 - beta2) beta2^i;
Cauchy-Schwarz).  The 8-bit states of these gradients, which give float32 states at most 1.5 lr, add to m at most a code
step, 2^-9 of a scale of at most 1 / 224 of the largest m, and keep sqrt(v) above 2^-16 of the largest: 0.6 lr more at
most, and a v one code down is half at least.  So no step passes that limit.
"""
import functools

import numpy as np
import pytest
import torch

import oracle
from test_adamw import HYPER, check_step, scalars, snapshot, states
import weight_quantized_mlp_amd as wq

LIMIT = 0.1 / np.sqrt(0.001 * (1 - 0.81 / 0.999))


def gradients(r, n, bits, signed):
    g = r.standard_normal(n)
    g = g if signed else np.abs(g)
    return np.where(np.arange(n) % 256 == 0, np.abs(g) + 1, g * 2.0 ** -bits).astype(np.float32) * np.float32(1e-3)


@pytest.mark.parametrize("signed", [False, True])
@pytest.mark.parametrize("bits", [0, 12, 14, 16, 18, 24])
def test_kept_steps_stay_within_those_of_float32_states(bits, signed):
    n = 16 * 256
    r = np.random.default_rng(bits)
    mc, vc = np.zeros(n, dtype=np.uint8), np.zeros(n, dtype=np.uint8)
    ms, vs = np.ones(n // 256, dtype=np.float32), np.ones(n // 256, dtype=np.float32)
    for t in range(1, 151):
        g = gradients(r, n, bits, signed)
        mc, ms, vc, vs, m, v = oracle.adamw8_states(mc, ms, vc, vs, g, t, 0.9, 0.999, 5, 0, keep_v=True)
        step = np.abs(m / (1 - 0.9 ** t)) / np.sqrt(v.astype(np.float64) / (1 - 0.999 ** t))
        assert step.max() <= LIMIT, t
        assert not ((vc == 0) & (v > 0)).any()


def test_refusals():
    x = torch.zeros(4)
    with pytest.raises(ValueError, match="keep_v"):
        wq.adamw_table([x], [x], [x], [x], keep_v=True)                 # float32 states
    A, MB = 1 << 32, 1 << 20
    t = (wq._AdamWTensor * 1)(wq._AdamWTensor(1000, *(A + MB * i for i in range(6)), None, 0, 1))
    for bits in (32 | wq.WQ_ADAMW_KEEP_V, wq.WQ_ADAMW_KEEP_V, 8 | 512):
        assert wq.lib().adamw_table_build(1, t, bits, A - MB, MB, None) == -1
    assert wq.lib().adamw_table_build(1, t, 8 | wq.WQ_ADAMW_KEEP_V, A - MB, 8, None) == -6      # its size is checked next


@pytest.mark.gpu
@pytest.mark.parametrize("keep", [False, True])
@pytest.mark.parametrize("bits", [14, 16, 18, 24, 40])
def test_kernel_states_of_uneven_blocks(bits, keep, monkeypatch):
    """Bit for bit the oracle's states, step after step, from zero states (as check_step compares them)."""
    monkeypatch.setattr(oracle, "adamw8_states", functools.partial(oracle.adamw8_states, keep_v=keep))
    n = 5 * 256 + 77
    s = states([n, 300], 8, torch.float32, torch.bfloat16, seed=bits)
    s["table"] = wq.adamw_table(s["p"], s["g"], s["m"], s["v"], s["copy"], s["ms"], s["vs"], keep_v=keep)
    for key in ("m", "v"):
        for t in s[key]:
            t.view(torch.uint8).zero_()
    r = np.random.default_rng(bits)
    before = snapshot(s)
    for t in range(1, 31):
        for g in s["g"]:
            g.copy_(torch.from_numpy(gradients(r, g.numel(), bits, t % 2 == 0)))
        before["g"] = [g.cpu().numpy() for g in s["g"]]
        step, lr = scalars(t, 1e-3)
        wq.adamw_run(s["table"], step, lr, seed=5, **HYPER)
        before = check_step(before, s, t, 1e-3, 5)
    v = np.concatenate(before["v"])
    assert (v > 0).all() == keep or bits < 16                           # every element had a gradient


@pytest.mark.gpu
def test_kept_states_of_values_that_are_not_finite():
    """NaN and infinite v are NaN codes, zeros stay zero."""
    n = 300
    z = lambda d: torch.zeros(n, dtype=d, device="cuda:0")
    g, m, v = z(torch.float32), z(torch.uint8), z(torch.uint8)
    g[:4] = torch.tensor([float("inf"), float("nan"), 1.0, 1e-12], device="cuda:0")
    sc = [torch.ones(2, device="cuda:0") for _ in range(2)]
    step, lr = scalars(1, 1e-3)
    wq.adamw_run(wq.adamw_table([z(torch.float32)], [g], [m], [v], None, sc[:1], sc[1:], keep_v=True), step, lr, **HYPER)
    v = v.cpu().numpy()
    assert np.all(v[:2] > 0x7B) and 0 < v[2] <= 0x7B and v[3] == 1 and not v[4:].any()
