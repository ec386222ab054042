"""AdamW where the second moment or eps is small: float32 subnormals of v, eps far below 1e-8."""
import numpy as np
import pytest
import torch

import weight_quantized_mlp_amd as wq
from adapter_common import DEV, U, host
from test_adamw import scalars


@pytest.mark.gpu
@pytest.mark.parametrize("t", [1, 10, 10 ** 6])
@pytest.mark.parametrize("eps", [1e-8, 1e-18, 1e-30, 2.0 ** -126, 0.0])
def test_small_second_moments(eps, t):
    """Updates of lr m / (sqrt(v) + eps) down to v = 2^-148: the root of a subnormal is an ordinary number."""
    r = np.random.default_rng(t)
    n = 4096
    v0 = (2.0 ** r.uniform(-148, -60, n)).astype(np.float32)
    m0 = (np.sqrt(v0.astype(np.float64)) * r.uniform(-1, 1, n)).astype(np.float32)
    up = lambda a: torch.from_numpy(a.copy()).to(DEV)
    p, m, v = torch.zeros(n, device=DEV), up(m0), up(v0)
    step, lr = scalars(t, 1.0)
    wq.adamw_run(wq.adamw_table([p], [torch.zeros(n, device=DEV)], [m], [v]), step, lr, eps=eps, weight_decay=0.0)
    m1, v1 = 0.9 * m0.astype(np.float64), 0.999 * v0.astype(np.float64)
    want = -(m1 / (1 - 0.9 ** t)) / (np.sqrt(v1 / (1 - 0.999 ** t)) + eps)
    got = host(p).astype(np.float64)
    # about ten float32 operations of two half steps each; v is rounded to 2^-149 as it decays and as it is corrected,
    # and the root halves that
    rel = 32 * U + 2.0 ** -149 / v1
    assert np.all(np.abs(got - want) <= rel * np.abs(want))
    assert np.all(np.abs(host(v) - v1) <= 2.0 ** -150 + 2 * U * v1)


@pytest.mark.gpu
@pytest.mark.parametrize("eps", [1e-60, 1e-45, 1e-40, 2.0 ** -126, 1e-30, 1e-8])
@pytest.mark.parametrize("bits", [32, 8])
def test_elements_without_gradients_stay(bits, eps):
    n = 700
    z = lambda d: torch.zeros(n, dtype=d, device=DEV)
    p = torch.ones(n, device=DEV)
    states = ([z(torch.float32)], [z(torch.float32)]) if bits == 32 else ([z(torch.uint8)], [z(torch.uint8)])
    scales = () if bits == 32 else (None, [torch.ones(3, device=DEV)], [torch.ones(3, device=DEV)])
    step, lr = scalars(1, 1e-3)
    wq.adamw_run(wq.adamw_table([p], [z(torch.float32)], *states, *scales), step, lr, eps=eps, weight_decay=0.0)
    assert np.all(host(p) == 1)
