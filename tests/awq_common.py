"""Seeded AWQ weights shared by the tests of the 4-bit linear and the routed experts."""
import numpy as np
import torch

import oracle
import synth
from adapter_common import DEV


def awq_weights(seed, E, N, K, layout, std=0.02):
    """(bank on the GPU, float64 [E, N, K])."""
    w = np.random.default_rng(seed).standard_normal((E, N, K)).astype(np.float32) * np.float32(std)
    codes, scales, zeros = synth.awq_quant(w)
    bank = torch.from_numpy(np.ascontiguousarray(oracle.awq_pack_bank(codes, scales, zeros, layout))).to(DEV)
    return bank, dequant(codes, scales, zeros)


def dequant(codes, scales, zeros):
    """float64 of RN_f16(q scale + RN_f16(-zero scale)); every product and sum before a rounding is exact in float64."""
    s = scales.view(np.float16).astype(np.float64)
    b = (-zeros.astype(np.float64) * s).astype(np.float16).astype(np.float64)
    v = codes.astype(np.float64) * np.repeat(s, 32, axis=-1) + np.repeat(b, 32, axis=-1)
    return v.astype(np.float16).astype(np.float64)
