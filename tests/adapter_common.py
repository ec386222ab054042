"""Inputs and error bounds shared by the adapter, input-gradient and optimizer tests.

Bounds.  u = 2^-24 is half a float32 step.  A float32 sum of n products in any order is off by at most
(n + 1) u sum |products| to first order; an n-term matrix-core sum may round or truncate each step, which at most
doubles that.  `dot_bound` is that worst case for a chain of two products.  For inputs of random sign the
rounding errors add like a random walk, so the error of a whole matrix in the 2-norm stays near sqrt(n) u times its
norm; `norm_bound` is 8 times that, which a rounding of any operand to 16 bits (up to 2^-8 relative or 2^-11) exceeds.
"""
import numpy as np
import torch

U = 2.0 ** -24
DEV = torch.device("cuda:0")


def randn(seed, shape, dtype=torch.float32, std=1.0):
    """(device tensor, its values in float64)."""
    v = torch.from_numpy(np.random.default_rng(seed).standard_normal(shape) * std).to(dtype)
    return v.to(DEV), v.double().numpy()


def runs(seed, M, E, requests):
    """int32 adapter ids of M rows: `requests` runs of random lengths, ids in [-1, E)."""
    r = np.random.default_rng(seed)
    cuts = np.sort(r.integers(0, M + 1, max(requests - 1, 0)))
    return r.integers(-1, E, requests)[np.searchsorted(cuts, np.arange(M), side="right")].astype(np.int32)


def rel2(got, ref):
    """2-norm of the error over the 2-norm of the reference, in float64."""
    got, ref = np.asarray(got, dtype=np.float64), np.asarray(ref, dtype=np.float64)
    n = np.linalg.norm(ref)
    return np.linalg.norm(got - ref) / n if n else np.linalg.norm(got)


def norm_bound(*lengths):
    return 8 * U * np.sqrt(sum(lengths) + 16)


def host(t):
    return t.detach().float().cpu().numpy() if t.dtype in (torch.bfloat16, torch.float16) else t.detach().cpu().numpy()
