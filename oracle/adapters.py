"""Low-rank adapters, input gradient and AdamW (oracle; test infrastructure only).

Definitions: include/wqmlp_adapters.h.  Everything is float64 except adamw8_ref, which follows the 8-bit
state form step by step in float32 (its codes are defined by float32 operations, each rounded by itself).
"""
import numpy as np


def lora_ref(x, a, b, scale, ids, y):
    """out[m] = y[m] + scale[e] (x[m] a[e]^T) b[e]^T, e = ids[m]; rows with ids outside [0, E) keep y."""
    x, a, b = (np.asarray(t, dtype=np.float64) for t in (x, a, b))
    out = np.array(y, dtype=np.float64)
    for e in range(a.shape[0]):
        at = np.flatnonzero(np.asarray(ids) == e)
        if at.size:
            out[at] += float(scale[e]) * ((x[at] @ a[e].T) @ b[e].T)
    return out


def lora_backward_ref(dy, x, a, b, scale, ids, dx0):
    """Gradients (dx, da, db) of lora_ref for the output gradient dy."""
    dy, x, a, b = (np.asarray(t, dtype=np.float64) for t in (dy, x, a, b))
    dx = np.array(dx0, dtype=np.float64)
    da, db = np.zeros_like(a), np.zeros_like(b)
    for e in range(a.shape[0]):
        at = np.flatnonzero(np.asarray(ids) == e)
        if at.size:
            s = float(scale[e])
            dt = s * (dy[at] @ b[e])
            da[e] = dt.T @ x[at]
            db[e] = s * (dy[at].T @ (x[at] @ a[e].T))
            dx[at] += dt @ a[e]
    return dx, da, db


def adamw_ref(p, g, m, v, t, lr, beta1, beta2, eps, weight_decay, grad_scale=1.0):
    """One AdamW step in float64: (p, m, v)."""
    p, g, m, v = (np.asarray(u, dtype=np.float64) for u in (p, g, m, v))
    g = g * grad_scale
    m = beta1 * m + (1 - beta1) * g
    v = beta2 * v + (1 - beta2) * g * g
    p = p * (1 - lr * weight_decay) - lr * (m / (1 - beta1 ** t)) / (np.sqrt(v / (1 - beta2 ** t)) + eps)
    return p, m, v


def _mix(h):
    h = np.asarray(h, dtype=np.uint64) & np.uint64(0xFFFFFFFF)
    low = np.uint64(0xFFFFFFFF)
    h ^= h >> np.uint64(16)
    h = (h * np.uint64(0x7FEB352D)) & low
    h ^= h >> np.uint64(15)
    h = (h * np.uint64(0x846CA68B)) & low
    return h ^ (h >> np.uint64(16))


def adamw_random_bits(n, seed, t, tensor):
    """(low, high) 16 random bits of each of a tensor's n elements at step t."""
    key = int(_mix((int(_mix((seed + 0x9E3779B9 * t) & 0xFFFFFFFF)) + tensor) & 0xFFFFFFFF))
    h = _mix((np.uint64(key) + np.arange(n, dtype=np.uint64) * np.uint64(0x9E3779B9)) & np.uint64(0xFFFFFFFF))
    return (h & np.uint64(0xFFFF)).astype(np.int64), (h >> np.uint64(16)).astype(np.int64)


def _grid(mant, emin, count):
    """Non-negative finite values of an 8-bit float with `mant` mantissa bits, smallest normal 2^emin: codes 0..count-1."""
    c = np.arange(count)
    ex, fr = c >> mant, c & ((1 << mant) - 1)
    return np.where(ex == 0, fr * 2.0 ** (emin - mant), (1 + fr / 2.0 ** mant) * 2.0 ** (emin + ex - 1.0))


E4M3_GRID, E5M2_GRID = _grid(3, -6, 127), _grid(2, -14, 124)


def stochastic_code(x, r, grid):
    """Code of x >= 0 on an ascending grid: the upper neighbour where the position between the neighbours, in units
    of 2^-16 (truncated), plus r reaches 2^16."""
    lo = np.searchsorted(grid, x, side="right") - 1
    hi = np.minimum(lo + 1, grid.size - 1)
    gap = np.where(hi > lo, grid[hi] - grid[lo], 1.0)
    pos = np.floor((x - grid[lo]) / gap * 65536.0)
    return np.where(pos + r >= 65536, hi, lo)


def adamw8_states(mc, ms, vc, vs, g, t, beta1, beta2, seed, tensor, grad_scale=1.0, block=256, keep_v=False):
    """New 8-bit states: (m codes, m scales, v codes, v scales, m, v), m and v the float32 states before rounding.
    The state updates are float32 operations, each rounded by itself.  keep_v: a positive v keeps a positive code."""
    f = np.float32
    n = mc.size
    at = np.arange(n) // block
    sign = np.where(mc & 0x80, f(-1), f(1))
    m = (sign * E4M3_GRID[mc & 0x7F].astype(f)) * ms[at]
    v = E5M2_GRID[vc & 0x7F].astype(f) * vs[at]
    g = np.asarray(g, dtype=f) * f(grad_scale)
    m = m * f(beta1) + g * f(1 - beta1)
    v = v * f(beta2) + (g * g) * f(1 - beta2)
    rm, rv = adamw_random_bits(n, seed, t, tensor)
    out = []
    for x, r, grid, most in ((m, rm, E4M3_GRID, 448.0), (v, rv, E5M2_GRID, 57344.0)):
        nb = (n + block - 1) // block
        amax = np.array([np.max(np.abs(x[block * i:block * (i + 1)])) for i in range(nb)], dtype=np.float64)
        e = np.zeros(nb)
        pos = amax > 0
        e[pos] = np.clip(np.ceil(np.log2(amax[pos] / most)), -100, 100)
        # log2 may be off by an ulp at a power of two: the smallest e with amax <= most 2^e
        e[pos & (amax > most * 2.0 ** e)] += 1
        e[pos & (amax <= most * 2.0 ** (e - 1)) & (e > -100)] -= 1
        sc = 2.0 ** e
        code = stochastic_code(np.abs(x).astype(np.float64) / sc[at], r, grid)
        if keep_v and grid is E5M2_GRID:
            code = np.where(x > 0, np.maximum(code, 1), code)
        out += [(code | np.where(np.signbit(x), 0x80, 0)).astype(np.uint8), sc.astype(f)]
    return out[0], out[1], out[2], out[3], m, v
