"""float64 references of the block calls (test infrastructure; plain loops and sums over NumPy arrays)."""
import numpy as np


def norm_ref(t, w, eps, offset):
    return t / np.sqrt(np.mean(t * t, axis=1, keepdims=True) + eps) * (offset + w)


def gate_rows(gate, M):
    """[M, H]: each gate row for its M / G consecutive rows; ones without a gate."""
    if gate is None:
        return 1.0
    g = np.atleast_2d(gate)
    return np.repeat(g, M // g.shape[0], axis=0)


def block_norm_ref(h, y, post, gate, alpha, pre, eps, offset, store=lambda v: v):
    """(h_out before its rounding, x).  store: rounds to the stream's type and back."""
    if y is not None:
        p = y if post is None else norm_ref(y, post, eps, offset)
        h = h + alpha * gate_rows(gate, h.shape[0]) * p
    return h, None if pre is None else norm_ref(store(h), pre, eps, offset)


def block_norm_backward_ref(h, y, dh, dx, post, gate, alpha, pre, eps, offset):
    """(dh_in, dy, dpost, dgate, dpre) for h as the forward call stored it; None where an input is absent."""
    M, H = h.shape
    du = np.zeros_like(h) if dh is None else dh.copy()
    dpre = dy = dpost = dgate = None
    if pre is not None:
        r = 1 / np.sqrt(np.mean(h * h, axis=1, keepdims=True) + eps)
        dn = dx * (offset + pre)
        du += r * dn - r ** 3 * h * np.mean(dn * h, axis=1, keepdims=True)
        dpre = np.sum(dx * h * r, axis=0)
    if y is not None:
        r = 1.0 if post is None else 1 / np.sqrt(np.mean(y * y, axis=1, keepdims=True) + eps)
        w = 1.0 if post is None else offset + post
        dp = alpha * gate_rows(gate, M) * du
        if gate is not None:
            g = np.atleast_2d(gate)
            dgate = np.sum((alpha * du * y * r * w).reshape(g.shape[0], M // g.shape[0], H), axis=1).reshape(np.shape(gate))
        if post is not None:
            dpost = np.sum(dp * y * r, axis=0)
            dy = r * dp * w - r ** 3 * y * np.mean(dp * w * y, axis=1, keepdims=True)
        else:
            dy = dp * 1.0
    return du, dy, dpost, dgate, dpre
