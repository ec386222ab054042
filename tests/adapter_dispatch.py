"""The library's rules that choose a kernel, restated, so that a test can assert which one its shape reaches.

Sources: lora_common.h (few_rows), lora_expand.hip (one_launch), lora_shrink.hip (shrink_parts), lora_outer.hip
(outer_*), linear_grad.hip (grad_plan).  A test that fails here after a rule changed needs another shape, not another
rule: its point is the kernel that it names.
"""


def up(a, b):
    return -(-a // b)


def few_rows(M, K, N, R, ws):
    """ws: bytes of an adapter's element.  True: the row kernels; False: the 32-row tiles."""
    mr = M * max(R, 16)
    return mr <= 16384 and mr * (K + N) * ws <= 300000000


def one_launch(M, K, N, R):
    return K * R <= 8192 and K * R * M * up(N, 256) <= 4 << 20


def shrink_parts(M, D, R, es, ws):
    """Parts of a tiled contraction over D (es: bytes of an element of the rows, ws: of the adapter's)."""
    tiles = up(M, 32) * up(R, 64)
    xb, wb = 32 * D * es, min(R, 64) * D * ws
    if tiles == 0 or tiles >= 256 or (xb <= 512 << 10 and xb + wb <= (512 << 10 if tiles <= 32 else 1536 << 10)):
        return 1
    s = min(8, 512 // tiles)
    if s <= 1:
        return 1
    nb = up(D, 64)
    return up(nb, up(nb, s))


def outer_tiles(D, E, R):
    return E * up(D, 64) * up(R, 16 if R <= 16 else 32 if R <= 32 else 64)


def outer_part_rows(M, parts):
    return up(up(max(M, 1), parts), 32) * 32


def outer_parts(M, D, E, R):
    """Parts of the rows of one weight gradient."""
    tiles, best, least = outer_tiles(D, E, R), 1, 1e30
    for p in range(1, 9):
        if p > 1 and M // p < 256:
            break
        if p > 1 and up(M, outer_part_rows(M, p)) != p:
            continue
        cost = up(tiles * p, 768) * 768 / (tiles * p) * M * 2.0 * D + (p * 8.0 * E * R * D if p > 1 else 0.0) + 28672.0 * tiles * p
        if cost < least:
            least, best = cost, p
    return best


def outer_one_wave(M, D, E, R):
    p = outer_parts(M, D, E, R)
    return outer_tiles(D, E, R) * p > 768 and outer_part_rows(M, p) <= max(32, 16 * min(E, 16))


def grad_plan(M, N, K, terms):
    """(activation blocks of 32 rows, whole tiles, split tiles, parts of each) of qlinear_backward's GEMM."""
    best, least = None, 1e30
    mb = 4
    while mb >= terms:
        bm = 32 * mb // terms
        if not (mb > terms and M <= bm // 2):
            tiles, steps = up(M, bm) * up(K, 256), up(N, 64)
            step_us = lambda wgs: max(0.9, 0.55 * min(2, up(wgs, 256)) * (0.25 + 0.1875 * mb))
            for split in (0, 1):
                tail = tiles % 512 if split else 0
                if split and tail == 0:
                    continue
                full = tiles - tail
                body = up(full, 512) * (steps * step_us(full) + 1.2 * mb) if full else 0.0
                for s in range(2, min(steps, max(1, 512 // tail)) + 1) if split else (1,):
                    per = up(steps, s)
                    S = up(steps, per) if split else 1
                    size = tail * S * bm * 256 * 4.0
                    if size > 64 << 20:
                        break
                    us = body + (per * step_us(tail * S) + 1.2 * mb + 2.5 + size * 2 / 4.5e6 if split else 0.0)
                    if us < least:
                        least, best = us, (mb, full, tail, S)
        mb //= 2
    return best
