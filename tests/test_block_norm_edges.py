"""The norms around a block at the edges of what their header allows: in place with parts absent, and calls without rows."""
import pytest
import torch

import weight_quantized_mlp_amd as wq
from adapter_common import DEV, randn

F32, BF16 = torch.float32, torch.bfloat16
gpu = pytest.mark.gpu


@gpu
@pytest.mark.parametrize("ht", [F32, BF16])
@pytest.mark.parametrize("H", [320, 5120, 12000, 16392])          # one, two and four chunks per thread, rows read again
@pytest.mark.parametrize("post,gate,pre", [(False, False, True), (True, False, False), (False, True, True), (True, True, True)])
def test_in_place_with_absent_parts(H, ht, post, gate, pre):
    """h_out = h and dh_in = dh give the bits of separate outputs, whichever parts are there."""
    M = 300
    h, y = randn(1, (M, H), ht)[0], randn(2, (M, H), BF16)[0]
    kw = dict(post=randn(3, (H,))[0] if post else None, gate=randn(4, (3, H))[0] if gate else None, alpha=0.7,
              pre=randn(5, (H,))[0] if pre else None)
    ho, x = wq.block_norm_run(h, y, **kw)
    into = h.clone()
    a, b = wq.block_norm_run(into, y, h_out=into, **kw)
    assert a is into and torch.equal(a, ho) and (not pre or torch.equal(b, x))
    dh, dx = randn(6, (M, H), ht)[0], randn(7, (M, H), ht)[0] if pre else None
    apart = wq.block_norm_backward(ho, y, dh, dx, **kw)
    for p, q in zip(wq.block_norm_backward(ho, y, dh, dx, dh_in=dh, **kw), apart):
        assert q is None or torch.equal(p, q)


def test_no_rows_and_no_gate_rows():
    """A gate for every row of an empty batch has G = M = 0 rows; with rows, G = 0 is refused."""
    L, A, none = wq.lib(), 1 << 32, None
    fwd = lambda M, G: L.block_norm_run(M, 64, none, 0, none, 0, A, A, 0, none, G, 0, 1.0, 0.0, 1e-6, none, none, 0, none)
    bwd = lambda M, G: L.block_norm_backward(M, 64, none, 0, none, 0, none, none, 0, A, A, 0, none, G, 0, 1.0, 0.0, 1e-6, none, 0, none,
                                             none, none, none, none, none)
    assert fwd(0, 0) == 0 and bwd(0, 0) == 0 and L.block_norm_backward_workspace_bytes(0, 64, 0) == 0
    assert fwd(4, 0) == -1 and bwd(4, 0) == -1 and L.block_norm_backward_workspace_bytes(4, 64, 0) == 0
    assert fwd(0, -1) == -1 and bwd(0, -1) == -1


@gpu
def test_an_empty_batch_with_a_gate_for_every_row():
    e = torch.empty((0, 64), device=DEV)
    w = torch.ones(64, device=DEV)
    ho, x = wq.block_norm_run(e, e, post=w, gate=e, pre=w)
    assert ho.shape == x.shape == (0, 64)
    dh, dy, dpost, dgate, dpre = wq.block_norm_backward(e, e, e, e, post=w, gate=e, pre=w, dpost=torch.ones(64, device=DEV))
    assert dh.shape == dy.shape == dgate.shape == (0, 64)
    assert (dpost == 0).all() and (dpre == 0).all()
    with pytest.raises(ValueError, match="divisor"):
        wq.block_norm_run(torch.ones((4, 64), device=DEV), torch.ones((4, 64), device=DEV), gate=e)


@gpu
def test_the_most_rows_there_may_be():
    """2^23 rows of 512 threads each: 2^32 threads, more than a grid dimension holds.  Every row's result is there, those around the
    middle and at the ends are a small call's."""
    M, H = 1 << 23, 3592
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 2 * M * H * 2 + (8 << 30):
        pytest.skip("needs 129 GB of device memory")
    h = torch.empty((M, H), dtype=BF16, device=DEV).fill_(2.0)
    rows = torch.tensor([0, 1, (1 << 22) - 1, 1 << 22, M - 1], device=DEV)
    h[rows] = randn(1, (5, H), BF16)[0]
    w = torch.ones(H, dtype=BF16, device=DEV)
    x = torch.zeros_like(h)
    wq.block_norm_run(h, pre=w, x=x)
    few = wq.block_norm_run(h[rows].contiguous(), pre=w, x_dtype=BF16)[1]
    assert torch.equal(x[rows], few)
    x[rows] = 1.0
    for r in range(0, M, 1 << 18):                                  # 2 / sqrt(4 + 1e-6) rounds to 1
        assert bool((x[r:r + (1 << 18)] == 1.0).all()), r
    del h, x
    torch.cuda.empty_cache()


@gpu
def test_no_rows_and_many_gate_rows():
    """Without rows the gate's gradient is zeros, all 2^32 + 2^23 of them."""
    G, H = 1 << 20, 4104
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < G * H * 6 + (4 << 30):
        pytest.skip("needs 30 GB of device memory")
    e = torch.empty((0, H), dtype=BF16, device=DEV)
    gate, dgate = torch.zeros((G, H), dtype=BF16, device=DEV), torch.full((G, H), 3.0, device=DEV)
    got = wq.block_norm_backward(e, e, gate=gate, dgate=dgate)[3]
    assert got is dgate
    for r in range(0, G, 1 << 16):
        assert not bool(dgate[r:r + (1 << 16)].any()), r
    del gate, dgate, got
    torch.cuda.empty_cache()


@gpu
def test_sums_of_runs_keep_small_ones():
    """32 runs of a row each: a sum of 2^24 and 31 ones.  Added in pairs the chain has five roundings, each at most half of the spacing
    (2) of what it forms: off by 5 at most.  One after the other, every one of them would be lost."""
    h = torch.ones((32, 64), device=DEV)
    dx = torch.ones((32, 64), device=DEV)
    dx[3] = 2.0 ** 24
    kw = dict(post=torch.ones(64, device=DEV), gate=torch.ones((1, 64), device=DEV), pre=torch.zeros(64, device=DEV), eps=0.0)
    dpre = wq.block_norm_backward(h, h, h, dx, **kw)[4]
    assert ((dpre.double() - (2.0 ** 24 + 31)).abs() <= 5).all(), dpre[0].item()
    _, _, dpost, dgate, _ = wq.block_norm_backward(h, h, dx, h, **kw)         # pre = 0: du = dh
    assert ((dpost.double() - (2.0 ** 24 + 31)).abs() <= 5).all() and ((dgate.double() - (2.0 ** 24 + 31)).abs() <= 5).all()
