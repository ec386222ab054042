"""awq_linear_run against float64 on the dequantised weights.

Bounds.  u = 2^-24.  Weights and float16 rows enter the products exactly; a bfloat16 element is off by at most 2^-39 of its row's
largest, a float32 one by 2^-22 of itself or 2^-39 of its row's largest.  A float32 sum of n products is off by at most 2 (n + 8) u
times the sum of magnitudes (an n-term matrix-core sum may round or truncate each step; parts and terms add a few more).  That
worst case holds element by element; in the 2-norm of the whole result the roundings add like a random walk, so `norm_bound` (8 sqrt(n)
u) holds, too, which a rounding of any operand to 16 bits would break.
"""
import numpy as np
import pytest
import torch

import weight_quantized_mlp_amd as wq
from adapter_common import DEV, U, host, norm_bound, randn, rel2
from awq_common import awq_weights

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
pytestmark = pytest.mark.gpu


def check(y, x64, w64, xt, what=""):
    K = x64.shape[1]
    ref = x64 @ w64.T
    got = host(y).astype(np.float64)
    finite = np.where(np.isfinite(x64), np.abs(x64), 0)
    mag, most = np.abs(x64) @ np.abs(w64).T, finite.max(axis=1, keepdims=True) * np.abs(w64).sum(axis=1)[None]
    tol = 2 * (K + 8) * U * mag + 2.0 ** -140
    if xt != F16:
        tol += 2.0 ** -39 * most
    if xt == F32:
        tol += 2.0 ** -22 * mag
    worst = np.max(np.abs(got - ref) / tol)
    assert worst <= 1, f"{what}: {worst:.2f} of the bound"
    err = rel2(got, ref)
    assert err <= norm_bound(K), f"{what}: {err:.2e} > {norm_bound(K):.2e}"


# rows 1 and 2: each wave its own rows; 3 .. 32: shared rows, one and two column tiles; above: the tile kernel with 4 and 8 (also for rows
# of more than 1024 groups); N and K inside and past a tile, a step, a part; contractions long enough to be split
SHAPES = [(1, 512, 256), (1, 1, 32), (2, 67, 320), (15, 40, 96), (16, 16, 128), (17, 33, 160), (32, 64, 8192), (3, 40, 12320), (31, 4100, 288),
          (5, 16400, 64), (33, 67, 320), (64, 256, 544), (65, 255, 4096), (127, 300, 32), (129, 67, 320), (300, 515, 1056), (513, 1030, 512),
          (40, 48, 16384), (1, 40, 32800), (2, 17, 32768), (1, 130, 12320), (4, 129, 1056), (9, 127, 2080), (24, 300, 4128), (16, 17408, 1024)]


@pytest.mark.parametrize("xt", [F32, BF16, F16])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_shapes(M, N, K, xt):
    layout = 3 + (M + N + K) % 2
    print("[awq linear]", M, N, K, xt, layout, flush=True)
    bank, w = awq_weights(M + N, 1, N, K, layout)
    x, xd = randn(K, (M, K), xt)
    guard = torch.full((M * N + 64,), 7.0, device=DEV)               # nothing is written behind the result
    y = wq.awq_linear_run(x, bank, N, layout, out=guard[: M * N].view(M, N))
    assert (guard[M * N:] == 7.0).all()
    check(y, xd, w[0], xt)


# fewer weight rows than a tile of 16 has, one more or less than whole tiles; rows of one group, of a step and a part of one
@pytest.mark.parametrize("K", [32, 96, 160, 544])
@pytest.mark.parametrize("M,N", [(33, 1), (40, 7), (64, 15), (65, 17), (130, 5), (130, 255), (200, 257)])
def test_narrow_tiles(M, N, K):
    for xt, layout in ((BF16, 3), (F32, 4)):
        print("[awq linear]", M, N, K, xt, layout, flush=True)
        bank, w = awq_weights(M + N, 1, N, K, layout)
        x, xd = randn(K, (M, K), xt)
        guard = torch.full((M * N + 64,), 7.0, device=DEV)
        y = wq.awq_linear_run(x, bank, N, layout, out=guard[: M * N].view(M, N))
        assert (guard[M * N:] == 7.0).all()
        check(y, xd, w[0], xt)


@pytest.mark.parametrize("xt", [F32, F16])
def test_whole_and_cut_tiles(xt):
    """More tiles than the chip runs at once: the first rounds whole, the rest cut into parts."""
    M, N, K = 1100, 16400, 1056
    bank, w = awq_weights(7, 1, N, K, 3)
    x, xd = randn(8, (M, K), xt)
    guard = torch.full((M * N + 64,), 7.0, device=DEV)
    y = wq.awq_linear_run(x, bank, N, out=guard[: M * N].view(M, N))
    assert (guard[M * N:] == 7.0).all()
    check(y, xd, w[0], xt)


@pytest.mark.parametrize("M,N,K", [(1, 96, 512), (20, 96, 512), (80, 96, 512)])
def test_both_layouts_give_the_same_bits(M, N, K):
    x, _ = randn(1, (M, K), BF16)
    a, _ = awq_weights(3, 1, N, K, 3)
    b, _ = awq_weights(3, 1, N, K, 4)
    assert torch.equal(wq.awq_linear_run(x, a, N, 3), wq.awq_linear_run(x, b, N, 4))


def test_equals_the_debug_decoder():
    """One-hot rows read every weight out as the decoder gives it."""
    N, K = 64, 128
    bank, w = awq_weights(5, 1, N, K, 3)
    for M in (32, 128):
        for k0 in range(0, K, M):
            x = torch.zeros((M, K), device=DEV, dtype=F16)
            x[torch.arange(M), torch.arange(k0, k0 + M)] = 1
            y = wq.awq_linear_run(x, bank, N)
            assert torch.equal(y, wq.awq_dequant_f16(bank, 1, N, K)[0, :, k0:k0 + M].T.float())
            assert np.array_equal(host(y), w[0][:, k0:k0 + M].T.astype(np.float32))


@pytest.mark.parametrize("xt", [F32, BF16])
@pytest.mark.parametrize("M", [3, 70])
def test_range_of_the_rows(M, xt):
    """Rows of any size are scaled: near the largest and smallest float32, zeros, and a large element beside small ones."""
    N, K = 80, 384
    bank, w = awq_weights(6, 1, N, K, 4, std=0.5)
    v = np.random.default_rng(2).standard_normal((M, K))
    v[0] *= 1e36
    v[1] *= 1e-36
    v[2] = 0
    if M > 3:
        v[3, 5] = 2.0 ** 30
    x = torch.from_numpy(v).to(xt).to(DEV)
    y = wq.awq_linear_run(x, bank, N, 4)
    assert (y[2] == 0).all()
    xd = x.double().cpu().numpy()
    for m in range(M):
        if m != 2:
            check(y[m:m + 1], xd[m:m + 1], w[0], xt, f"row {m}")


@pytest.mark.parametrize("xt", [F32, BF16, F16])
@pytest.mark.parametrize("M", [1, 7, 40])
def test_infinities_and_nan_stay_in_their_row(M, xt):
    N, K = 48, 160                                                     # a last step of one group
    bank, w = awq_weights(8, 1, N, K, 3)
    x, xd = randn(4, (M, K), xt)
    clean = wq.awq_linear_run(x, bank, N)
    for value, at in ((float("inf"), K - 1), (float("nan"), 3), (-float("inf"), 130)):
        x2 = x.clone()
        x2[M - 1, at] = value
        y = wq.awq_linear_run(x2, bank, N)
        assert torch.equal(y[: M - 1], clean[: M - 1])
        col = w[0][:, at]
        with np.errstate(invalid="ignore"):
            np.testing.assert_array_equal(host(y[M - 1]), (np.sign(col) * value).astype(np.float32))     # 0 * inf is NaN


def test_an_infinite_scale_stays_in_its_row_of_weights():
    N, K, M = 32, 160, 5
    w0 = np.random.default_rng(1).standard_normal((1, N, K)).astype(np.float32)
    import oracle
    import synth
    codes, scales, zeros = synth.awq_quant(w0)
    s = scales.view(np.float16).copy()
    s[0, 4, 4] = np.inf                                                # the group of the last, short step
    broken = torch.from_numpy(oracle.awq_pack_bank(codes, s.view(np.uint16), zeros, 3)).to(DEV)
    whole = torch.from_numpy(oracle.awq_pack_bank(codes, scales, zeros, 3)).to(DEV)
    for M in (5, 50):
        x, _ = randn(1, (M, K), BF16)
        a, b = wq.awq_linear_run(x, broken, N), wq.awq_linear_run(x, whole, N)
        rest = [n for n in range(N) if n != 4]
        assert torch.equal(a[:, rest], b[:, rest]) and not torch.isfinite(a[:, 4]).any()


@pytest.mark.parametrize("M", [4, 32, 100])
def test_rows_do_not_see_each_other(M):
    """The same row at any place of a batch of this size gives the same bits."""
    N, K = 70, 1024
    bank, _ = awq_weights(9, 1, N, K, 3)
    x, _ = randn(3, (M, K), F32)
    y = wq.awq_linear_run(x, bank, N)
    turned = wq.awq_linear_run(x.flip(0).contiguous(), bank, N)
    assert torch.equal(y.flip(0), turned)


def test_weights_past_4_GiB():
    """Rows of weights, scales and zeros whose byte offsets pass 2^32."""
    N, K, M = (1 << 23) - 40, 1088, 2
    ng = K // 32
    nb = wq.awq_bank_bytes(1, N, K, 3)
    assert nb > (1 << 32) + (1 << 28)
    bank = torch.empty(nb, dtype=torch.uint8, device=DEV)
    for at in range(0, nb, 1 << 28):                                   # codes and zeros: any byte; the scales follow below
        n = min(1 << 28, nb - at)
        bank[at:at + n] = torch.randint(0, 256, (n,), dtype=torch.uint8, device=DEV)
    at1 = N * K // 2
    at2 = at1 + (2 * N * ng + 15) // 16 * 16
    for n0 in range(0, N, 1 << 21):
        n1 = min(N, n0 + (1 << 21))
        s = (torch.rand(((n1 - n0) * ng,), device=DEV) * 0.01 + 0.005).half()
        bank[at1 + 2 * n0 * ng: at1 + 2 * n1 * ng] = s.view(torch.uint8)
    x, xd = randn(1, (M, K), BF16)
    y = wq.awq_linear_run(x, bank, N)
    y40 = wq.awq_linear_run(torch.cat([x] * 20), bank, N)              # the tile kernel
    rows = np.array([0, 1, N // 2, N - 300, N - 2, N - 1])
    r = torch.from_numpy(rows).to(DEV)
    codes = bank[:at1].view(N, K // 2)[r].cpu().numpy()
    q = np.stack([codes & 15, codes >> 4], axis=2).reshape(len(rows), K)
    s = bank[at1:at1 + 2 * N * ng].view(torch.float16).view(N, ng)[r].cpu().numpy().astype(np.float64)
    z = bank[at2:at2 + N * ng].view(N, ng)[r].cpu().numpy().astype(np.float64)
    b = (-z * s).astype(np.float16).astype(np.float64)
    w = (q * np.repeat(s, 32, 1) + np.repeat(b, 32, 1)).astype(np.float16).astype(np.float64)
    check(y[:, r], xd, w, BF16)
    check(y40[38:, r], xd, w, BF16)


@pytest.mark.parametrize("M,N,K", [(1, 640, 8192), (40, 300, 2048)])
def test_a_replayed_graph_reads_new_values(M, N, K):
    bank, _ = awq_weights(2, 1, N, K, 3)
    x, _ = randn(1, (M, K), BF16)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        wq.awq_linear_run(x, bank, N)
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = wq.awq_linear_run(x, bank, N)
    for i in range(3):
        x.copy_(randn(20 + i, (M, K), BF16)[0])
        want = wq.awq_linear_run(x, bank, N)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)


def test_empty_and_refused_calls():
    bank, _ = awq_weights(2, 1, 48, 64, 3)
    assert wq.awq_linear_run(torch.empty((0, 64), device=DEV), bank, 48).shape == (0, 48)
    x, _ = randn(1, (4, 64), F32)
    with pytest.raises(TypeError):
        wq.awq_linear_run(x.double(), bank, 48)
    with pytest.raises(ValueError):
        wq.awq_linear_run(x, bank, 49)
    with pytest.raises(ValueError):
        wq.awq_linear_run(x, bank, 48, meta_layout=4)
    with pytest.raises(ValueError, match="contiguous"):
        wq.awq_linear_run(x.t().contiguous().t(), bank, 48)
    assert wq.awq_linear_workspace_bytes(40, 48, 64, F32) > 64          # rows that are packed first
    with pytest.raises(wq.WQError):
        wq.awq_linear_run(x.repeat(10, 1), bank, 48, workspace=torch.empty(64, dtype=torch.uint8, device=DEV))
    with pytest.raises(wq.WQError):
        wq.awq_linear_run(x, bank, 48, out=x.view(-1)[:192].view(4, 48))
