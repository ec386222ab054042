"""adamw_table / adamw_run against the float64 step and the bit-exact 8-bit state form."""
import numpy as np
import pytest
import torch

import oracle
import weight_quantized_mlp_amd as wq
from adapter_common import DEV, U, host, rel2

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
HYPER = dict(beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01)


def states(sizes, bits, gt, copy, seed=0):
    r = np.random.default_rng(seed)
    up = lambda a, d=F32: torch.from_numpy(np.ascontiguousarray(a)).to(d).to(DEV)
    s = dict(p=[], g=[], m=[], v=[], ms=[], vs=[], copy=[], bits=bits)
    for n in sizes:
        s["p"].append(up(r.standard_normal(n) * 0.02))
        s["g"].append(up(r.standard_normal(n) * 10.0 ** r.uniform(-5, -1, n), gt))
        if bits == 32:
            s["m"].append(up(r.standard_normal(n) * 1e-3))
            s["v"].append(up(r.standard_normal(n) ** 2 * 1e-6))
        else:
            nb = (n + 255) // 256
            mc = r.integers(0, 256, n).astype(np.uint8)
            mc[(mc & 0x7F) == 0x7F] = 0x05                              # no NaN codes
            s["m"].append(torch.from_numpy(mc).to(DEV).view(torch.float8_e4m3fn))
            s["v"].append(torch.from_numpy(r.integers(0, 124, n).astype(np.uint8)).to(DEV).view(torch.float8_e5m2))
            s["ms"].append(up(2.0 ** r.integers(-24, -12, nb)))
            s["vs"].append(up(2.0 ** r.integers(-50, -30, nb)))
        if copy is not None:
            s["copy"].append(torch.zeros(n, dtype=copy, device=DEV))
    s["table"] = wq.adamw_table(s["p"], s["g"], s["m"], s["v"], s["copy"] or None, s["ms"] or None, s["vs"] or None)
    return s


def snapshot(s):
    codes = lambda ts: [t.view(torch.uint8).cpu().numpy().copy() if t.dtype not in (F32,) else host(t).copy() for t in ts]
    return dict(p=[host(t).copy() for t in s["p"]], g=[host(t).copy() for t in s["g"]], m=codes(s["m"]), v=codes(s["v"]),
                ms=[host(t).copy() for t in s["ms"]], vs=[host(t).copy() for t in s["vs"]])


def scalars(t, lr):
    return torch.tensor([t], dtype=torch.int64, device=DEV), torch.tensor([lr], device=DEV)


def check_step(before, s, t, lr, seed, grad_scale=1.0):
    after = snapshot(s)
    for i, p in enumerate(before["p"]):
        if s["bits"] == 8:
            mc, ms, vc, vs, m, v = oracle.adamw8_states(before["m"][i], before["ms"][i], before["v"][i], before["vs"][i],
                                                        before["g"][i], t, HYPER["beta1"], HYPER["beta2"], seed, i, grad_scale)
            assert np.array_equal(after["ms"][i], ms) and np.array_equal(after["vs"][i], vs), i
            assert np.array_equal(after["m"][i], mc) and np.array_equal(after["v"][i], vc), i
            lr64 = float(np.float32(lr))
            upd = (m.astype(np.float64) / (1 - HYPER["beta1"] ** t)) / (np.sqrt(v.astype(np.float64) / (1 - HYPER["beta2"] ** t)) + HYPER["eps"])
            want = p.astype(np.float64) * (1 - lr64 * HYPER["weight_decay"]) - lr64 * upd
        else:
            want, m, v = oracle.adamw_ref(p, before["g"][i], before["m"][i], before["v"][i], t, float(np.float32(lr)),
                                          grad_scale=float(np.float32(grad_scale)), **HYPER)
            gi = before["g"][i].astype(np.float64) * grad_scale
            # three roundings of products of the constants (rounded themselves) and one of the sum: at most 4 half steps
            assert np.all(np.abs(after["m"][i] - m) <= 4 * U * (np.abs(before["m"][i]) + 0.1 * np.abs(gi)))
            assert np.all(np.abs(after["v"][i] - v) <= 5 * U * (np.abs(before["v"][i]) + 0.001 * gi ** 2))
            upd = (m / (1 - HYPER["beta1"] ** t)) / (np.sqrt(v / (1 - HYPER["beta2"] ** t)) + HYPER["eps"])
            mag = (0.9 * np.abs(before["m"][i]) + 0.1 * np.abs(gi)) / np.maximum(np.abs(m), 1e-300)   # m may cancel
            upd = np.abs(upd) * np.maximum(mag, 1.0)
        # p: its own two roundings, and the step's: about ten float32 operations, each 2 half steps (root and
        # reciprocal of one unit), the constant 1 - lr wd half a step
        tol = 4 * U * np.abs(p) + 32 * U * float(np.float32(lr)) * np.abs(upd)
        assert np.all(np.abs(after["p"][i] - want) <= tol + 1e-45), i
        if s["copy"]:
            assert torch.equal(s["copy"][i], s["p"][i].to(s["copy"][i].dtype))
    return after


SIZES = [[1], [255], [256, 257], [4096], [4097, 1, 0, 12289], [3, 0, 5], [81920, 278528, 17], [1] * 70 + [5000] + [2] * 300]


@pytest.mark.gpu
@pytest.mark.parametrize("gt,copy", [(F32, None), (BF16, BF16), (F32, F16)])
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}t{sum(s)}")
def test_steps(sizes, bits, gt, copy):
    print("[adamw]", len(sizes), sum(sizes), bits, gt, copy, flush=True)
    s = states(sizes, bits, gt, copy, seed=sum(sizes))
    before = snapshot(s)
    for t in (1, 2, 1000):
        step, lr = scalars(t, 1e-2 / t)
        wq.adamw_run(s["table"], step, lr, seed=5 + t, grad_scale=0.5, **HYPER)
        before = check_step(before, s, t, 1e-2 / t, 5 + t, 0.5)


@pytest.mark.gpu
def test_zero_states_and_zero_gradients():
    for bits in (32, 8):
        s = states([600], bits, F32, None)
        for key in ("m", "v", "ms", "vs"):
            for t in s[key]:
                t.zero_() if t.dtype == F32 else t.view(torch.uint8).zero_()
        s["g"][0][:300] = 0
        before = snapshot(s)
        step, lr = scalars(1, 1e-3)
        wq.adamw_run(s["table"], step, lr, **HYPER)
        after = check_step(before, s, 1, 1e-3, 0)
        assert np.isfinite(after["p"][0]).all()


@pytest.mark.gpu
def test_values_that_are_not_finite():
    """A NaN or infinite gradient reaches its own element's parameter and states, and no other's."""
    for bits in (32, 8):
        s = states([1024], bits, F32, None, seed=4)
        c = states([1024], bits, F32, None, seed=4)
        s["g"][0][300], s["g"][0][301] = float("nan"), float("inf")
        step, lr = scalars(3, 1e-3)
        for u in (s, c):
            wq.adamw_run(u["table"], step, lr, **HYPER)
        bad, clean = snapshot(s), snapshot(c)
        keep = np.delete(np.arange(1024), (300, 301))
        assert np.array_equal(bad["p"][0][keep], clean["p"][0][keep])
        assert not np.isfinite(bad["p"][0][300])
        if bits == 8:
            other = np.r_[0:256, 512:1024]                              # the blocks beside
            assert np.array_equal(bad["m"][0][other], clean["m"][0][other])
            assert (bad["m"][0][300] & 0x7F) == 0x7F and (bad["v"][0][300] & 0x7F) > 0x7B
            assert np.all((bad["m"][0][256:300] & 0x7F) != 0x7F)
        else:
            assert np.array_equal(bad["m"][0][keep], clean["m"][0][keep])


@pytest.mark.gpu
def test_a_state_that_is_not_finite_leaves_its_block_alone():
    """The other elements of the block get the codes and scales that they get beside zeros."""
    s, c = (states([700], 8, F32, None, seed=6) for _ in range(2))
    at = [256, 300, 301, 511, 699]
    for u in (s, c):
        u["m"][0].view(torch.uint8)[at] = 0
        u["v"][0].view(torch.uint8)[at] = 0
        u["g"][0][at] = 0
    s["g"][0][at] = torch.tensor([float("inf"), float("nan"), float("-inf"), 3e38, float("inf")], device=DEV)  # 3e38: v infinite
    step, lr = scalars(5, 1e-3)
    for u in (s, c):
        wq.adamw_run(u["table"], step, lr, seed=3, **HYPER)
    bad, clean = snapshot(s), snapshot(c)
    keep = np.delete(np.arange(700), at)
    for k in ("p", "v"):
        assert np.array_equal(bad[k][0][keep], clean[k][0][keep]), k
    # m: 0.1 * 3e38 is finite and rules its block (256 .. 511), at the largest scale
    assert np.array_equal(bad["m"][0][:256], clean["m"][0][:256]) and np.array_equal(bad["m"][0][512:699], clean["m"][0][512:699])
    assert np.array_equal(bad["vs"][0], clean["vs"][0]) and bad["ms"][0][1] == 2.0 ** 100
    assert np.array_equal(bad["ms"][0][[0, 2]], clean["ms"][0][[0, 2]])
    assert np.all((bad["v"][0][at] & 0x7F) > 0x7B) and np.all((bad["m"][0][[256, 300, 301, 699]] & 0x7F) == 0x7F)


@pytest.mark.gpu
def test_eight_bit_states_follow_the_moving_average():
    """Over many steps on one gradient v approaches g^2, which rounding to nearest would not: a step moves v by
    0.1% where codes are 25% apart.  The mean over n elements of the stochastic walk is off by its spread / sqrt(n);
    a code step is at most 2^-2 relative and some 300 roundings random, so the mean's error is far below 10%."""
    n, T = 1 << 16, 300
    s = states([n], 8, F32, None)
    for key in ("m", "v"):
        s[key][0].view(torch.uint8).zero_()
    s["g"][0].fill_(1e-3)
    step, lr = scalars(0, 0.0)
    for _ in range(T):
        step += 1
        wq.adamw_run(s["table"], step, lr, seed=9, **HYPER)
    v = s["v"][0].float().view(-1, 256) * s["vs"][0][:, None]
    m = s["m"][0].float().view(-1, 256) * s["ms"][0][:, None]
    assert abs(v.mean().item() / ((1 - 0.999 ** T) * 1e-6) - 1) < 0.1
    assert abs(m.mean().item() / ((1 - 0.9 ** T) * 1e-3) - 1) < 0.1


@pytest.mark.gpu
def test_graph_replays_with_a_moving_step():
    for bits in (32, 8):
        a, b = states([5000, 300], bits, F32, BF16, seed=8), states([5000, 300], bits, F32, BF16, seed=8)
        step, lr = scalars(0, 1e-3)
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            wq.adamw_run(a["table"], step, lr, seed=2, **HYPER)
        for t in (1, 2, 3, 4):
            step.fill_(t)
            lr.fill_(1e-3 / t)
            g.replay()
            wq.adamw_run(b["table"], step, lr, seed=2, **HYPER)
            torch.cuda.synchronize()
            x, y = snapshot(a), snapshot(b)
            assert all(np.array_equal(u, w) for k in x for u, w in zip(x[k], y[k])), t
            assert all(torch.equal(u, w) for u, w in zip(a["copy"], b["copy"]))


@pytest.mark.gpu
def test_a_tensor_past_4_GiB():
    n = (1 << 30) + 4099                                               # p, m, v: 4.3 GB each
    p = torch.zeros(n, device=DEV)
    g = torch.zeros(n, device=DEV, dtype=BF16)
    m, v = torch.zeros(n, device=DEV), torch.zeros(n, device=DEV)
    at = torch.tensor([0, 1, (1 << 30) - 1, 1 << 30, n - 1], device=DEV)
    g[at] = torch.tensor([1.0, 2.0, 3.0, 4.0, 5.0], device=DEV, dtype=BF16)
    step, lr = scalars(1, 1e-3)
    wq.adamw_run(wq.adamw_table([p], [g], [m], [v]), step, lr, weight_decay=0.0)
    # at the first step from zero states every parameter with a gradient moves by lr (eps aside)
    assert np.allclose(host(p[at]), -1e-3, rtol=1e-4) and int((p != 0).sum()) == 5
    assert np.allclose(host(m[at]), [0.1, 0.2, 0.3, 0.4, 0.5], rtol=1e-6)


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("gt,copy", [(BF16, F16), (F32, BF16)])
def test_tensors_of_a_large_table_step_as_in_a_small_one(bits, gt, copy):
    """Large tables take other access hints; the same tensors at the same places step to the same bits."""
    sizes = [100003, 1, 257, 4099, 300]
    small, large = states(sizes, bits, gt, copy), states(sizes, bits, gt, copy)
    n = 21 << 20
    z = lambda d: torch.zeros(n, dtype=d, device=DEV)
    big = dict(p=z(F32), g=torch.ones(n, dtype=gt, device=DEV), m=z(F32 if bits == 32 else torch.uint8),
               v=z(F32 if bits == 32 else torch.uint8), copy=z(copy))
    if bits == 8:
        big.update(ms=torch.zeros(n // 256, device=DEV), vs=torch.zeros(n // 256, device=DEV))
    if bits == 8:
        large["m"], large["v"] = [[t.view(torch.uint8) for t in large[k]] for k in ("m", "v")]
    for k, t in big.items():
        large[k].append(t)
    large["table"] = wq.adamw_table(large["p"], large["g"], large["m"], large["v"], large["copy"], large["ms"] or None,
                                    large["vs"] or None)
    step, lr = scalars(1, 1e-3)
    for s in (small, large):
        wq.adamw_run(s["table"], step, lr, seed=9, **HYPER)
    a, b = snapshot(small), snapshot(large)
    for k in a:
        for u, w in zip(a[k], b[k][:-1] if b[k] else []):
            assert np.array_equal(u, w), k
    assert all(torch.equal(u, w) for u, w in zip(small["copy"], large["copy"]))
    # unit gradients from zero states: the update (of the states before their rounding) is lr, up to eps = 1e-8 and
    # some eight float32 roundings of 2^-24 each
    assert float((big["p"] + 1e-3).abs().max()) <= 1e-3 * 1e-6


@pytest.mark.gpu
@pytest.mark.parametrize("count", [255, 256, 257, 513, 65535, 65537, 70000])
def test_many_small_tensors(count):
    """Every tensor of a long table is found: one, two and three steps of the search, empty tensors among them."""
    r = np.random.default_rng(count)
    sizes = r.integers(0, 9, count)
    sizes[r.random(count) < 0.3] = 0
    if count > 60000:
        sizes[1000:2000] = 0                                           # a long empty run, and a tensor of many chunks
        sizes[2000] = 3 * 4096 + 5
    at = np.concatenate(([0], np.cumsum((sizes + 7) // 8 * 8)))          # 16-byte aligned places in flat buffers
    p, pd = torch.zeros(at[-1] + 8, device=DEV), r.standard_normal(at[-1] + 8).astype(np.float32)
    p.copy_(torch.from_numpy(pd))
    g = torch.from_numpy(r.standard_normal(at[-1] + 8)).to(BF16).to(DEV)
    m, v = torch.zeros_like(p), torch.zeros_like(p)
    cut = lambda b: [b[a:a + n] for a, n in zip(at.tolist(), sizes.tolist())]
    step, lr = scalars(1, 1e-3)
    wq.adamw_run(wq.adamw_table(cut(p), cut(g), cut(m), cut(v)), step, lr, **HYPER)
    want, wm, wv = oracle.adamw_ref(pd, host(g), 0 * pd, 0 * pd, 1, float(np.float32(1e-3)), HYPER["beta1"], HYPER["beta2"],
                                    HYPER["eps"], HYPER["weight_decay"])
    on = np.zeros(at[-1] + 8, dtype=bool)
    for a, n in zip(at, sizes):
        on[a:a + n] = True
    # as in check_step; from zero states the step is lr itself, up to eps
    assert np.all(np.abs(host(p) - want)[on] <= 4 * U * np.abs(pd[on]) + 32 * U * 1e-3)
    assert np.all(np.abs(host(m) - wm)[on] <= 4 * U * np.abs(wm[on])) and np.all(np.abs(host(v) - wv)[on] <= 5 * U * np.abs(wv[on]))
    assert np.array_equal(host(p)[~on], pd[~on]) and not host(m)[~on].any() and not host(v)[~on].any()


@pytest.mark.gpu
def test_a_table_of_the_other_form_is_left_alone():
    s = states([1000], 32, F32, None)
    before = snapshot(s)
    s["table"].bits = 8
    step, lr = scalars(1, 1e-3)
    wq.adamw_run(s["table"], step, lr)
    torch.cuda.synchronize()
    after = snapshot(s)
    assert all(np.array_equal(u, w) for k in before for u, w in zip(before[k], after[k]))


def test_the_mix_spreads_its_bits():
    """Of 2^16 elements' 16-bit draws each bit is set near half the time (five sigma), and neighbours are uncorrelated."""
    n = 1 << 16
    for seed, t, tensor in ((0, 1, 0), (17, 7, 3), (2 ** 32 - 1, 100000, 1000)):
        for r in oracle.adamw_random_bits(n, seed, t, tensor):
            for b in range(16):
                ones = np.sum((r >> b) & 1)
                assert abs(ones - n / 2) < 5 * np.sqrt(n) / 2
            z = r / 65536.0 - 0.5
            assert abs(np.mean(z[1:] * z[:-1])) < 5 / 12 / np.sqrt(n)


def test_stochastic_codes_of_the_oracle():
    """Exact grid values keep their code for every draw; between two codes the upper is taken in proportion."""
    for grid in (oracle.E4M3_GRID, oracle.E5M2_GRID):
        r = np.arange(0, 65536, 257)
        for c in range(grid.size):
            assert np.all(oracle.stochastic_code(np.full(r.size, grid[c]), r, grid) == c)
        x = grid[20] + 0.25 * (grid[21] - grid[20])
        assert abs(np.mean(oracle.stochastic_code(np.full(65536, x), np.arange(65536), grid) - 20) - 0.25) < 1e-4
