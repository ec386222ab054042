"""The adapters' 32-row tile kernels against the float64 oracle.

Every shape asserts, by the restated dispatch rules, that it reaches the kernels it is there for: small shapes go to the
row kernels instead, whatever a test about tiles means to show.
"""
import numpy as np
import pytest
import torch

import oracle
import weight_quantized_mlp_amd as wq
from adapter_common import DEV, U, host, norm_bound, randn, rel2
from adapter_dispatch import few_rows, one_launch, outer_one_wave, outer_parts, shrink_parts, up
from test_lora import forward, ids_for, problem

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
BYTES = {F32: 4, BF16: 2, F16: 2}
name = lambda s: "x".join(str(v).replace("torch.", "") for v in s) if isinstance(s, tuple) else None


def tiled(shape):
    M, K, N, E, R, xt, wt = shape
    return not few_rows(M, K, N, R, BYTES[wt]) and not one_launch(M, K, N, R)


def check_forward(p, shape):
    K, R, n = shape[1], shape[4], p["n"]
    got = host(forward(p)).astype(np.float64)
    ref = oracle.lora_ref(n["x"], n["a"], n["b"], n["scale"], n["ids"], n["y"])
    size = oracle.lora_ref(abs(n["x"]), abs(n["a"]), abs(n["b"]), n["scale"], n["ids"], 0 * n["y"])
    # the two chained sums, the scale's products and the last addition
    assert np.all(np.abs(got - ref) <= 2 * (K + R + 8) * U * size + 2 * U * np.abs(ref))
    part = np.linalg.norm(ref - n["y"])
    assert np.linalg.norm(got - ref) <= norm_bound(K, R) * part + 2 * U * np.linalg.norm(ref)
    off = (n["ids"] < 0) | (n["ids"] >= shape[3])
    assert np.array_equal(got[off], n["y"][off])                      # rows without an adapter: y itself


def check_backward(p, shape, dyt, dxt, base=True):
    M, K, N, E, R = shape[:5]
    n = p["n"]
    dy, dyd = randn(M + N, (M, N), dyt, 1e-3)
    dx0, dxd = randn(M + K, (M, K), dxt, 1e-3) if base else (None, np.zeros((M, K)))
    dx, da, db = wq.lora_backward(dy, p["x"], p["a"], p["b"], p["scale"], p["ids"], dx0, dx_dtype=dxt)
    rx, ra, rb = oracle.lora_backward_ref(dyd, n["x"], n["a"], n["b"], n["scale"], n["ids"], dxd)
    rows = np.array([np.sum(n["ids"] == e) for e in range(E)])
    assert da.dtype == db.dtype == F32 and dx.dtype == dxt
    assert rel2(host(da), ra) <= norm_bound(N, rows.max())
    assert rel2(host(db), rb) <= norm_bound(K, rows.max())
    assert not host(da)[rows == 0].any() and not host(db)[rows == 0].any()
    # dx: a chain of N and R terms, the addition, one rounding to its type (eps / 2 relative at most)
    eps = torch.finfo(dxt).eps / 2
    tiny = 2.0 ** -25 if dxt == F16 else 0.0                            # half of float16's smallest step
    assert np.linalg.norm(host(dx) - rx) <= norm_bound(N, R) * np.linalg.norm(rx - dxd) + (2 * U + eps) * np.linalg.norm(rx) + \
        tiny * np.sqrt(rx.size)
    size, sa, sb = oracle.lora_backward_ref(abs(dyd), abs(n["x"]), abs(n["a"]), abs(n["b"]), n["scale"], n["ids"], 0 * dxd)
    assert np.all(np.abs(host(dx) - rx) <= 2 * (N + R + 8) * U * size * (1 + 2 ** -8) + (eps + 2 * U) * abs(rx) + tiny)
    c = rows[:, None, None]
    assert np.all(np.abs(host(da) - ra) <= 2 * (N + c + 8) * U * sa)
    assert np.all(np.abs(host(db) - rb) <= 2 * (K + c + 8) * U * sb)


# every pair of types; every rank class of the three kernels with each type of weights; tiles of many adapters
TYPES = [(300, 208, 150, 5, 64, xt, wt) for xt in (F32, BF16, F16) for wt in (F32, BF16, F16)]
RANKS = [(up(16385, max(R, 16)) + 3, 1040, 131, 3, R, F32 if wt == F16 else BF16, wt) for R in (8, 16, 24, 32, 40, 64, 72, 128, 136, 256)
         for wt in (F32, BF16, F16)]
MANY = [(300, 208, 96, 70, 64, BF16, BF16), (1300, 336, 67, 70, 32, F16, F32), (2080, 144, 67, 40, 16, F32, BF16)]
SHAPES = TYPES + RANKS + MANY


def test_the_shapes_reach_the_tiles():
    assert all(tiled(s) for s in SHAPES)
    M, K, N, E, R = MANY[1][:5]
    assert max(2, 512 // (up(M, 32) * up(R, 32))) < 20                  # workgroups per tile: fewer than its random rows' adapters


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["runs", "random", "bad"])
@pytest.mark.parametrize("shape", SHAPES, ids=name)
def test_forward(shape, kind):
    print("[lora]", shape, kind, flush=True)
    check_forward(problem(shape, kind, seed=21), shape)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["runs", "random"])
@pytest.mark.parametrize("dyt,dxt", [(F32, F32), (BF16, BF16), (F32, BF16), (BF16, F16)])
@pytest.mark.parametrize("shape", SHAPES, ids=name)
def test_backward(shape, dyt, dxt, kind):
    print("[lora_backward]", shape, dyt, dxt, kind, flush=True)
    check_backward(problem(shape, kind, seed=22), shape, dyt, dxt, base=kind == "runs")


# a long contraction on few tiles is split, in either product; the last: rows few, b too large for the row form of dy b
SPLIT = [(320, 5120, 515, 3, 64, BF16, BF16), (320, 5120, 515, 3, 64, F32, F32), (1030, 9216, 67, 2, 16, BF16, F16),
         (330, 208, 7007, 3, 64, F16, F32), (70, 4112, 5121, 2, 256, F16, BF16), (61, 1040, 7007, 32, 64, BF16, BF16)]


def test_the_shapes_are_split():
    for s in SPLIT:
        M, K, N, E, R, xt, wt = s
        x, dy = shrink_parts(M, K, R, BYTES[xt], BYTES[wt]), shrink_parts(M, N, R, 4, BYTES[wt])
        assert tiled(s) and max(x, dy) > 1 or (M == 61 and dy > 1 and N * R * BYTES[wt] > 512 << 10), s
    assert {shrink_parts(s[0], s[1], s[4], BYTES[s[5]], BYTES[s[6]]) > 1 for s in SPLIT} == {True, False}


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["runs", "random", "bad"])
@pytest.mark.parametrize("shape", SPLIT, ids=name)
def test_split_contractions(shape, kind):
    print("[lora split]", shape, kind, flush=True)
    p = problem(shape, kind, seed=23)
    check_forward(p, shape)
    for dyt, dxt in ((F32, F32), (BF16, BF16)):
        check_backward(p, shape, dyt, dxt)


# weight gradients whose rows are split over workgroups; and those of one wave per workgroup
PARTS = [(2100, 192, 131, 1, 16, BF16, BF16), (2100, 192, 131, 1, 64, F32, F32), (4500, 80, 67, 2, 24, F16, BF16)]
ONE_WAVE = [(96, 5120, 4099, 16, 16, F32, BF16), (40, 5600, 5601, 9, 56, BF16, F32), (130, 3200, 3331, 16, 32, F16, F16)]


def test_the_shapes_reach_the_forms_of_the_weight_gradients():
    for M, K, N, E, R, _, _ in PARTS:
        assert outer_parts(M, K, E, R) > 1 and outer_parts(M, N, E, R) > 1
    for M, K, N, E, R, _, _ in ONE_WAVE:
        assert outer_one_wave(M, K, E, R) and outer_one_wave(M, N, E, R)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["runs", "one", "random"])
@pytest.mark.parametrize("shape", PARTS + ONE_WAVE, ids=name)
def test_forms_of_the_weight_gradients(shape, kind):
    print("[lora outer]", shape, kind, flush=True)
    p = problem(shape, kind, seed=24)
    for dyt, dxt in ((F32, BF16), (BF16, F32)):
        check_backward(p, shape, dyt, dxt)


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(300, 208, 150, 4, 64, BF16, BF16), (300, 208, 150, 4, 64, F32, F16), (1030, 528, 96, 4, 16, F16, F32),
                                   (70, 144, 131, 4, 256, BF16, BF16), (320, 5120, 131, 4, 64, BF16, BF16)], ids=name)
def test_values_that_a_row_must_not_see(shape):
    """Adapters that share every tile: NaN and infinities in another's weights, in a masked row's x and dy."""
    M, K, N, E, R = shape[:5]
    assert tiled(shape)
    p = problem(shape, "random", seed=3)
    ids = torch.arange(M, device=DEV, dtype=torch.int32) % E
    ids[ids == 3] = -1                                                # adapter 3 is loaded, no row names it
    p["ids"] = ids
    dy = torch.randn((M, N), device=DEV, generator=torch.Generator(DEV).manual_seed(1))
    back = lambda: wq.lora_backward(dy, p["x"], p["a"], p["b"], p["scale"], p["ids"], None, dx_dtype=F32)
    clean = host(forward(p))
    cx, ca, cb = (host(t) for t in back())
    for e, bad in ((3, float("nan")), (2, float("inf"))):
        p["a"][e] = bad
        p["b"][e, ::2] = -bad
        p["scale"][e] = bad
    p["x"][ids == -1] = float("nan")
    dy[ids == -1] = float("nan")
    got = host(forward(p))
    at = ids.cpu().numpy()
    keep = np.isin(at, (0, 1, -1))
    assert np.isfinite(clean).all() and np.array_equal(got[keep], clean[keep])
    assert not np.isfinite(got[at == 2]).all()
    dx, da, db = (host(t) for t in back())
    assert np.array_equal(dx[keep], cx[keep]) and not dx[at == -1].any()
    assert np.array_equal(da[[0, 1]], ca[[0, 1]]) and np.array_equal(db[[0, 1]], cb[[0, 1]])
    assert not da[3].any() and not db[3].any()                        # no row: zero, whatever the adapter holds
    # a row's own NaN and infinity stay in the row, and in its adapter's gradients
    p["x"][0] = float("nan")                                          # rows 0 and 1: adapters 0 and 1
    dy[1, :2] = float("inf")
    mx, ma, mb = (host(t) for t in back())
    keep[[0, 1]] = False
    assert np.array_equal(host(forward(p))[keep], clean[keep]) and np.array_equal(mx[keep], cx[keep])
    assert np.isnan(ma[0]).all() and np.isnan(mb[0]).all() and not np.isfinite(ma[1]).all() and not np.isfinite(mb[1]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("xt,wt,M,K,R", [(F32, F16, 290, 208, 64), (F32, BF16, 290, 208, 64), (BF16, BF16, 290, 208, 64),
                                         (BF16, BF16, 520, 272, 32), (F32, F32, 520, 272, 32), (F16, F32, 1030, 528, 16), (BF16, F16, 70, 1040, 256)])
def test_a_row_alone_on_its_adapter(xt, wt, M, K, R):
    """Every row of a tile in turn alone on one adapter, the others on another or on none."""
    N, E = 64, 32
    shape = (M, K, N, E, R, xt, wt)
    assert tiled(shape)
    p = problem(shape, "one")
    n = p["n"]
    for rest in (-1, 3):
        for r in range(32):
            ids = np.full(M, rest, dtype=np.int32)
            ids[r::32] = 30
            p["ids"].copy_(torch.from_numpy(ids))
            ref = oracle.lora_ref(n["x"], n["a"], n["b"], n["scale"], ids, n["y"])
            at = ids == 30
            got = host(forward(p))
            # each of the lone rows by itself, so that one of them left out cannot hide among the others
            err, size = np.linalg.norm(got - ref, axis=1), np.linalg.norm(ref - n["y"], axis=1)
            assert np.all(err[at] <= norm_bound(K, R) * size[at] + 2 * U * np.linalg.norm(ref, axis=1)[at]), (rest, r)
            assert rel2(got[~at], ref[~at]) <= norm_bound(K, R), (rest, r)


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(300, 320, 260, 4, 64, BF16, BF16), (320, 5120, 515, 4, 64, F32, BF16),
                                   (2100, 192, 131, 4, 16, BF16, F32)], ids=name)
def test_graph_replays_streams_and_in_place(shape):
    """Captured, on other streams at once and in place, the tiles give the eager call's bits."""
    M, K, N, E, R = shape[:5]
    assert tiled(shape)
    p = problem(shape, "runs")
    dy, _ = randn(9, (M, N), F32, 1e-3)
    dx0, _ = randn(10, (M, K), BF16, 1e-3)
    out, dx = torch.empty_like(p["y"]), torch.empty((M, K), dtype=BF16, device=DEV)
    da, db = torch.empty((E, R, K), device=DEV), torch.empty((E, N, R), device=DEV)
    w1 = torch.empty(max(1, wq.lora_workspace_bytes(M, K, N, E, R)), dtype=torch.uint8, device=DEV)
    w2 = torch.empty(wq.lora_workspace_bytes(M, K, N, E, R, True), dtype=torch.uint8, device=DEV)
    args = lambda: (dy, p["x"], p["a"], p["b"], p["scale"], p["ids"])

    def both():
        forward(p, out=out, workspace=w1)
        wq.lora_backward(*args(), dx0, dx, da, db, workspace=w2)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        both()
    for i in range(4):
        p["x"].normal_()
        p["ids"].copy_(torch.from_numpy(ids_for(["runs", "random", "none", "bad"][i], M, E, i)))
        both()
        torch.cuda.synchronize()
        want = [host(t).copy() for t in (out, dx, da, db)]
        for t in (out, dx, da, db):
            t.fill_(float("nan"))
        w1.fill_(0xFF)
        w2.fill_(0xFF)
        g.replay()
        torch.cuda.synchronize()
        assert all(np.array_equal(host(t), w) for t, w in zip((out, dx, da, db), want)), i
    s2 = torch.cuda.Stream()
    with torch.cuda.stream(s):
        o1 = forward(p)
    with torch.cuda.stream(s2):
        g2 = wq.lora_backward(*args(), dx0)
    torch.cuda.synchronize()
    assert all(np.array_equal(host(t), w) for t, w in zip((o1, *g2), want))
    y, d = p["y"].clone(), dx0.clone()
    wq.lora_run(p["x"], p["a"], p["b"], p["scale"], p["ids"], y, out=y)
    wq.lora_backward(*args(), d, dx=d, need=(True, False, False))
    assert np.array_equal(host(y), want[0]) and np.array_equal(host(d), want[1])


@pytest.mark.gpu
@pytest.mark.parametrize("power", [-100, -112, -124])
@pytest.mark.parametrize("shape", [(300, 208, 150, 3, 64, F32, F32), (300, 208, 150, 3, 64, F32, BF16), (320, 5120, 131, 3, 64, F32, F16)], ids=name)
def test_operands_near_the_smallest_bfloat16_step(shape, power):
    """A float32 operand keeps its bits down to 2^-133: each is off by 2^-134 at most, beside float32's own roundings."""
    M, K, N, E, R = shape[:5]
    assert tiled(shape)
    p = problem(shape, "random", seed=5)
    p["x"] = p["x"] * 2.0 ** power                                     # exact
    n = dict(p["n"], x=p["x"].double().cpu().numpy(), y=np.zeros((M, N)))
    got = host(wq.lora_run(p["x"], p["a"], p["b"], p["scale"], p["ids"], None)).astype(np.float64)
    ref = oracle.lora_ref(n["x"], n["a"], n["b"], n["scale"], n["ids"], n["y"])
    size = oracle.lora_ref(abs(n["x"]), abs(n["a"]), abs(n["b"]), n["scale"], n["ids"], n["y"])
    # an error of 2^-134 in every x against a, and in every element of the scaled intermediate against b; float32 subnormals
    off = oracle.lora_ref(np.full((M, K), 2.0 ** -134), abs(n["a"]), abs(n["b"]), n["scale"], n["ids"], n["y"])
    off += 2.0 ** -134 * np.abs(n["b"]).sum(2).max() + 2.0 ** -149 * (K + R)
    assert np.all(np.abs(got - ref) <= 2 * (K + R + 8) * U * size + 2 * U * np.abs(ref) + off)
