"""Low-rank adapters beside a projection (lora_run, lora_backward) against the float64 oracle."""
import numpy as np
import pytest
import torch

import oracle
import weight_quantized_mlp_amd as wq
from adapter_common import DEV, U, host, norm_bound, randn, rel2, runs

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16

# M, K, N, E, R, x, w: one token to several tiles, odd N, every rank class, every pair of types
SHAPES = [
    (1, 16, 1, 1, 8, F32, F32), (1, 256, 512, 1, 8, F32, BF16), (2, 48, 67, 3, 16, BF16, BF16),
    (17, 320, 67, 2, 24, F16, F16), (31, 272, 131, 5, 40, BF16, F16), (33, 5120, 258, 32, 16, BF16, BF16),
    (61, 1040, 1001, 32, 64, F32, F16), (64, 512, 256, 1, 128, BF16, F32), (65, 336, 513, 4, 72, F16, BF16),
    (129, 320, 67, 2, 8, F32, F32), (130, 2064, 777, 70, 32, F32, BF16), (300, 640, 1300, 3, 256, BF16, BF16),
    (515, 144, 96, 600, 8, F16, F32), (1027, 1280, 515, 6, 96, BF16, BF16),
]


def ids_for(kind, M, E, seed):
    r = np.random.default_rng(seed)
    if kind == "runs":
        return runs(seed, M, E, min(M, 7))
    if kind == "random":
        return r.integers(0, E, M).astype(np.int32)
    if kind == "one":
        return np.full(M, E - 1, dtype=np.int32)
    if kind == "none":
        return np.full(M, -1, dtype=np.int32)
    bad = np.array([E, E + 1, -1, -7, 2 ** 31 - 1, -2 ** 31], dtype=np.int64)
    return np.where(r.random(M) < 0.5, r.integers(0, E, M), bad[r.integers(0, bad.size, M)]).astype(np.int32)


def problem(shape, kind, seed=0):
    M, K, N, E, R, xt, wt = shape
    s = 1000 * M + K + seed
    x, xd = randn(s, (M, K), xt)
    a, ad = randn(s + 1, (E, R, K), wt, K ** -0.5)
    b, bd = randn(s + 2, (E, N, R), wt, 0.3)
    y, yd = randn(s + 3, (M, N), F32, 1.5)
    sc = np.random.default_rng(s + 4).uniform(0.5, 2.0, E).astype(np.float32)
    ids = ids_for(kind, M, E, s + 5)
    return dict(x=x, a=a, b=b, y=y, scale=torch.from_numpy(sc).to(DEV), ids=torch.from_numpy(ids).to(DEV),
                n=dict(x=xd, a=ad, b=bd, y=yd, scale=sc, ids=ids))


def forward(p, **kw):
    return wq.lora_run(p["x"], p["a"], p["b"], p["scale"], p["ids"], p["y"], **kw)


@pytest.mark.parametrize("kind", ["runs", "random", "one", "none", "bad"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(str(v).replace("torch.", "") for v in s))
def test_forward(shape, kind):
    print("[lora]", shape, kind, flush=True)
    M, K, N, E, R = shape[:5]
    p = problem(shape, kind)
    n = p["n"]
    got = host(forward(p)).astype(np.float64)
    ref = oracle.lora_ref(n["x"], n["a"], n["b"], n["scale"], n["ids"], n["y"])
    size = oracle.lora_ref(abs(n["x"]), abs(n["a"]), abs(n["b"]), n["scale"], n["ids"], 0 * n["y"])
    # the two chained sums, the scale's products and the last addition
    assert np.all(np.abs(got - ref) <= 2 * (K + R + 8) * U * size + 2 * U * np.abs(ref))
    assert rel2(got - n["y"], ref - n["y"]) <= norm_bound(K, R) + 4 * U * np.linalg.norm(n["y"]) / max(
        np.linalg.norm(ref - n["y"]), 1e-30) or not (ref - n["y"]).any()
    off = (n["ids"] < 0) | (n["ids"] >= E)
    assert np.array_equal(got[off], n["y"][off])                      # rows without an adapter: y itself


def test_forward_in_place_and_without_base():
    p = problem((67, 160, 130, 3, 16, BF16, BF16), "runs")
    want = host(forward(p))
    part = host(wq.lora_run(p["x"], p["a"], p["b"], p["scale"], p["ids"], None))
    n = p["n"]
    zero = oracle.lora_ref(n["x"], n["a"], n["b"], n["scale"], n["ids"], 0 * n["y"])
    assert rel2(part, zero) <= norm_bound(160, 16)
    out = forward(p, out=p["y"])
    assert out.data_ptr() == p["y"].data_ptr()
    assert np.array_equal(host(out), want)


@pytest.mark.parametrize("M", [5, 64, 200])
def test_values_that_a_row_must_not_see(M):
    """NaN and infinities in another adapter's weights, in a masked row's x, in nothing's scale."""
    E = 4
    p = problem((M, 208, 150, E, 16, BF16, BF16), "random", seed=3)
    ids = torch.arange(M, device=DEV, dtype=torch.int32) % E
    ids[ids == 3] = -1                                                # adapter 3 is loaded, no row names it
    p["ids"] = ids
    clean = host(forward(p))
    for e, bad in ((3, float("nan")), (2, float("inf"))):
        p["a"][e] = bad
        p["b"][e, ::2] = -bad
        p["scale"][e] = bad
    p["x"][ids == -1] = float("nan")
    got = host(forward(p))
    keep = np.isin(ids.cpu().numpy(), (0, 1, -1))
    assert np.isfinite(clean).all() and np.array_equal(got[keep], clean[keep])
    assert not np.isfinite(got[ids.cpu().numpy() == 2]).all()
    dy = torch.randn((M, 150), device=DEV, generator=torch.Generator(DEV).manual_seed(1))
    dy[ids == -1] = float("nan")
    dx, da, db = wq.lora_backward(dy, p["x"], p["a"], p["b"], p["scale"], p["ids"], None, dx_dtype=F32)
    assert np.isfinite(host(dx)[keep]).all() and np.isfinite(host(da)[[0, 1]]).all() and np.isfinite(host(db)[[0, 1]]).all()
    assert not host(dx)[ids.cpu().numpy() == -1].any()
    assert not host(da)[3].any() and not host(db)[3].any()            # no row: zero, whatever the adapter holds


def test_zero_rows():
    p = problem((4, 64, 48, 3, 8, F32, F32), "one")
    out = wq.lora_run(p["x"][:0], p["a"], p["b"], p["scale"], p["ids"][:0], p["y"][:0])
    assert out.shape == (0, 48)
    da = torch.full((3, 8, 64), 7.0, device=DEV)
    db = torch.full((3, 48, 8), 7.0, device=DEV)
    dx, da, db = wq.lora_backward(p["y"][:0], p["x"][:0], p["a"], p["b"], p["scale"], p["ids"][:0], da=da, db=db)
    assert dx.shape == (0, 64) and not host(da).any() and not host(db).any()


def backward_refs(p, dyd, dxd):
    n = p["n"]
    return oracle.lora_backward_ref(dyd, n["x"], n["a"], n["b"], n["scale"], n["ids"], dxd)


@pytest.mark.parametrize("kind", ["runs", "random", "one", "none", "bad"])
@pytest.mark.parametrize("dyt,dxt", [(F32, F32), (BF16, BF16), (F32, BF16), (BF16, F16)])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(str(v).replace("torch.", "") for v in s))
def test_backward(shape, dyt, dxt, kind):
    print("[lora_backward]", shape, dyt, dxt, kind, flush=True)
    M, K, N, E, R = shape[:5]
    p = problem(shape, kind, seed=7)
    dy, dyd = randn(M + N, (M, N), dyt, 1e-3)
    dx0, dxd = randn(M + K, (M, K), dxt, 1e-3)
    dx, da, db = wq.lora_backward(dy, p["x"], p["a"], p["b"], p["scale"], p["ids"], dx0)
    rx, ra, rb = backward_refs(p, dyd, dxd)
    n = p["n"]
    rows = np.array([np.sum(n["ids"] == e) for e in range(E)])
    assert da.dtype == db.dtype == F32 and dx.dtype == dxt
    assert rel2(host(da), ra) <= norm_bound(N, rows.max())
    assert rel2(host(db), rb) <= norm_bound(K, rows.max())
    assert not host(da)[rows == 0].any() and not host(db)[rows == 0].any()
    # dx: a chain of N and R terms, the addition, one rounding to its type (eps / 2 relative at most)
    part = np.linalg.norm(rx - dxd) / max(np.linalg.norm(rx), 1e-30)
    assert rel2(host(dx), rx) <= norm_bound(N, R) * part + 2 * U + torch.finfo(dxt).eps / 2
    aa, bb = abs(n["a"]), abs(n["b"])
    size, sa, sb = oracle.lora_backward_ref(abs(dyd), abs(n["x"]), aa, bb, n["scale"], n["ids"], 0 * dxd)
    tiny = {F32: 0.0, BF16: 0.0, F16: 2.0 ** -25}[dxt]                 # half of float16's smallest step
    assert np.all(np.abs(host(dx) - rx) <= 2 * (N + R + 8) * U * size * (1 + 2 ** -8) + (torch.finfo(dxt).eps / 2 + 2 * U) * abs(rx) + tiny)
    c = rows[:, None, None]
    assert np.all(np.abs(host(da) - ra) <= 2 * (N + c + 8) * U * sa)
    assert np.all(np.abs(host(db) - rb) <= 2 * (K + c + 8) * U * sb)


@pytest.mark.parametrize("dyt", [F32, BF16])
def test_columns_that_end_inside_a_piece(dyt):
    """Every remainder of N by the 4 or 8 elements of a 16-byte piece, and rows shorter than one."""
    for N in list(range(1, 18)) + list(range(121, 129)):
        print("[lora_backward] N", N, dyt, flush=True)
        p = problem((70, 48, N, 2, 8, BF16, BF16), "runs", seed=N)
        dy, dyd = randn(N, (70, N), dyt, 1e-3)
        dx, da, db = wq.lora_backward(dy, p["x"], p["a"], p["b"], p["scale"], p["ids"], dx_dtype=F32)
        rx, ra, rb = backward_refs(p, dyd, np.zeros((70, 48)))
        assert rel2(host(db), rb) <= norm_bound(48, 70), N
        assert rel2(host(da), ra) <= norm_bound(N, 70), N
        assert rel2(host(dx), rx) <= norm_bound(N, 8) + 2 * U, N


@pytest.mark.parametrize("M,K,N,E,R", [(33, 5120, 1280, 16, 16), (70, 5120, 5120, 8, 8), (300, 640, 512, 3, 24),
                                       (61, 1040, 7007, 32, 64)])
def test_each_gradient_is_the_same_without_the_others(M, K, N, E, R):
    p = problem((M, K, N, E, R, BF16, BF16), "runs", seed=3)
    dy, _ = randn(M, (M, N), BF16, 1e-3)
    args = (dy, p["x"], p["a"], p["b"], p["scale"], p["ids"])
    whole = wq.lora_backward(*args)
    for i in range(1, 7):
        need = tuple(bool(i >> j & 1) for j in range(3))
        for got, want, on in zip(wq.lora_backward(*args, need=need), whole, need):
            assert (got is not None) == on and (not on or torch.equal(got, want)), need


def test_backward_in_place_and_parts():
    p = problem((150, 192, 140, 3, 16, BF16, BF16), "runs")
    dy, _ = randn(1, (150, 140), F32, 1e-3)
    dx0, _ = randn(2, (150, 192), BF16, 1e-3)
    args = (dy, p["x"], p["a"], p["b"], p["scale"], p["ids"])
    dx, da, db = wq.lora_backward(*args, dx0)
    for need in ((True, False, False), (False, True, False), (False, False, True), (False, True, True)):
        got = wq.lora_backward(*args, dx0 if need[0] else None, need=need)
        for g, w, on in zip(got, (dx, da, db), need):
            assert (g is None) == (not on)
            assert g is None or np.array_equal(host(g), host(w))
    inplace = wq.lora_backward(*args, dx0, dx=dx0, need=(True, False, False))[0]
    assert inplace.data_ptr() == dx0.data_ptr() and np.array_equal(host(inplace), host(dx))


def test_gradients_against_differences():
    """lora_run is linear in each of x, a and b: <dy, f(p + d) - f(p)> is the gradient's product with d."""
    M, K, N, E, R = 70, 96, 83, 2, 8
    p = problem((M, K, N, E, R, F32, F32), "runs", seed=11)
    dy, dyd = randn(5, (M, N), F32)
    dx, da, db = wq.lora_backward(dy, p["x"], p["a"], p["b"], p["scale"], p["ids"])
    base = host(forward(p)).astype(np.float64)
    for name, grad in (("x", dx), ("a", da), ("b", db)):
        d, dd = randn(ord(name), tuple(p[name].shape), F32)
        q = dict(p)
        q[name] = p[name] + d
        step = (q[name] - p[name]).double().cpu().numpy()               # the step as it was rounded
        moved = host(forward(q)).astype(np.float64)
        want = np.sum(dyd * (moved - base))
        got = np.sum(host(grad).astype(np.float64) * step)
        # rounding of the two forward results (norm_bound of their norms) against |dy|, of the gradient against |d|
        tol = norm_bound(K, R) * np.linalg.norm(dyd) * (np.linalg.norm(moved) + np.linalg.norm(base))
        tol += norm_bound(N, M) * np.linalg.norm(host(grad)) * np.linalg.norm(dd)
        assert abs(got - want) <= tol, name
        assert abs(want) > 10 * tol or abs(got - want) <= 0.1 * abs(want) + tol


def test_same_rows_same_bits_and_other_streams():
    """A call's results are the same bits on any stream, and two calls at once do not disturb each other."""
    p = problem((200, 512, 700, 5, 32, BF16, BF16), "runs")
    q = problem((77, 512, 700, 5, 32, BF16, BF16), "random", seed=2)
    dy, _ = randn(3, (200, 700), F32, 1e-3)
    want, wantq = host(forward(p)), host(forward(q))
    wantg = [host(t) for t in wq.lora_backward(dy, p["x"], p["a"], p["b"], p["scale"], p["ids"])]
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(s1):
            o1 = forward(p)
            g1 = wq.lora_backward(dy, p["x"], p["a"], p["b"], p["scale"], p["ids"])
        with torch.cuda.stream(s2):
            o2 = forward(q)
        torch.cuda.synchronize()
        assert np.array_equal(host(o1), want) and np.array_equal(host(o2), wantq)
        assert all(np.array_equal(host(t), w) for t, w in zip(g1, wantg))


def test_rows_past_4_GiB():
    M, K, N, R = 63000, 64, 17408, 8          # y and out: 4.4 GB each
    g = torch.Generator(DEV).manual_seed(5)
    x = torch.randn((M, K), device=DEV, generator=g, dtype=BF16)
    a = torch.randn((2, R, K), device=DEV, generator=g, dtype=BF16)
    b = torch.randn((2, N, R), device=DEV, generator=g, dtype=BF16)
    y = torch.randn((M, N), device=DEV, generator=g)
    ids = (torch.arange(M, device=DEV) % 3 - 1).to(torch.int32)
    scale = torch.tensor([0.5, 2.0], device=DEV)
    rows = [0, 1, 2, 61679, 61680, 61681, 61682, M - 2, M - 1]
    ref = oracle.lora_ref(*(t.double().cpu().numpy() for t in (x[rows], a, b)), scale.cpu().numpy(),
                          ids[rows].cpu().numpy(), y[rows].double().cpu().numpy())
    out = wq.lora_run(x, a, b, scale, ids, y, out=y)
    assert rel2(host(out[rows]), ref) <= norm_bound(K, R)
    dx, da, db = wq.lora_backward(y, x, a, b, scale, ids)
    rdx = oracle.lora_backward_ref(*(t.double().cpu().numpy() for t in (y[rows], x[rows], a, b)), scale.cpu().numpy(),
                                   ids[rows].cpu().numpy(), np.zeros((len(rows), K)))[0]
    assert rel2(host(dx[rows]), rdx) <= norm_bound(N, R) + torch.finfo(BF16).eps / 2
    on = torch.nonzero(ids == 1).flatten()
    t = x[on].double() @ a[1].double().T.contiguous()
    rdb = 2.0 * (y[on].double().T.contiguous() @ t)
    assert rel2(host(db[1]), rdb.cpu().numpy()) <= norm_bound(K, M // 3)


def test_many_rows_that_end_inside_a_line():
    """N odd and 2^25 outputs or more: rows share lines, which large outputs write through the caches."""
    M, K, N, R = 2113, 32, 16001, 24
    x, xd = randn(1, (M, K), F16)
    a, ad = randn(2, (3, R, K), BF16)
    b, bd = randn(3, (3, N, R), BF16)
    y, yd = randn(4, (M, N), F32)
    ids = ids_for("runs", M, 3, 8)
    scale = np.array([0.5, 2.0, 1.25], dtype=np.float32)
    at = np.r_[0:40, 1000:1040, M - 40:M]
    ref = oracle.lora_ref(xd[at], ad, bd, scale, ids[at], yd[at])
    args = (x, a, b, torch.from_numpy(scale).to(DEV), torch.from_numpy(ids).to(DEV))
    got = wq.lora_run(*args, y)
    part = np.linalg.norm(ref - yd[at]) / np.linalg.norm(ref)
    assert rel2(host(got)[at], ref) <= norm_bound(K, R) * part + 2 * U
    off = ids < 0
    assert np.array_equal(host(got)[off], host(y)[off])
    assert torch.equal(wq.lora_run(*args, y, out=y), got)              # in place: the same bits


def test_graph_replays():
    """Forward and backward captured once; every replay equals the eager call on the inputs then in place."""
    p = problem((130, 320, 260, 4, 16, BF16, BF16), "runs")
    dy, _ = randn(9, (130, 260), F32, 1e-3)
    out = torch.empty_like(p["y"])
    dx = torch.empty((130, 320), dtype=BF16, device=DEV)
    da, db = torch.empty((4, 16, 320), device=DEV), torch.empty((4, 260, 16), device=DEV)
    w1 = torch.empty(wq.lora_workspace_bytes(130, 320, 260, 4, 16), dtype=torch.uint8, device=DEV)
    w2 = torch.empty(wq.lora_workspace_bytes(130, 320, 260, 4, 16, True), dtype=torch.uint8, device=DEV)

    def both():
        forward(p, out=out, workspace=w1)
        wq.lora_backward(dy, p["x"], p["a"], p["b"], p["scale"], p["ids"], None, dx, da, db, workspace=w2)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        both()
    for i in range(4):
        p["x"].normal_()
        p["ids"].copy_(torch.from_numpy(ids_for(["runs", "random", "none", "bad"][i], 130, 4, i)))
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


@pytest.mark.parametrize("xt,wt,R", [(F32, F16, 64), (F32, BF16, 64), (BF16, BF16, 64), (BF16, BF16, 32), (F32, F32, 32)])
def test_a_row_alone_on_its_adapter(xt, wt, R):
    """Every row of a tile in turn alone on one adapter, the others on another or on none."""
    M, K, N, E = 70, 1040, 64, 32
    p = problem((M, K, N, E, R, xt, wt), "one")
    n = p["n"]
    for rest in (-1, 3):
        for r in range(M):
            ids = np.full(M, rest, dtype=np.int32)
            ids[r] = 30
            p["ids"].copy_(torch.from_numpy(ids))
            ref = oracle.lora_ref(n["x"], n["a"], n["b"], n["scale"], ids, n["y"])
            assert rel2(host(forward(p)) - n["y"], ref - n["y"]) <= norm_bound(K, R) + 1e-6, (rest, r)
