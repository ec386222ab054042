"""block_norm_run and block_norm_backward against float64, element by element.

Bounds.  u = 2^-24.  A sum of n float32 terms in some order is off by at most (its longest chain of additions) u times the
sum of magnitudes.  A row's longest chain here is 8 elements per chunk times the chunks of one thread (4 in held rows, H / 4096
in longer ones), 6 steps across a wave and 8 across the waves: below 48 for rows of up to 16384, below 176 for the longest tested
(131072: 256 + 14, bound 512 u).  Each elementwise step adds at most 8 more.  K = 128 (512 for long rows) covers a row sum, what it
is multiplied into and a second sum over that.  A result rounded to type t adds finfo(t).eps / 2 of itself, and float16 results below
its smallest normal half of the smallest step, 2^-25.  Sums over M rows add at most M u of their magnitudes.
"""
import numpy as np
import pytest
import torch

import oracle
import weight_quantized_mlp_amd as wq
from adapter_common import DEV, U, host, randn

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
EPS = 1e-6
pytestmark = pytest.mark.gpu


def chain(H):
    return 128 if H <= 16384 else 512


def near(got, ref, mag, dtype, factor, what):
    got = host(got).astype(np.float64)
    tol = factor * U * mag + torch.finfo(dtype).eps / 2 * np.abs(ref) * (1 if dtype != F32 else 0) + (2.0 ** -25 if dtype == F16 else 2.0 ** -140)
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), f"{what}: {np.count_nonzero(bad)} of {bad.size}, worst {np.max(np.abs(got - ref) / tol):.2f} of the bound"


def case(M, H, G=1, ht=F32, yt=F32, xt=F32, wt=F32, gt=F32, y=True, post=True, gate=True, pre=True, seed=1):
    c = dict(M=M, H=H, xt=xt)
    c["h"] = randn(seed, (M, H), ht, 3.0)
    c["y"] = randn(seed + 1, (M, H), yt, 0.3) if y else (None, None)
    c["post"] = randn(seed + 2, (H,), wt, 0.5) if y and post else (None, None)
    c["pre"] = randn(seed + 3, (H,), wt, 0.5) if pre else (None, None)
    c["gate"] = randn(seed + 4, (G, H), gt) if y and gate else (None, None)
    return c


def forward(c, alpha=0.7, offset=1.0, **kw):
    (h, hd), (y, yd), (post, postd), (pre, pred), (gate, gated) = (c[k] for k in ("h", "y", "post", "pre", "gate"))
    H = c["H"]
    ho, x = wq.block_norm_run(h.clone(), y, post=post, gate=gate, alpha=alpha, pre=pre, eps=EPS, offset=offset,
                              x_dtype=c["xt"] if pre is not None else None, **kw)
    ref, _ = oracle.block_norm_ref(hd, yd, postd, gated, alpha, None, EPS, offset)
    if y is not None:
        mag = np.abs(hd) + np.abs(ref - hd)
        near(ho, ref, mag, h.dtype, chain(H), "h_out")
    else:
        assert torch.equal(ho, h)
    if pre is not None:      # of the stream as it is stored
        assert x.dtype == c["xt"]
        refx = oracle.norm_ref(host(ho).astype(np.float64), pred, EPS, offset)
        near(x, refx, np.abs(refx), c["xt"], chain(H), "x")
    else:
        assert x is None
    return ho, x


def backward(c, alpha=0.7, offset=1.0, dh=True, need=(True,) * 5, inplace=False, seed=50):
    (h, hd), (y, yd), (post, postd), (pre, pred), (gate, gated) = (c[k] for k in ("h", "y", "post", "pre", "gate"))
    M, H = c["M"], c["H"]
    dh, dhd = randn(seed, (M, H), h.dtype) if dh else (None, None)
    dx, dxd = randn(seed + 1, (M, H), c["xt"]) if pre is not None else (None, None)
    got = wq.block_norm_backward(h, y, dh, dx, post=post, gate=gate, alpha=alpha, pre=pre, eps=EPS, offset=offset, need=need,
                                 dh_in=dh if inplace else None)
    ref = oracle.block_norm_backward_ref(hd, yd, dhd, dxd, postd, gated, alpha, pred, EPS, offset)
    # magnitudes: the same sums over absolute values
    A = np.abs
    du = np.zeros((M, H)) if dhd is None else A(dhd)
    dpre = 0
    if pre is not None:
        r = 1 / np.sqrt(np.mean(hd * hd, axis=1, keepdims=True) + EPS)
        dn = A(dxd * (offset + pred))
        du = du + r * dn + r ** 3 * A(hd) * np.mean(dn * A(hd), axis=1, keepdims=True)
        dpre = np.sum(A(dxd * hd * r), axis=0)
    mags = [du, 0, 0, 0, dpre]
    if y is not None:
        ry = 1.0 if post is None else 1 / np.sqrt(np.mean(yd * yd, axis=1, keepdims=True) + EPS)
        w = 1.0 if post is None else A(offset + postd)
        dp = abs(alpha) * A(oracle.gate_rows(gated, M)) * du
        mags[1] = dp
        if gate is not None:
            G = gated.shape[0]
            mags[3] = np.sum((abs(alpha) * du * A(yd) * ry * w).reshape(G, M // G, H), axis=1)
        if post is not None:
            mags[2] = np.sum(dp * A(yd) * ry, axis=0)
            mags[1] = ry * dp * w + ry ** 3 * A(yd) * np.mean(dp * w * A(yd), axis=1, keepdims=True)
    types = [h.dtype, y.dtype if y is not None else F32, F32, F32, F32]
    for i, name in enumerate(("dh", "dy", "dpost", "dgate", "dpre")):
        if ref[i] is None or not need[i]:
            assert got[i] is None
            continue
        # a chain for each of the two row sums a value may come through, and the sum over the rows
        near(got[i], ref[i], mags[i], types[i], 2 * chain(H) + (M if i >= 2 else 0), name)
    if inplace:
        assert got[0].data_ptr() == dh.data_ptr()
    return got


# held rows of 1, 2 and 4 chunks per thread with whole and partial waves, and rows read again for every pass
SIZES = [(1, 8), (1, 2560), (3, 64), (129, 320), (5, 4096), (7, 4104), (3, 8192), (2, 8200), (4, 16384), (3, 16392), (2, 131072), (700, 72)]


@pytest.mark.parametrize("M,H", SIZES)
def test_sizes(M, H):
    print("[block norm]", M, H, flush=True)
    c = case(M, H)
    forward(c)
    backward(c)


@pytest.mark.parametrize("H", [320, 16392])
@pytest.mark.parametrize("ht,yt,xt,wt,gt", [(BF16, BF16, BF16, BF16, BF16), (F16, F16, F16, F16, F16), (F32, BF16, F16, BF16, F32),
                                            (BF16, F32, F32, F32, F16), (F16, F32, BF16, F16, BF16), (F32, F16, F32, F32, F32),
                                            (BF16, F16, BF16, F32, BF16), (F32, F32, BF16, F32, BF16)])
def test_types(ht, yt, xt, wt, gt, H):
    c = case(13, H, 13, ht, yt, xt, wt, gt)
    forward(c, offset=0.0)
    backward(c, offset=0.0)


@pytest.mark.parametrize("H", [512, 16400])
@pytest.mark.parametrize("y,post,gate,pre", [(False, False, False, True), (True, False, False, True), (True, False, False, False),
                                             (True, True, False, False), (True, False, True, True), (True, True, False, True),
                                             (True, False, True, False), (True, True, True, False)])
def test_absent_parts(y, post, gate, pre, H):
    for dh in (True, False):
        c = case(12, H, 3, y=y, post=post, gate=gate, pre=pre)
        forward(c)
        backward(c, dh=dh)


# gate rows longer than a run of rows, as long, shorter (whole gate rows per run), one row each, and M past the number of runs
@pytest.mark.parametrize("H", [64, 16392])
@pytest.mark.parametrize("M,G", [(1, 1), (130, 1), (130, 13), (130, 130), (1024, 1), (1024, 512), (1024, 1024), (1026, 27), (1500, 500),
                                 (1539, 3), (2050, 1025)])
def test_gate_rows(M, G, H):
    if H > 1000 and M > 1100:        # the float64 reference of long rows takes fewer of them
        M, G = M // 10, 1
    c = case(M, H, G, BF16, BF16, BF16)
    forward(c)
    backward(c)


@pytest.mark.parametrize("which", range(5))
@pytest.mark.parametrize("H", [64, 16392])
def test_each_gradient_alone_is_that_of_all(which, H):
    c = case(40, H, 4)
    everything = backward(c)
    need = tuple(i == which for i in range(5))
    assert torch.equal(backward(c, need=need)[which], everything[which])


@pytest.mark.parametrize("H", [64, 8200, 16392])
def test_in_place(H):
    for ht in (F32, BF16):
        c = case(9, H, 3, ht)
        ho, x = forward(c)
        h = c["h"][0].clone()
        a, b = wq.block_norm_run(h, c["y"][0], post=c["post"][0], gate=c["gate"][0], alpha=0.7, pre=c["pre"][0], eps=EPS, offset=1.0,
                                 x_dtype=F32, h_out=h)
        assert a is h and torch.equal(h, ho) and torch.equal(b, x)
        apart = backward(c)
        for p, q in zip(backward(c, inplace=True), apart):
            assert torch.equal(p, q)


def test_rows_do_not_see_each_other():
    """A row's result is that of a call on it alone, whatever the others hold; a NaN or an infinity stays in its row."""
    c = case(6, 320, 1)
    ho, x = forward(c)
    h, y = c["h"][0].clone(), c["y"][0].clone()
    h[1, 7], y[3, 100], y[4, 5] = float("nan"), float("inf"), float("nan")
    kw = dict(post=c["post"][0], gate=c["gate"][0], alpha=0.7, pre=c["pre"][0], eps=EPS, offset=1.0)
    a, b = wq.block_norm_run(h, y, **kw)
    for m in range(6):
        if m in (1, 3, 4):
            assert not torch.isfinite(b[m]).all()
        else:
            assert torch.equal(a[m], ho[m]) and torch.equal(b[m], x[m])
            one, _ = wq.block_norm_run(h[m:m + 1].contiguous(), y[m:m + 1].contiguous(), **kw)
            assert torch.equal(one[0], a[m])
    dx, dh = randn(9, (6, 320))[0], randn(10, (6, 320))[0]
    whole = wq.block_norm_backward(c["h"][0], c["y"][0], dh, dx, **kw)
    broken = wq.block_norm_backward(h, y, dh, dx, **kw)
    for m in (0, 2, 5):
        assert torch.equal(whole[0][m], broken[0][m]) and torch.equal(whole[1][m], broken[1][m])


def test_an_infinity_in_the_stream_passes_without_a_norm():
    """Without pre, h takes part in the backward pass by nothing: dh passes through it, infinities and NaN or not."""
    for H in (64, 16392):
        h, dh, y = randn(1, (3, H))[0], randn(2, (3, H))[0], randn(3, (3, H))[0]
        h[1, 3], y[2, 5] = float("inf"), float("inf")
        got = wq.block_norm_backward(h, y, dh, alpha=0.5)
        assert torch.equal(got[0], dh) and torch.equal(got[1], dh * 0.5)
        h[0, 0] = float("nan")
        assert torch.equal(wq.block_norm_backward(h, y, dh, alpha=0.5)[0], dh)


def test_zero_rows_and_small_values():
    """Rows of zeros have no direction: eps alone keeps them finite; values whose squares vanish beside eps scale by eps^-1/2."""
    h, y = torch.zeros((3, 256), device=DEV), torch.zeros((3, 256), device=DEV)
    h[1] = 1e-30
    w = torch.ones(256, device=DEV)
    ho, x = wq.block_norm_run(h, y, post=w, pre=w, eps=EPS)
    assert torch.equal(ho, h) and torch.isfinite(x).all()
    assert (x[0] == 0).all() and torch.allclose(x[1], torch.full_like(x[1], 1e-27), rtol=1e-5, atol=0)
    g = wq.block_norm_backward(ho, y, torch.ones_like(h), torch.ones_like(h), post=w, pre=w, eps=EPS)
    assert all(t is None or torch.isfinite(t).all() for t in g)


@pytest.mark.parametrize("H", [64, 16392])
def test_gradients_against_differences(H):
    M, G, alpha, offset = 6, 3, 0.7, 1.0
    c = case(M, H, G)
    (h0, h0d), (y, yd), (post, postd), (pre, pred), (gate, gated) = (c[k] for k in ("h", "y", "post", "pre", "gate"))
    kw = dict(post=post, gate=gate, alpha=alpha, pre=pre, eps=EPS, offset=offset)
    ho, _ = wq.block_norm_run(h0, y, **kw)
    (ca, cad), (cb, cbd) = randn(30, (M, H)), randn(31, (M, H))          # loss: sum(ca h_out) + sum(cb x)
    got = wq.block_norm_backward(ho, y, ca, cb, **kw)

    def loss(h, y, post, gate, pre):
        ho, x = oracle.block_norm_ref(h, y, post, gate, alpha, pre, EPS, offset)
        return np.sum(cad * ho) + np.sum(cbd * x)
    at = [h0d, yd, postd, gated, pred]
    for i in range(5):
        d = np.random.default_rng(i).standard_normal(at[i].shape)
        d += host(got[i]) / np.linalg.norm(host(got[i])) * np.sqrt(d.size)
        t = 1e-5
        up, down = [list(at) for _ in range(2)]
        up[i], down[i] = at[i] + t * d, at[i] - t * d
        slope = (loss(*up) - loss(*down)) / (2 * t)
        want = np.sum(host(got[i]).astype(np.float64) * d)
        # second-order differences leave about t^2 of the third derivative; float32 gradients their 2^-24 times a few
        assert abs(want - slope) <= 1e-4 * abs(slope) + 1e-6 * np.linalg.norm(d), (i, want, slope)


def test_a_replayed_graph_reads_new_values():
    """Forward and backward captured once, replayed on changed inputs, with eager calls and synchronisations in between."""
    c = case(300, 640, 3, BF16, BF16, BF16, BF16, BF16)
    h, y, post, pre, gate = (c[k][0] for k in ("h", "y", "post", "pre", "gate"))
    dh, dx = randn(7, (300, 640), BF16)[0], randn(8, (300, 640), BF16)[0]
    kw = dict(post=post, gate=gate, alpha=0.7, pre=pre, eps=EPS)

    def step():
        ho, x = wq.block_norm_run(h, y, x_dtype=BF16, **kw)
        return (ho, x) + wq.block_norm_backward(ho, y, dh, dx, **kw)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = step()
    for i in range(3):
        h.copy_(randn(100 + i, (300, 640), BF16)[0])
        dx.copy_(randn(200 + i, (300, 640), BF16)[0])
        want = step()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert torch.equal(a, b)


def test_two_streams_at_once():
    cs = [case(600, 2048, 3, BF16, BF16, BF16, seed=s) for s in (1, 11)]
    dxs = [randn(5 + i, (600, 2048), BF16)[0] for i in range(2)]
    run = lambda c, dx: wq.block_norm_backward(c["h"][0], c["y"][0], None, dx, post=c["post"][0], gate=c["gate"][0], pre=c["pre"][0])
    want = [run(c, dx) for c, dx in zip(cs, dxs)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    got = []
    for s, c, dx in zip(streams, cs, dxs):
        with torch.cuda.stream(s):
            got.append([run(c, dx) for _ in range(5)])
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        for r in g:
            assert all(torch.equal(a, b) for a, b in zip(w, r))


def test_no_rows():
    e = lambda *s: torch.empty(s, device=DEV)
    w, gate = torch.ones(64, device=DEV), torch.ones((1, 64), device=DEV)
    ho, x = wq.block_norm_run(e(0, 64), e(0, 64), post=w, gate=gate, pre=w)
    assert ho.shape == x.shape == (0, 64)
    got = wq.block_norm_backward(e(0, 64), e(0, 64), e(0, 64), e(0, 64), post=w, gate=gate, pre=w,
                                 dpost=torch.ones(64, device=DEV), dgate=torch.ones((1, 64), device=DEV))
    assert got[0].shape == got[1].shape == (0, 64)
    assert all((t == 0).all() for t in got[2:])


def test_refusals_of_the_binding():
    c = case(12, 64, 3)
    h, y, post, pre, gate = (c[k][0] for k in ("h", "y", "post", "pre", "gate"))
    with pytest.raises(ValueError, match="divisor"):
        wq.block_norm_run(h, y, gate=torch.ones((5, 64), device=DEV))
    with pytest.raises(ValueError, match="nothing to do"):
        wq.block_norm_run(h)
    with pytest.raises(ValueError, match="need y"):
        wq.block_norm_run(h, post=post, pre=pre)
    with pytest.raises(ValueError, match="need pre"):
        wq.block_norm_run(h, y, x_dtype=F32)
    with pytest.raises(TypeError, match="x_dtype"):
        wq.block_norm_run(h, pre=pre, x_dtype=BF16, x=torch.empty_like(h))
    with pytest.raises(TypeError):
        wq.block_norm_run(h, y, post=post, pre=pre.to(BF16))
    with pytest.raises(ValueError, match="contiguous"):
        wq.block_norm_run(h, y.t().contiguous().t(), pre=pre)
    with pytest.raises(ValueError, match="elements"):
        wq.block_norm_run(h, y[:6].contiguous(), pre=pre)
    with pytest.raises(ValueError, match="come together"):
        wq.block_norm_backward(h, y, dx=h, post=post)
    with pytest.raises(ValueError, match="not computed"):
        wq.block_norm_backward(h, y, dx=h, pre=pre, dpost=torch.empty(64, device=DEV))
    with pytest.raises(wq.WQError):
        wq.block_norm_run(h, h, pre=pre, h_out=h)                    # in place over y, too
    with pytest.raises(wq.WQError):
        wq.block_norm_backward(h, y, h, h, pre=pre, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
