"""moe_awq_run against float64: router, choice, experts and sum.

Bounds.  u = 2^-24.  ids must be those of the float64 logits rounded to float32.  Weights: the difference of two float32 logits is
rounded once (an absolute error of u |difference| becomes a relative one of exp), exp is good to 2 u, sums of up to 16 (512 for the
softmax over all: 8 terms per lane and 6 steps across a wave) add at most 16 u: (24 + |difference|) u, 64 u for differences up to 40.
A product of n terms is off by at most 2 (n + 8) u times its sum of magnitudes, and by 2^-22 of it where float32 values enter as two
terms; where rows are scaled, by 2^-39 of the row's largest times the sum of the weights' magnitudes.  |silu'| <= 1.1, so
d act <= 1.1 dg |u| + |silu(g)| du + 8 u |act|.  out sums topk products and is rounded once to its type.
"""
import numpy as np
import pytest
import torch

import weight_quantized_mlp_amd as wq
from adapter_common import DEV, U, host, norm_bound, randn, rel2
from awq_common import awq_weights

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
pytestmark = pytest.mark.gpu
_cache = {}


def layer(E, H, I, layout):
    if (E, H, I, layout) not in _cache:
        _cache[E, H, I, layout] = awq_weights(1, E, 2 * I, H, layout) + awq_weights(2, E, H, I, layout)
    return _cache[E, H, I, layout]


def route_ref(xd, rd, topk, renorm):
    """ids and float64 weights of the float32-rounded float64 logits, ties to the lower index."""
    logits = (xd @ rd.T).astype(np.float32)
    ids = np.argsort(-logits, axis=1, kind="stable")[:, :topk]
    l64 = logits.astype(np.float64)
    top = np.take_along_axis(l64, ids, axis=1)
    p = np.exp(top - top[:, :1])
    total = p.sum(axis=1, keepdims=True) if renorm else np.exp(l64 - top[:, :1]).sum(axis=1, keepdims=True)
    return ids, p / total


def linear_bound(x, w, xt):
    """|x| |w|^T and how far the kernel's x w^T may be off."""
    mag = np.abs(x) @ np.abs(w).T
    b = 2 * (x.shape[1] + 8) * U * mag
    if xt != F16:
        b += 2.0 ** -39 * np.abs(x).max(axis=1, keepdims=True) * np.abs(w).sum(axis=1)[None]
    if xt == F32:
        b += 2.0 ** -22 * mag
    return b


def layer_ref(xd, xt, ids, weights, w13, w2):
    """(out, bound) in float64; ids outside the experts contribute nothing."""
    E, I2, H = w13.shape
    I = I2 // 2
    out, bound = np.zeros_like(xd), np.zeros_like(xd)
    for e in np.unique(ids):
        if e < 0 or e >= E:
            continue
        rows, k = np.nonzero(ids == e)
        x = xd[rows]
        g, u = x @ w13[e, :I].T, x @ w13[e, I:].T
        dg, du = linear_bound(x, w13[e, :I], xt), linear_bound(x, w13[e, I:], xt)
        silu = g / (1 + np.exp(-g))
        act = silu * u
        dact = 1.1 * dg * np.abs(u) + np.abs(silu) * du + 1.1 * dg * du + 8 * U * np.abs(act)
        y = act @ w2[e].T
        dy = dact @ np.abs(w2[e]).T + linear_bound(act, w2[e], F32)
        wt = weights[rows, k][:, None]
        np.add.at(out, rows, wt * y)
        np.add.at(bound, rows, np.abs(wt) * (dy + 32 * U * np.abs(y)))
    return out, bound


def check(got, ref, bound, dtype, H, weights_u=0):
    g = host(got).astype(np.float64)
    tol = bound + weights_u * U * np.abs(ref) + (torch.finfo(dtype).eps / 2 * np.abs(ref) * 1.01 if dtype != F32 else 0) + (2.0 ** -25 if dtype == F16 else 1e-37)
    assert np.all(np.abs(g - ref) <= tol), np.max(np.abs(g - ref) / tol)
    err = rel2(got.double().cpu().numpy(), ref)
    assert err <= norm_bound(2 * H) + (torch.finfo(dtype).eps / 2 if dtype != F32 else 0), err


# M, E, topk, H, I: routes fewer, as many and more than experts; one expert for all (more than 16 tokens each: several passes); contractions of
# one group, a few steps and enough for all waves; float32 rows staged in parts
SHAPES = [(1, 16, 4, 256, 64), (1, 1, 1, 32, 32), (2, 8, 2, 320, 96), (3, 64, 10, 2560, 160), (5, 4, 4, 64, 288), (17, 2, 2, 160, 64),
          (37, 16, 3, 1056, 544), (40, 1, 1, 2592, 32), (130, 12, 6, 512, 192), (256, 40, 16, 96, 64)]


@pytest.mark.parametrize("xt,rt,ot", [(F32, F32, F32), (BF16, BF16, F32), (F16, F32, F32), (BF16, F16, BF16), (F16, F16, F16)])
@pytest.mark.parametrize("M,E,topk,H,I", SHAPES)
def test_layer(M, E, topk, H, I, xt, rt, ot):
    layout, renorm = 3 + (M + E) % 2, (M + topk) % 3 != 0
    print("[moe layer]", M, E, topk, H, I, xt, rt, ot, layout, renorm, flush=True)
    b13, w13, b2, w2 = layer(E, H, I, layout)
    x, xd = randn(M + H, (M, H), xt)
    router, rd = randn(E + 1, (E, H), rt, 2 * H ** -0.5)
    guard = torch.full((M * H + 64,), 7.0, device=DEV, dtype=ot)
    out, ids, weights = wq.moe_awq_run(x, b13, b2, E, I, topk, router=router, renorm=renorm, meta_layout=layout,
                                       out=guard[: M * H].view(M, H))
    assert (guard[M * H:] == 7.0).all() and ids.dtype == torch.int32 and weights.dtype == F32
    ref_ids, ref_w = route_ref(xd, rd, topk, renorm)
    assert np.array_equal(host(ids), ref_ids)
    assert np.all(np.abs(host(weights) - ref_w) <= 64 * U * ref_w)
    ref, bound = layer_ref(xd, xt, ref_ids, ref_w, w13, w2)
    check(out, ref, bound, ot, H + I, 64)
    # the same ids and weights given
    again, _, _ = wq.moe_awq_run(x, b13, b2, E, I, ids=ids, weights=weights, meta_layout=layout, dtype=ot)
    assert torch.equal(again, out)


def test_given_routes_out_of_range_and_repeated():
    """Ids outside the experts count for nothing, repeated ones once each with their own weight, weights of any sign and size."""
    M, E, topk, H, I = 9, 6, 8, 128, 64
    b13, w13, b2, w2 = layer(E, H, I, 3)
    x, xd = randn(3, (M, H), BF16)
    r = np.random.default_rng(1)
    ids = r.integers(-2, E + 2, (M, topk)).astype(np.int32)
    ids[0], ids[1], ids[2] = -1, 3, [0, 0, 1 << 30, -(1 << 31), E, 5, 5, 5]
    wt = r.standard_normal((M, topk)).astype(np.float32)
    wt[3] = 0
    out, _, _ = wq.moe_awq_run(x, b13, b2, E, I, ids=torch.from_numpy(ids).to(DEV), weights=torch.from_numpy(wt).to(DEV), dtype=F32)
    ref, bound = layer_ref(xd, BF16, ids, wt.astype(np.float64), w13, w2)
    g = host(out)
    assert np.all(np.abs(g - ref) <= bound + 1e-37)
    assert (g[0] == 0).all() and (g[3] == 0).all()
    none = torch.full((M, topk), -1, dtype=torch.int32, device=DEV)
    assert (wq.moe_awq_run(x, b13, b2, E, I, ids=none, weights=torch.ones((M, topk), device=DEV))[0] == 0).all()


def test_ties_and_values_that_are_no_numbers():
    """Equal logits go to the lower index, -0 equals 0, NaN comes last, an infinity first."""
    E, H, I, topk = 8, 64, 32, 5
    b13, _, b2, _ = layer(E, H, I, 3)
    x = torch.zeros((3, H), device=DEV)
    x[:, 0] = 1
    x[1, 0] = -1
    router = torch.zeros((E, H), device=DEV)
    router[:, 0] = torch.tensor([0.0, 2.0, -0.0, 2.0, 1.0, -1.0, 2.0, 0.0])
    _, ids, w = wq.moe_awq_run(x, b13, b2, E, I, topk, router=router)
    assert ids[0].tolist() == [1, 3, 6, 4, 0] and ids[1].tolist() == [5, 0, 2, 7, 4]
    assert torch.allclose(w.sum(dim=1), torch.ones(3, device=DEV)) and w[0, 0] == w[0, 1] == w[0, 2]
    router[:, 0] = torch.tensor([float("nan"), 1.0, float("inf"), float("nan"), -float("inf"), 0.5, 1.0, -3.0])
    x[:, 0] = 1
    _, ids, w = wq.moe_awq_run(x, b13, b2, E, I, 8, router=router)
    assert ids[0].tolist() == [2, 1, 6, 5, 7, 4, 0, 3]
    x[1, 5] = float("nan")                                              # every logit of that row is NaN, the others stay
    clean = wq.moe_awq_run(x[::2].contiguous(), b13, b2, E, I, 3, router=router.nan_to_num(0, 1, -1))
    out, ids, w = wq.moe_awq_run(x, b13, b2, E, I, 3, router=router.nan_to_num(0, 1, -1))
    assert ids[1].tolist() == [0, 1, 2] and torch.isnan(out[1]).all()
    assert torch.equal(out[::2], clean[0]) and torch.equal(ids[::2], clean[1])


@pytest.mark.parametrize("xt", [F32, BF16, F16])
def test_a_token_is_the_same_in_every_batch(xt):
    """The same bits alone, among others, at another place and next to rows of NaN, whether a workgroup belongs to a route or an expert."""
    M, E, topk, H, I = 40, 6, 3, 2592, 160
    b13, _, b2, _ = layer(E, H, I, 3)
    x, _ = randn(5, (M, H), xt)
    router, _ = randn(6, (E, H), F32, H ** -0.5)
    run = lambda t: wq.moe_awq_run(t.contiguous(), b13, b2, E, I, topk, router=router, dtype=F32)
    out, ids, w = run(x)
    for rows in ([0], [7], [3, 39], list(range(20)), list(range(39, -1, -1))):
        o, i, ww = run(x[rows])
        assert torch.equal(o, out[rows]) and torch.equal(i, ids[rows]) and torch.equal(ww, w[rows])
    bad = x.clone()
    bad[1::2] = float("nan")
    o, i, _ = run(bad)
    assert torch.equal(o[::2], out[::2]) and torch.equal(i[::2], ids[::2])


def test_agrees_with_the_single_token_step():
    """moe_awq_m1_run rounds gate, up, act and each route's result to float16: four roundings of 2^-11 at most each, which random signs
    leave near 2^-11 of the result's norm; four times that."""
    E, topk, H, I = 16, 4, 256, 64
    b13, _, b2, _ = layer(E, H, I, 3)
    x, _ = randn(1, (1, H), F16)
    router, _ = randn(2, (E, H), F32, H ** -0.5)
    out, ids, w = wq.moe_awq_run(x, b13, b2, E, I, topk, router=router, dtype=F32)
    step, _ = wq.moe_awq_m1_run(x[0].contiguous(), ids[0].contiguous(), w[0].contiguous(), b13, b2, E, I)
    assert rel2(host(step), host(out[0])) <= 4 * 2.0 ** -11


def test_gates_far_from_zero():
    """silu of large gates of either sign: no overflow, and act rows of unlike sizes keep their precision."""
    M, E, topk, H, I = 4, 3, 2, 64, 64
    b13, w13, b2, w2 = layer(E, H, I, 4)
    x, xd = randn(8, (M, H), F32, 1.0)
    scale = np.array([1e4, 1e-4, 1e12, 1.0])[:, None]
    x, xd = (x * torch.from_numpy(scale).float().to(DEV)), None
    xd = x.double().cpu().numpy()
    ids = torch.tensor([[0, 1], [1, 2], [2, 0], [0, 2]], dtype=torch.int32, device=DEV)
    w = torch.full((M, topk), 0.5, device=DEV)
    out, _, _ = wq.moe_awq_run(x, b13, b2, E, I, ids=ids, weights=w, meta_layout=4)
    with np.errstate(over="ignore"):
        ref, bound = layer_ref(xd, F32, host(ids), host(w).astype(np.float64), w13, w2)
    g = host(out)
    # where a gate is so far below zero that silu underflows, float32 gives 0: 2^-126 of what it multiplies
    assert np.all(np.abs(g - ref) <= bound + 1e-37 * np.abs(xd).max(axis=1, keepdims=True))


@pytest.mark.parametrize("M", [1, 12])
def test_a_replayed_graph_reads_new_values(M):
    E, topk, H, I = 32, 4, 512, 96
    b13, _, b2, _ = layer(E, H, I, 3)
    x, _ = randn(1, (M, H), BF16)
    router, _ = randn(2, (E, H), BF16, H ** -0.5)
    run = lambda: wq.moe_awq_run(x, b13, b2, E, I, topk, router=router)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        run()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = run()
    for i in range(3):
        x.copy_(randn(20 + i, (M, H), BF16)[0])
        want = run()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_two_streams_at_once():
    E, topk, H, I = 32, 4, 512, 96
    b13, _, b2, _ = layer(E, H, I, 3)
    xs = [randn(i, (11 + i, H), BF16)[0] for i in range(2)]
    router, _ = randn(2, (E, H), BF16, H ** -0.5)
    want = [wq.moe_awq_run(x, b13, b2, E, I, topk, router=router) for x in xs]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in xs], []
    for s, x in zip(streams, xs):
        with torch.cuda.stream(s):
            got.append([wq.moe_awq_run(x, b13, b2, E, I, topk, router=router) for _ in range(10)])
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        for r in g:
            assert all(torch.equal(a, b) for a, b in zip(w, r))


def test_experts_past_4_GiB():
    """The last experts of a bank whose byte offsets pass 2^32 give what a small bank of just them gives."""
    E, topk, H, I, M = 3700, 2, 2560, 160, 3
    n13, n2 = wq.awq_bank_bytes(1, 2 * I, H), wq.awq_bank_bytes(1, H, I)
    s13, w13, s2, w2 = layer(2, H, I, 3)
    b13 = torch.zeros((E, n13), dtype=torch.uint8, device=DEV)
    E2 = E
    b2 = torch.zeros((E2, n2), dtype=torch.uint8, device=DEV)
    while b13.numel() <= 1 << 32:                                       # (a larger bank where the sizes above do not pass it)
        E *= 3
        b13 = torch.zeros((E, n13), dtype=torch.uint8, device=DEV)
        b2 = torch.zeros((E, n2), dtype=torch.uint8, device=DEV)
    b13[E - 2:] = s13.view(2, n13)
    b2[E - 2:] = s2.view(2, n2)
    x, _ = randn(1, (M, H), BF16)
    ids = torch.tensor([[0, 1], [1, 0], [1, 1]], dtype=torch.int32, device=DEV)
    w = torch.tensor([[0.3, 0.7], [0.5, 0.5], [1.0, -0.5]], device=DEV)
    small, _, _ = wq.moe_awq_run(x, s13, s2, 2, I, ids=ids, weights=w)
    large, _, _ = wq.moe_awq_run(x, b13.view(-1), b2.view(-1), E, I, ids=ids + (E - 2), weights=w)
    assert torch.equal(small, large)


def test_empty_and_refused_calls():
    E, topk, H, I = 4, 2, 64, 32
    b13, _, b2, _ = layer(E, H, I, 3)
    router = torch.ones((E, H), device=DEV)
    out, ids, w = wq.moe_awq_run(torch.empty((0, H), device=DEV), b13, b2, E, I, topk, router=router)
    assert out.shape == (0, H) and ids.shape == w.shape == (0, topk)
    x, _ = randn(1, (3, H))
    with pytest.raises(ValueError, match="topk must be given"):
        wq.moe_awq_run(x, b13, b2, E, I, router=router)
    with pytest.raises(ValueError, match="without router"):
        wq.moe_awq_run(x, b13, b2, E, I, topk)
    with pytest.raises(wq.WQError):
        wq.moe_awq_run(x, b13, b2, E, I, 5, router=router)              # more than there are
    with pytest.raises(wq.WQError):
        wq.moe_awq_run(torch.zeros((257, H), device=DEV), b13, b2, E, I, topk, router=router)
    with pytest.raises(ValueError):
        wq.moe_awq_run(x, b13, b2, E, I, topk, router=router[:2].contiguous())
    with pytest.raises(TypeError):
        wq.moe_awq_run(x, b13, b2, E, I, ids=torch.zeros((3, 2), dtype=torch.int64, device=DEV), weights=torch.ones((3, 2), device=DEV))
    with pytest.raises(TypeError, match="out is"):
        wq.moe_awq_run(x, b13, b2, E, I, topk, router=router, dtype=BF16, out=torch.empty_like(x))
    with pytest.raises(wq.WQError):
        wq.moe_awq_run(x, b13, b2, E, I, topk, router=router, out=x)
    with pytest.raises(wq.WQError):
        wq.moe_awq_run(x, b13, b2, E, I, topk, router=router, workspace=torch.empty(64, dtype=torch.uint8, device=DEV))


@pytest.mark.parametrize("E,topk", [(65, 16), (200, 10), (300, 7), (512, 16), (1000, 10), (1024, 1), (1500, 16), (5000, 3)])
@pytest.mark.parametrize("renorm", [True, False])
def test_choice_among_many_experts(E, topk, renorm):
    """Every number of experts per lane, and more than a wave keeps; half of the logits in ties."""
    M, H, I = 5, 32, 32
    nb13, nb2 = wq.awq_bank_bytes(E, 2 * I, H, 3), wq.awq_bank_bytes(E, H, I, 3)
    b13, b2 = torch.zeros(nb13, dtype=torch.uint8, device=DEV), torch.zeros(nb2, dtype=torch.uint8, device=DEV)
    x, xd = randn(E, (M, H), F32)
    router, rd = randn(E + 1, (E, H), F32, 0.5)
    router[E // 2:] = router[:E - E // 2].clone()
    rd[E // 2:] = rd[:E - E // 2].copy()
    out, ids, weights = wq.moe_awq_run(x, b13, b2, E, I, topk, router=router, renorm=renorm)
    ref_ids, ref_w = route_ref(xd, rd, topk, renorm)
    assert np.array_equal(host(ids), ref_ids)
    assert np.all(np.abs(host(weights) - ref_w) <= (64 + E / 32) * U * ref_w)      # (without renorm, E / 64 terms per lane)
    assert (out == 0).all()                                                        # (zero scales)
