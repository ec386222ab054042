"""The block calls together, as a model would use them: a serving chain (norm, 4-bit MLP, norm with gate and residual, routed experts,
norm) and a training chain (norm, frozen 4-bit projection with an adapter, norm, and all their gradients).

Serving is checked stage by stage against float64 on what the stage before stored, with the bounds of the single calls: u = 2^-24; a
row sum of the norms and what it enters is off by at most 128 u of its magnitudes (rows below 16384); a product of n terms by
2 (n + 8) u of its sum of magnitudes, 2^-22 of it for float32 operands and 2^-39 of the row's largest times the weights' magnitudes;
a result rounded to 16 bits by half a step.

Training is in float32 throughout and checked end to end in the 2-norm.  Every sum of n terms errs by about sqrt(n) u of its norm for
inputs of random sign, two-term operands by 2^-22; norm_bound over all lengths of a gradient's way is 8 times their root sum of squares.
The ways of a gradient (through the projection, the adapter, the stream) add where they meet: at most four of them.
"""
import numpy as np
import pytest
import torch

import oracle
import weight_quantized_mlp_amd as wq
from adapter_common import DEV, U, host, norm_bound, randn, rel2
from awq_common import awq_weights
from test_moe_layer import layer, layer_ref, linear_bound, route_ref

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
EPS, ALPHA = 1e-6, 0.5
pytestmark = pytest.mark.gpu


def f64(t):
    return t.double().cpu().numpy()


def near(got, ref, bound, what):
    g = f64(got)
    t = torch.finfo(got.dtype).eps / 2 if got.dtype != F32 else 0
    tol = bound + t * np.abs(ref) * 1.01 + (2.0 ** -25 if got.dtype == F16 else 1e-37)
    assert np.all(np.abs(g - ref) <= tol), f"{what}: {np.max(np.abs(g - ref) / tol):.2f} of the bound"


class Model:
    """Two blocks: a SwiGLU MLP from two 4-bit linears, then routed experts; the types of the stream and of the blocks' inputs."""
    H, I, E, topk, EI = 320, 416, 12, 3, 96

    def __init__(self, ht, xt, layout):
        self.ht, self.xt, self.layout = ht, xt, layout
        self.up, self.up64 = awq_weights(11, 1, 2 * self.I, self.H, layout)
        self.down, self.down64 = awq_weights(12, 1, self.H, self.I, layout)
        self.w13, self.w1364, self.w2, self.w264 = layer(self.E, self.H, self.EI, layout)
        self.router, self.router64 = randn(13, (self.E, self.H), xt, 2 * self.H ** -0.5)
        self.norms = [randn(14 + i, (self.H,), BF16, 0.3) for i in range(5)]
        self.gate, self.gate64 = randn(20, (self.H,), F32)

    def workspace(self, M):
        n = max(wq.awq_linear_workspace_bytes(M, 2 * self.I, self.H, self.xt), wq.awq_linear_workspace_bytes(M, self.H, self.I, self.xt),
                wq.moe_awq_workspace_bytes(M, self.E, self.topk, self.H, self.EI))
        return torch.empty(n, dtype=torch.uint8, device=DEV)

    def run(self, h, ws):
        """Every stage's result; the stream is updated in a copy of h, one workspace serves all calls."""
        n = [t for t, _ in self.norms]
        s = {"h0": h}
        _, s["x0"] = wq.block_norm_run(h, pre=n[0], eps=EPS, offset=1.0, x_dtype=self.xt)
        s["gu"] = wq.awq_linear_run(s["x0"], self.up, 2 * self.I, self.layout, workspace=ws)
        s["act"] = (torch.nn.functional.silu(s["gu"][:, :self.I]) * s["gu"][:, self.I:]).to(self.xt)
        s["y0"] = wq.awq_linear_run(s["act"], self.down, self.H, self.layout, workspace=ws)
        s["h1"], s["x1"] = wq.block_norm_run(h, s["y0"], post=n[1], gate=self.gate, alpha=ALPHA, pre=n[2], eps=EPS, offset=1.0,
                                             x_dtype=self.xt)
        s["y1"], s["ids"], s["weights"] = wq.moe_awq_run(s["x1"], self.w13, self.w2, self.E, self.EI, self.topk, router=self.router,
                                                         meta_layout=self.layout, dtype=F32, workspace=ws)
        stream = s["h1"].clone()
        s["h2"], s["x2"] = wq.block_norm_run(stream, s["y1"], post=n[3], pre=n[4], eps=EPS, offset=1.0, h_out=stream, x_dtype=F32)
        return s


TYPES = [(BF16, BF16, 3), (F32, F32, 4), (F16, F16, 3), (F32, BF16, 4)]


@pytest.mark.parametrize("ht,xt,layout", TYPES)
@pytest.mark.parametrize("M", [1, 2, 7, 40, 150])
def test_serving(M, ht, xt, layout):
    print("[chain]", M, ht, xt, layout, flush=True)
    m = Model(ht, xt, layout)
    s = m.run(randn(M, (M, m.H), ht, 2.0)[0], m.workspace(M))
    v = {k: f64(t) for k, t in s.items()}
    n = [w for _, w in m.norms]

    def norm(h, w, got, what):
        ref = oracle.norm_ref(h, w, EPS, 1.0)
        near(got, ref, 128 * U * np.abs(ref), what)

    norm(v["h0"], n[0], s["x0"], "x0")
    near(s["gu"], v["x0"] @ m.up64[0].T, linear_bound(v["x0"], m.up64[0], xt), "gu")
    near(s["y0"], v["act"] @ m.down64[0].T, linear_bound(v["act"], m.down64[0], xt), "y0")
    p = ALPHA * m.gate64 * oracle.norm_ref(v["y0"], n[1], EPS, 1.0)
    near(s["h1"], v["h0"] + p, 128 * U * (np.abs(v["h0"]) + np.abs(p)), "h1")
    norm(v["h1"], n[2], s["x1"], "x1")
    ids, weights = route_ref(v["x1"], m.router64, m.topk, True)
    assert np.array_equal(host(s["ids"]), ids)
    ref, bound = layer_ref(v["x1"], xt, ids, weights, m.w1364, m.w264)
    near(s["y1"], ref, bound + 64 * U * np.abs(ref), "y1")
    p = oracle.norm_ref(v["y1"], n[3], EPS, 1.0)
    near(s["h2"], v["h1"] + p, 128 * U * (np.abs(v["h1"]) + np.abs(p)), "h2")
    norm(v["h2"], n[4], s["x2"], "x2")


@pytest.mark.parametrize("M", [1, 24, 70])
def test_serving_in_a_graph(M):
    """Replays follow the stream's new values, whatever ran in between, with one workspace for all calls of the chain."""
    m = Model(BF16, BF16, 3)
    h, ws = torch.empty((M, m.H), dtype=BF16, device=DEV), m.workspace(M)
    inputs = [randn(30 + i, (M, m.H), BF16, 1.0 + i)[0] for i in range(4)]
    want = [m.run(x, ws) for x in inputs]
    side = torch.cuda.Stream()
    h.copy_(inputs[0])
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        m.run(h, ws)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s = m.run(h, ws)
    for x, w in zip(inputs, want):
        h.copy_(x)
        g.replay()
        ws.clone().sum().item()                                 # (eager work and a synchronisation between replays)
        for k in ("gu", "y0", "h1", "ids", "weights", "y1", "h2", "x2"):
            assert torch.equal(s[k], w[k]), k


@pytest.mark.parametrize("M", [2, 24, 70])
def test_serving_on_two_streams(M):
    m = Model(F32, F16, 4)
    inputs = [randn(40 + i, (M, m.H), F32)[0] for i in range(2)]
    spaces = [m.workspace(M) for _ in inputs]
    want = [m.run(x, spaces[0]) for x in inputs]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in inputs], []
    for s, x, ws in zip(streams, inputs, spaces):
        with torch.cuda.stream(s):
            for _ in range(4):
                r = m.run(x, ws)
            got.append(r)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        for k in ("gu", "y0", "h1", "y1", "h2", "x2"):
            assert torch.equal(a[k], b[k]), k


class Training:
    """h1, x = norm(h + alpha gate norm(y)); t = x W^T + adapter; h2, z = norm(h1 + gate2 norm(t)); the loss is linear in z and h2."""
    M, H, E, R, G = 96, 256, 3, 8, 6

    def __init__(self, seed):
        H, M = self.H, self.M
        self.bank, w = awq_weights(seed, 1, H, H, 3, std=0.06)
        self.w64 = torch.from_numpy(w[0])
        shapes = dict(h=(M, H), y=(M, H), post=(H,), gate=(self.G, H), pre=(H,), a=(self.E, self.R, H), b=(self.E, H, self.R),
                      post2=(H,), gate2=(H,), pre2=(H,), cz=(M, H), ch=(M, H))
        std = dict(a=H ** -0.5, post=0.3, pre=0.3, post2=0.3, pre2=0.3)
        self.p = {k: randn(seed + i, s, F32, std.get(k, 1.0))[0] for i, (k, s) in enumerate(shapes.items())}
        self.scale = torch.tensor([0.5, 2.0, 1.0], device=DEV)
        ids = np.random.default_rng(seed).integers(-1, self.E, M).astype(np.int32)
        self.ids = torch.from_numpy(np.sort(ids)).to(DEV)

    def gradients(self):
        p = self.p
        h1, x = wq.block_norm_run(p["h"], p["y"], post=p["post"], gate=p["gate"], alpha=ALPHA, pre=p["pre"], eps=EPS, offset=1.0)
        t = wq.awq_linear_run(x, self.bank, self.H)
        t = wq.lora_run(x, p["a"], p["b"], self.scale, self.ids, t)
        h2, _ = wq.block_norm_run(h1, t, post=p["post2"], gate=p["gate2"], pre=p["pre2"], eps=EPS, offset=1.0)
        g = {}
        dh1, dt, g["post2"], g["gate2"], g["pre2"] = wq.block_norm_backward(h2, t, p["ch"], p["cz"], post=p["post2"], gate=p["gate2"],
                                                                            pre=p["pre2"], eps=EPS, offset=1.0)
        dx = wq.awq_linear_backward(dt, self.bank, self.H)
        dx, g["a"], g["b"] = wq.lora_backward(dt, x, p["a"], p["b"], self.scale, self.ids, dx0=dx, dx=dx)
        g["h"], g["y"], g["post"], g["gate"], g["pre"] = wq.block_norm_backward(
            h1, p["y"], dh1, dx, post=p["post"], gate=p["gate"], alpha=ALPHA, pre=p["pre"], eps=EPS, offset=1.0, dh_in=dh1)
        return g

    def loss(self, p):
        """In float64 on the CPU."""
        def norm(t, w):
            return t / torch.sqrt((t * t).mean(dim=1, keepdim=True) + EPS) * (1 + w)
        h1 = p["h"] + ALPHA * p["gate"].repeat_interleave(self.M // self.G, dim=0) * norm(p["y"], p["post"])
        x = norm(h1, p["pre"])
        t = x @ self.w64.T
        ids, scale = self.ids.cpu(), self.scale.double().cpu()
        for e in range(self.E):
            rows = (ids == e).double()[:, None]
            t = t + rows * scale[e] * ((x @ p["a"][e].T) @ p["b"][e].T)
        h2 = h1 + p["gate2"] * norm(t, p["post2"])
        return (norm(h2, p["pre2"]) * p["cz"]).sum() + (h2 * p["ch"]).sum()

    def bound(self):
        lengths = 2 * (4 * self.H + 2 * self.R) + 2 * self.M
        return 4 * norm_bound(lengths) + 2.0 ** -20


@pytest.mark.parametrize("seed", [1, 50])
def test_training(seed):
    """Every gradient of the chain against the formula's, and all of them together against differences of the loss."""
    c = Training(seed)
    got = {k: v.double().cpu() for k, v in c.gradients().items()}
    p = {k: v.double().cpu().requires_grad_(k in got) for k, v in c.p.items()}
    c.loss(p).backward()
    for k, v in got.items():
        err = rel2(v.numpy(), p[k].grad.numpy())
        assert err <= c.bound(), f"{k}: {err:.2e} > {c.bound():.2e}"
    # along random directions: the difference's own error is of order step^2 and 2^-52 / step, far below the bound
    with torch.no_grad():
        for i, k in enumerate(got):
            d = torch.from_numpy(np.random.default_rng(seed + i).standard_normal(got[k].shape))
            step = 1e-5
            up, down = ({n: (v + s * d if n == k else v) for n, v in p.items()} for s in (step, -step))
            diff = (c.loss(up) - c.loss(down)).item() / (2 * step)
            slack = (c.bound() + 1e-6) * (got[k].norm() * d.norm()).item()
            assert abs(diff - (got[k] * d).sum().item()) <= slack, k


def test_training_step_in_a_graph():
    """Forward and backward in one graph; replays follow new parameters, with eager runs of the same calls between them."""
    c = Training(7)
    c.gradients()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        static = c.gradients()
    for i in range(3):
        for k in ("h", "y", "a", "gate", "pre2"):
            c.p[k].copy_(randn(60 + 10 * i, tuple(c.p[k].shape))[0])
        want = c.gradients()
        g.replay()
        torch.cuda.synchronize()
        for k, v in want.items():
            assert torch.equal(static[k], v), (i, k)
