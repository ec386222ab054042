"""Workloads of the 4-bit block operators: a linear with 4-bit weights and group scales and the gradient through it, a
routed mixture of 4-bit experts for the tokens of a decode step, and the norms before and after a block with its gate and
residual, forward and backward.

listed() names the fixed cases, draw() gives further ones of the same ranges, prepare() makes their inputs on the GPU,
run() makes one pass (the library's entry points where `own` is set, elementary torch operations in 32 bits otherwise),
work() counts what a pass cannot do without and exact() gives its result from 64-bit arithmetic.

Sizes are those of the library's own workloads (hidden 5120, intermediate 17408; 512 experts of 160 on hidden 2560 with 10
per token; the tail shape 129 x 67 x 320) and generic ones between them.
"""
import torch

own = False

DEV = "cuda:0"
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
GROUP = 32                      # weights per scale
EPS = 1e-6


def listed():
    return [
        # one token through the gate projection: a decode step, bound by the weights' bytes
        dict(name="linear-token", op="linear", M=1, K=5120, N=17408, layout=3, x="f16"),
        # 13 rows through the down projection: a small decode batch, or a draft being verified
        dict(name="linear-batch", op="linear", M=13, K=17408, N=5120, layout=4, x="bf16"),
        # a prompt of 2049 tokens through the gate projection
        dict(name="linear-prompt", op="linear", M=2049, K=5120, N=17408, layout=3, x="bf16"),
        # gradient through a frozen 4-bit projection: the tail shape, float32 on both sides, ...
        dict(name="linear-grad-tail", op="linear_grad", M=129, N=67, K=320, layout=3, dy="f32", dx="f32"),
        # ... and a training batch through the gate projection
        dict(name="linear-grad", op="linear_grad", M=1024, N=17408, K=5120, layout=4, dy="bf16", dx="bf16"),
        # the experts of one token, router included: what a single request waits for in every layer
        dict(name="moe-token", op="moe", M=1, E=512, topk=10, H=2560, I=160, layout=3, x="f16", router="f32"),
        # the experts of a decode batch of 37 requests: most of the 512 experts, one or two tokens each
        dict(name="moe-batch", op="moe", M=37, E=512, topk=10, H=2560, I=160, layout=3, x="bf16", router="bf16"),
        # 130 tokens on 64 experts (a short prompt): a dozen tokens for each expert, float32 rows
        dict(name="moe-rows", op="moe", M=130, E=64, topk=6, H=1024, I=704, layout=4, x="f32", router="f32"),
        # one token between two blocks: norm of the block's result, gate, residual, norm before the next block
        dict(name="norm-token", op="norm", M=1, H=2560, h="bf16", y="bf16", x="bf16", w="bf16", G=1, g="bf16", offset=0.0),
        # a prompt between two blocks, float32 residual stream
        dict(name="norm-prompt", op="norm", M=8191, H=5120, h="f32", y="f32", x="bf16", w="f32", G=1, g="f32", offset=1.0),
        # gradients, three sequences with a gate row each, float32
        dict(name="norm-grad-tail", op="norm_grad", M=129, H=320, h="f32", y="f32", x="f32", w="f32", G=3, g="f32", offset=0.0),
        # gradients of a training batch: two sequences of 2048 rows
        dict(name="norm-grad", op="norm_grad", M=4096, H=5120, h="bf16", y="bf16", x="bf16", w="bf16", G=2, g="bf16", offset=0.0),
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["linear", "linear", "linear_grad", "moe", "moe", "norm", "norm_grad"])
    kind = lambda *of: rng.choice(of or ("f32", "bf16", "f16"))
    if op in ("linear", "linear_grad"):
        M, N, K = _log(rng, 1, 2049), _log(rng, 64, 17408), 32 * _log(rng, 4, 544)
        while M * N * K > 1024 * 17408 * 5120:
            M = max(1, M // 2)
        c = dict(op=op, M=M, N=N, K=K, layout=rng.choice([3, 4]))
        return dict(c, x=kind()) if op == "linear" else dict(c, dy=kind("f32", "bf16"), dx=kind("f32", "bf16"))
    if op == "moe":
        E = _log(rng, 4, 512)
        M, topk, H, I = _log(rng, 1, 130), rng.randint(1, min(10, E)), 32 * _log(rng, 4, 80), 32 * _log(rng, 2, 22)
        while M > 1 and M * topk * H * I > 130 * 6 * 1024 * 704:
            M = max(1, M // 2)
        return dict(op=op, M=M, E=E, topk=topk, H=H, I=I, layout=rng.choice([3, 4]), x=kind(), router=kind())
    G, each, H = rng.choice([1, 1, rng.randint(2, 16)]), _log(rng, 1, 4096), 8 * _log(rng, 8, 1000)
    if rng.random() < 0.2:      # a gate of its own for every row
        G, each = each, 1
    while G * each * H > 4096 * 5120:
        each, G = max(1, each // 2), G if each > 1 else max(1, G // 2)
    return dict(op=op, M=G * each, H=H, h=kind(), y=kind(), x=kind(), w=kind(), G=G, g=kind(), offset=rng.choice([0.0, 1.0]))


# ---- inputs ---------------------------------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _randn(g, shape, dtype=torch.float32, std=1.0):
    return (torch.randn(shape, generator=g, device=DEV, dtype=torch.float32) * std).to(dtype)


def _bank(g, E, N, K, layout):
    """E experts of an [N, K] weight as the library's bank: rounded to 4 bits per group of 32 between the group's least and
    largest value.  Per expert, every plane padded to 16 bytes: codes [N][K/2] (low nibble first), float16 scales
    [N][K/32], then the zeros as bytes (layout 3) or float16(-zero * scale) (layout 4)."""
    out, step = [], max(1, (1 << 27) // (N * K))
    pad = lambda t: torch.nn.functional.pad(t, (0, -t.shape[1] % 16))
    for e0 in range(0, E, step):
        n = min(step, E - e0)
        w = _randn(g, (n, N * K // GROUP, GROUP), std=0.02)
        lo, hi = w.amin(dim=2), w.amax(dim=2)
        s = ((hi - lo) / 15).half()
        s = torch.where(s > 0, s, torch.full_like(s, 1e-3))
        z = (-lo / s.float()).round().clamp(0, 15)
        q = ((w / s.float()[..., None]).round() + z[..., None]).clamp(0, 15).to(torch.uint8).view(n, N * K // 2, 2)
        last = z.to(torch.uint8) if layout == 3 else (-(z * s.float())).half().view(torch.uint8).view(n, -1)
        out.append(torch.cat([pad(q[..., 0] | (q[..., 1] << 4)), pad(s.view(torch.uint8).view(n, -1)), pad(last)], dim=1))
    return torch.cat(out).view(-1)


def prepare(case, seed):
    g, c = _gen(seed), case
    if c["op"] == "linear":
        return dict(c, x=_randn(g, (c["M"], c["K"]), DT[c["x"]]), bank=_bank(g, 1, c["N"], c["K"], c["layout"]))
    if c["op"] == "linear_grad":   # a loss gradient: small values, the rows of masked tokens all zero
        live = (torch.rand((c["M"], 1), generator=g, device=DEV) > 0.05).float()
        return dict(c, dy=(_randn(g, (c["M"], c["N"]), std=1e-3) * live).to(DT[c["dy"]]), dx=DT[c["dx"]],
                    bank=_bank(g, 1, c["N"], c["K"], c["layout"]))
    if c["op"] == "moe":
        M, E, H, I = c["M"], c["E"], c["H"], c["I"]
        return dict(c, x=_randn(g, (M, H), DT[c["x"]]), router=_randn(g, (E, H), DT[c["router"]], H ** -0.5),
                    w13=_bank(g, E, 2 * I, H, c["layout"]), w2=_bank(g, E, H, I, c["layout"]))
    M, H = c["M"], c["H"]
    s = dict(c, h=_randn(g, (M, H), DT[c["h"]], 3.0), y=_randn(g, (M, H), DT[c["y"]], 0.3), alpha=0.7, x=DT[c["x"]],
             post=_randn(g, (H,), DT[c["w"]], 0.2), pre=_randn(g, (H,), DT[c["w"]], 0.2), gate=_randn(g, (c["G"], H), DT[c["g"]]))
    if c["offset"] == 0.0:
        s["post"], s["pre"] = s["post"] + 1, s["pre"] + 1
    if c["op"] == "norm_grad":   # h: the stream after the block, as the forward pass left it
        s["dh"], s["dx"] = _randn(g, (M, H), DT[c["h"]], 1e-3), _randn(g, (M, H), DT[c["x"]], 1e-3)
    return s


# ---- one pass -------------------------------------------------------------------------------------------------
def run(state):
    return _own(state) if own else _plain(state)


def _own(s):
    import weight_quantized_mlp_amd as wq
    if s["op"] == "linear":
        return wq.awq_linear_run(s["x"], s["bank"], s["N"], s["layout"])
    if s["op"] == "linear_grad":
        return wq.awq_linear_backward(s["dy"], s["bank"], s["K"], s["layout"], dtype=s["dx"])
    if s["op"] == "moe":
        out, ids, weights = wq.moe_awq_run(s["x"], s["w13"], s["w2"], s["E"], s["I"], s["topk"], router=s["router"],
                                           meta_layout=s["layout"])
        return dict(out=out, ids=ids, weights=weights)
    if s["op"] == "norm":
        h, x = wq.block_norm_run(s["h"], s["y"], post=s["post"], gate=s["gate"], alpha=s["alpha"], pre=s["pre"], eps=EPS,
                                 offset=s["offset"], x_dtype=s["x"])
        return dict(h=h, x=x)
    dh, dy, dpost, dgate, dpre = wq.block_norm_backward(s["h"], s["y"], s["dh"], s["dx"], post=s["post"], gate=s["gate"],
                                                        alpha=s["alpha"], pre=s["pre"], eps=EPS, offset=s["offset"])
    return dict(dh=dh, dy=dy, dpost=dpost, dgate=dgate, dpre=dpre)


def _plain(s):
    if s["op"] == "linear":
        return s["x"].float() @ _dequant(s["bank"], 1, s["N"], s["K"], s["layout"])[0].T
    if s["op"] == "linear_grad":
        return (s["dy"].float() @ _dequant(s["bank"], 1, s["N"], s["K"], s["layout"])[0]).to(s["dx"])
    if s["op"] == "moe":
        return _plain_moe(s)
    if s["op"] == "norm":
        v = s["y"].float()
        v = v * torch.rsqrt((v * v).mean(dim=1, keepdim=True) + EPS) * (s["post"].float() + s["offset"])
        gate = s["gate"].float().repeat_interleave(s["M"] // s["G"], dim=0)
        h = (s["h"].float() + s["alpha"] * gate * v).to(s["h"].dtype)
        u = h.float()
        x = u * torch.rsqrt((u * u).mean(dim=1, keepdim=True) + EPS) * (s["pre"].float() + s["offset"])
        return dict(h=h, x=x.to(s["x"]))
    return _plain_norm_grad(s)


def _dequant(bank, E, N, K, layout, experts=None):
    """float32 weights [E, N, K] (or of the named experts): float16(q * scale + float16(-zero * scale)), one rounding."""
    up = lambda n: (n + 15) // 16 * 16
    at1 = up(N * K // 2)
    at2 = at1 + up(N * K // GROUP * 2)
    planes = bank.view(E, -1)
    if experts is not None:
        planes = planes[experts]
    n = planes.shape[0]
    groups = N * K // GROUP
    q = planes[:, : N * K // 2]
    q = torch.stack([q & 15, q >> 4], dim=2).view(n, groups, GROUP).float()
    s = planes[:, at1 : at1 + 2 * groups].contiguous().view(torch.float16).float()
    if layout == 3:
        b = (-(planes[:, at2 : at2 + groups].float() * s)).half().float()
    else:
        b = planes[:, at2 : at2 + 2 * groups].contiguous().view(torch.float16).float()
    return (q.mul_(s[..., None]).add_(b[..., None])).half().float().view(n, N, K)


def _plain_moe(s):
    M, E, topk, H, I = s["M"], s["E"], s["topk"], s["H"], s["I"]
    # which experts: the logits in 64 bits, so that two of them next to each other keep their order, rounded to 32
    logits = (s["x"].double() @ s["router"].double().T).float()
    order = torch.sort(logits, dim=1, descending=True, stable=True)
    ids, top = order.indices[:, :topk], order.values[:, :topk]
    p = torch.exp(top - top[:, :1])
    weights = p / p.sum(dim=1, keepdim=True)
    x = s["x"].float().repeat_interleave(topk, dim=0)
    used = ids.reshape(-1)
    gu = torch.bmm(_dequant(s["w13"], E, 2 * I, H, s["layout"], used), x[:, :, None])[:, :, 0]
    act = gu[:, :I] / (1 + torch.exp(-gu[:, :I])) * gu[:, I:]
    y = torch.bmm(_dequant(s["w2"], E, H, I, s["layout"], used), act[:, :, None])[:, :, 0]
    out = (y.view(M, topk, H) * weights[:, :, None]).sum(dim=1)
    return dict(out=out.to(s["x"].dtype), ids=ids.to(torch.int32), weights=weights)


def _plain_norm_grad(s):
    M, H, G = s["M"], s["H"], s["G"]
    u, v, dx = s["h"].float(), s["y"].float(), s["dx"].float()
    ru = torch.rsqrt((u * u).mean(dim=1, keepdim=True) + EPS)
    rv = torch.rsqrt((v * v).mean(dim=1, keepdim=True) + EPS)
    n, p = u * ru, v * rv
    dn = dx * (s["pre"].float() + s["offset"])
    du = s["dh"].float() + ru * (dn - n * (dn * n).mean(dim=1, keepdim=True))
    w, gate = s["post"].float() + s["offset"], s["gate"].float().repeat_interleave(M // G, dim=0)
    da = s["alpha"] * du
    db = da * gate
    dp = db * w
    dy = rv * (dp - p * (dp * p).mean(dim=1, keepdim=True))
    return dict(dh=du.to(s["h"].dtype), dy=dy.to(s["y"].dtype), dpost=(db * p).sum(dim=0),
                dgate=(da * p * w).view(G, M // G, H).sum(dim=1), dpre=(dx * n).sum(dim=0))


# ---- counts and exact results -----------------------------------------------------------------------------------
def _weight_bytes(N, K, layout):
    return N * K // 2 + N * K // GROUP * layout


def work(case):
    c = case
    if c["op"] in ("linear", "linear_grad"):
        M, N, K = c["M"], c["N"], c["K"]
        rows = M * K * SIZE[c["x"]] + 4 * M * N if c["op"] == "linear" else M * N * SIZE[c["dy"]] + M * K * SIZE[c["dx"]]
        return dict(bytes=rows + _weight_bytes(N, K, c["layout"]), flops=2 * M * N * K)
    if c["op"] == "moe":
        M, E, topk, H, I = c["M"], c["E"], c["topk"], c["H"], c["I"]
        used = E * (1 - (1 - topk / E) ** M)       # experts that M tokens reach on average
        per = _weight_bytes(2 * I, H, c["layout"]) + _weight_bytes(H, I, c["layout"])
        return dict(bytes=int(used * per) + E * H * SIZE[c["router"]] + 2 * M * H * SIZE[c["x"]] + 8 * M * topk,
                    flops=2 * M * (E * H + 3 * topk * H * I))
    M, H = c["M"], c["H"]
    small = (2 * SIZE[c["w"]] + c["G"] * SIZE[c["g"]]) * H
    if c["op"] == "norm":
        return dict(bytes=M * H * (2 * SIZE[c["h"]] + SIZE[c["y"]] + SIZE[c["x"]]) + small, flops=12 * M * H)
    return dict(bytes=M * H * (3 * SIZE[c["h"]] + 2 * SIZE[c["y"]] + SIZE[c["x"]]) + small + 4 * (2 + c["G"]) * H, flops=30 * M * H)


def _exact_weight(bank, at, N, K, layout):
    """float64 [N, K] of the expert whose bytes start at `at`, value by value from the definition."""
    D = torch.float64
    nk, ng = N * K, N * (K // GROUP)
    r16 = lambda n: -(-n // 16) * 16
    code = bank[at : at + nk // 2].to(torch.int16)
    q = torch.empty((nk,), dtype=D, device=bank.device)
    q[0::2], q[1::2] = (code % 16).to(D), (code // 16).to(D)
    at += r16(nk // 2)
    scale = bank[at : at + 2 * ng].clone().view(torch.float16).to(D)
    at += r16(2 * ng)
    if layout == 3:
        bias = (-bank[at : at + ng].to(D) * scale).to(torch.float16).to(D)
    else:
        bias = bank[at : at + 2 * ng].clone().view(torch.float16).to(D)
    return (q.view(ng, GROUP) * scale[:, None] + bias[:, None]).to(torch.float16).to(D).view(N, K)


def exact(case, seed):
    s, D = prepare(case, seed), torch.float64
    if s["op"] == "linear":
        w = _exact_weight(s["bank"], 0, s["N"], s["K"], s["layout"])
        return s["x"].to(D) @ w.t().contiguous()
    if s["op"] == "linear_grad":
        return s["dy"].to(D) @ _exact_weight(s["bank"], 0, s["N"], s["K"], s["layout"])
    if s["op"] == "moe":
        M, E, topk, H, I = s["M"], s["E"], s["topk"], s["H"], s["I"]
        x = s["x"].to(D)
        logits = x @ s["router"].to(D).t().contiguous()
        top, ids = torch.topk(logits, topk, dim=1)
        weights = torch.softmax(top, dim=1)
        out = torch.zeros((M, H), dtype=D, device=x.device)
        b13, b2 = s["w13"].numel() // E, s["w2"].numel() // E
        for e in sorted(set(ids.flatten().tolist())):
            rows, k = torch.nonzero(ids == e, as_tuple=True)
            gu = x[rows] @ _exact_weight(s["w13"], e * b13, 2 * I, H, s["layout"]).t().contiguous()
            act = gu[:, :I] * torch.sigmoid(gu[:, :I]) * gu[:, I:]
            y = act @ _exact_weight(s["w2"], e * b2, H, I, s["layout"]).t().contiguous()
            out[rows] += weights[rows, k][:, None] * y
        return dict(out=out, ids=None, weights=weights)
    h, y = s["h"].to(D), s["y"].to(D)
    post, pre = s["post"].to(D) + s["offset"], s["pre"].to(D) + s["offset"]
    M, H, G = s["M"], s["H"], s["G"]
    gate = s["gate"].to(D)[torch.arange(M, device=h.device) // (M // G)]
    norm = lambda t: t / torch.sqrt(t.pow(2).sum(dim=1, keepdim=True) / H + EPS)
    if s["op"] == "norm":
        h = h + s["alpha"] * gate * norm(y) * post
        return dict(h=h, x=norm(h.to(s["h"].dtype).to(D)) * pre)
    dx, dh = s["dx"].to(D), s["dh"].to(D)

    def through(t, dn):   # gradient of norm(t) times dn
        r = 1 / torch.sqrt(t.pow(2).sum(dim=1, keepdim=True) / H + EPS)
        return r * dn - r.pow(3) / H * t * (t * dn).sum(dim=1, keepdim=True)

    du = dh + through(h, dx * pre)
    p = norm(y)
    return dict(dh=du, dy=through(y, s["alpha"] * du * gate * post), dpost=(s["alpha"] * du * gate * p).sum(dim=0),
                dgate=(s["alpha"] * du * p * post).view(G, M // G, H).sum(dim=1), dpre=(dx * norm(h)).sum(dim=0))
