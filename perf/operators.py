"""Workloads of the adapter and training operators: low-rank adapters beside a shared quantised projection
(forward and backward), the input gradient of a frozen quantised projection, and the AdamW step.

listed() names the fixed cases, draw() gives further ones of the same ranges, prepare() makes their inputs on the
GPU, run() makes one pass (the library's entry points where `own` is set, elementary torch operations in 32 bits
otherwise), work() counts what a pass cannot do without and exact() gives its result from 64-bit arithmetic.

Sizes are those of the library's own workloads (hidden 5120, intermediate 17408; the tiny MLP's 256 and 512; the
tail shape 129 x 67 x 320) and generic ones between them.
"""
import torch

own = False

DEV = "cuda:0"
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
BLOCK = 256                     # elements per scale of the 8-bit optimizer states
BETA1, BETA2, EPS, DECAY = 0.9, 0.999, 1e-8, 0.01


def listed():
    return [
        # one token of one request on the tiny projection: two launches' latency
        dict(name="adapters-token", op="lora", M=1, K=256, N=512, E=1, R=8, x="f32", w="bf16", requests=1),
        # a decode step of 61 requests, 32 adapters loaded, some requests without one
        dict(name="adapters-decode", op="lora", M=61, K=5120, N=17408, E=32, R=16, x="bf16", w="bf16", requests=61),
        # a prefill batch of 11 requests of ragged lengths on 8 adapters
        dict(name="adapters-prefill", op="lora", M=4099, K=5120, N=17408, E=8, R=64, x="bf16", w="bf16", requests=11),
        # the tail shape: nothing a multiple of a tile, float32 master adapters
        dict(name="adapters-grad-tail", op="lora_backward", M=129, K=320, N=67, E=2, R=8, x="f32", dy="f32", dx="f32",
             w="f32", requests=3),
        # fine-tuning one adapter on the gate projection
        dict(name="adapters-grad-one", op="lora_backward", M=4096, K=5120, N=17408, E=1, R=16, x="bf16", dy="f32",
             dx="bf16", w="bf16", requests=1),
        # six adapters trained at once on the down projection, a ragged batch
        dict(name="adapters-grad-many", op="lora_backward", M=2047, K=17408, N=5120, E=6, R=32, x="bf16", dy="bf16",
             dx="bf16", w="bf16", requests=9),
        # gradient through a frozen projection: the tail shape, ...
        dict(name="linear-grad-tail", op="qlinear_backward", fmt="fp8", M=129, N=67, K=320, dy="f32", dx="f32"),
        # ... a short FP8 batch through the gate projection, ...
        dict(name="linear-grad-fp8", op="qlinear_backward", fmt="fp8", M=512, N=17408, K=5120, dy="bf16", dx="bf16"),
        # ... and a long NVFP4 batch through the down projection
        dict(name="linear-grad-nvfp4", op="qlinear_backward", fmt="nvfp4", M=4096, N=5120, K=17408, dy="f32", dx="bf16"),
        # the optimizer on one layer's adapters (gate, up, down at rank 16), float32 states
        dict(name="adamw-adapters", op="adamw", bits=32, sizes="81920,278528,81920,278528,278528,81920", g="f32", copy="bf16"),
        # the adapters of many layers at once, 8-bit states, sizes that end inside a block
        dict(name="adamw-many-8bit", op="adamw", bits=8, sizes=",".join(["1310720", "4456448", "517", "1114113"] * 12), g="f32",
             copy="bf16"),
        # whole projections in float32 states
        dict(name="adamw-dense", op="adamw", bits=32, sizes="89128960,89128960,17408", g="bf16", copy="none"),
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["lora", "lora", "lora_backward", "lora_backward", "qlinear_backward", "qlinear_backward", "adamw"])
    if op == "adamw":
        count, top = _log(rng, 1, 60), _log(rng, 2000, 4000000)
        sizes = [str(max(1, _log(rng, max(1, top // 100), top))) for _ in range(count)]
        return dict(op=op, bits=rng.choice([8, 32]), sizes=",".join(sizes), g=rng.choice(["f32", "bf16"]),
                    copy=rng.choice(["none", "bf16", "f16"]))
    if op == "qlinear_backward":
        fmt = rng.choice(["fp8", "nvfp4"])
        step = 16 if fmt == "fp8" else 64
        M, N, K = _log(rng, 1, 4096), _log(rng, 64, 17408), step * _log(rng, max(1, 128 // step), 17408 // step)
        while M * N * K > 4096 * 5120 * 17408:
            M = max(1, M // 2)
        return dict(op=op, fmt=fmt, M=M, N=N, K=K, dy=rng.choice(["f32", "bf16"]), dx=rng.choice(["f32", "bf16"]))
    M, K, N = _log(rng, 1, 4096), 16 * _log(rng, 8, 1088), _log(rng, 64, 17408)
    E, R = _log(rng, 1, 32), 8 * _log(rng, 1, 16)
    while M * (K + N) * R > 4096 * 22528 * 64:
        R = max(8, R // 16 * 8)
        M = max(1, M * 3 // 4)
    c = dict(op=op, M=M, K=K, N=N, E=E, R=R, x=rng.choice(["f32", "bf16", "f16"]), w=rng.choice(["f32", "bf16", "f16"]),
             requests=rng.randint(1, max(1, min(M, 64))))
    if op == "lora_backward":
        c["dy"], c["dx"] = rng.choice(["f32", "bf16"]), rng.choice(["f32", "bf16"])
    return c


# ---- inputs ---------------------------------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _randn(g, shape, dtype=torch.float32, std=1.0):
    return (torch.randn(shape, generator=g, device=DEV, dtype=torch.float32) * std).to(dtype)


def _ids(g, M, E, requests):
    """Adapter of each row: `requests` runs of consecutive rows, each on a random adapter or (1 in 16) on none."""
    which = torch.randint(0, E, (requests,), generator=g, device=DEV)
    none = torch.rand((requests,), generator=g, device=DEV) < 1 / 16
    which[none] = -1
    if requests == 1:
        which[0] = 0
    ends = torch.randperm(M - 1, generator=g, device=DEV)[: requests - 1].sort().values + 1 if requests > 1 else torch.zeros(0, dtype=torch.int64, device=DEV)
    return which[torch.searchsorted(ends, torch.arange(M, device=DEV), right=True)].to(torch.int32)


def _fp8_weight(g, N, K):
    w = _randn(g, (N, K), std=0.02)
    s = w.abs().amax(dim=1) / 448.0
    return (w / s[:, None]).to(torch.float8_e4m3fn).view(torch.uint8), s


E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _nvfp4_weight(g, N, K):
    """36-byte records {4 E4M3 group scales, 32 bytes of E2M1 pairs, low nibble first} and the global scale."""
    w = _randn(g, (N, K // 16, 16), std=0.02)
    gs = 448.0 * 6.0 / 0.12
    d = (w.abs().amax(dim=2) / 6.0 * gs).clamp(2.0 ** -9, 448.0).to(torch.float8_e4m3fn)
    u = w * (gs / d.float())[:, :, None]
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=DEV)
    q = torch.bucketize(u.abs(), edges).to(torch.uint8) | ((u < 0).to(torch.uint8) << 3)
    q = q.view(N, K // 64, 32, 2)
    return torch.cat([d.view(torch.uint8).view(N, K // 64, 4), q[..., 0] | (q[..., 1] << 4)], dim=2).contiguous(), gs


def _grad_rows(g, M, N, dtype):
    """A loss gradient: small values, the rows of masked tokens all zero."""
    live = (torch.rand((M, 1), generator=g, device=DEV) > 0.05).float()
    return (_randn(g, (M, N), std=1e-3) * live).to(dtype)


def prepare(case, seed):
    g, c = _gen(seed), case
    if c["op"] in ("lora", "lora_backward"):
        M, K, N, E, R = c["M"], c["K"], c["N"], c["E"], c["R"]
        s = dict(op=c["op"], x=_randn(g, (M, K), DT[c["x"]]), a=_randn(g, (E, R, K), DT[c["w"]], K ** -0.5),
                 b=_randn(g, (E, N, R), DT[c["w"]], 0.05), scale=torch.rand((E,), generator=g, device=DEV) * 2 + 0.5,
                 ids=_ids(g, M, E, c["requests"]))
        if c["op"] == "lora":
            s["y"] = _randn(g, (M, N), std=1.5)
        else:
            s["dy"], s["dx"] = _grad_rows(g, M, N, DT[c["dy"]]), _randn(g, (M, K), DT[c["dx"]], 1e-3)
        return s
    if c["op"] == "qlinear_backward":
        s = dict(op=c["op"], fmt=c["fmt"], dy=_grad_rows(g, c["M"], c["N"], DT[c["dy"]]), dx=DT[c["dx"]])
        if c["fmt"] == "fp8":
            s["w"], s["scale"] = _fp8_weight(g, c["N"], c["K"])
            s["gs"] = 1.0
        else:
            (s["w"], s["gs"]), s["scale"] = _nvfp4_weight(g, c["N"], c["K"]), None
        return s
    sizes = [int(n) for n in c["sizes"].split(",")]
    s = dict(op="adamw", bits=c["bits"], seed=17, t=7, p=[], g=[], m=[], v=[], ms=[], vs=[], copy=[],
             step=torch.tensor([7], dtype=torch.int64, device=DEV), lr=torch.tensor([1e-3], device=DEV))
    for n in sizes:
        s["p"].append(_randn(g, (n,), std=0.02))
        s["g"].append(_randn(g, (n,), DT[c["g"]], 1e-3))
        m, v = _randn(g, (n,), std=3e-4), _randn(g, (n,), std=1e-3).square()
        if c["bits"] == 8:   # states as an earlier step left them: codes and one power-of-two scale per block
            for x, dtype, most, codes, scales in ((m, torch.float8_e4m3fn, 448.0, "m", "ms"), (v, torch.float8_e5m2, 57344.0, "v", "vs")):
                xb = torch.nn.functional.pad(x, (0, -n % BLOCK)).view(-1, BLOCK)
                sc = torch.exp2(torch.ceil(torch.log2(xb.abs().amax(dim=1) / most)))
                s[codes].append((xb / sc[:, None]).to(dtype).view(-1)[:n].clone())
                s[scales].append(sc)
        else:
            s["m"].append(m)
            s["v"].append(v)
        if c["copy"] != "none":
            s["copy"].append(s["p"][-1].to(DT[c["copy"]]))
    if own:
        import weight_quantized_mlp_amd as wq
        s["table"] = wq.adamw_table(s["p"], s["g"], s["m"], s["v"], s["copy"] or None, s["ms"] or None, s["vs"] or None)
    return s


# ---- one pass -------------------------------------------------------------------------------------------------
def run(state):
    return _own(state) if own else _plain(state)


def _own(s):
    import weight_quantized_mlp_amd as wq
    if s["op"] == "lora":
        return wq.lora_run(s["x"], s["a"], s["b"], s["scale"], s["ids"], s["y"])
    if s["op"] == "lora_backward":
        dx, da, db = wq.lora_backward(s["dy"], s["x"], s["a"], s["b"], s["scale"], s["ids"], s["dx"])
        return dict(dx=dx, da=da, db=db)
    if s["op"] == "qlinear_backward":
        fmt = wq.WQ_FMT_FP8W if s["fmt"] == "fp8" else wq.WQ_FMT_NVFP4
        return wq.qlinear_backward(fmt, s["dy"], s["w"], s["scale"], s["gs"], dtype=s["dx"])
    wq.adamw_run(s["table"], s["step"], s["lr"], BETA1, BETA2, EPS, DECAY, seed=s["seed"])
    return _adamw_outputs(s)


def _adamw_outputs(s):
    # one tensor of each size: at most 64 outputs, and every kind of tensor among them
    at = sorted({t.numel(): i for i, t in reversed(list(enumerate(s["p"])))}.values())[:9]
    pick = lambda ts: [ts[i] for i in at] if ts else []
    return dict(p=pick(s["p"]), m=pick(s["m"]), v=pick(s["v"]), ms=pick(s["ms"]), vs=pick(s["vs"]), copy=pick(s["copy"]))


def _plain(s):
    if s["op"] == "lora":
        T, A, B = _adapter_terms(s)
        return s["y"] + T @ B
    if s["op"] == "lora_backward":
        T, A, B = _adapter_terms(s)
        x, dy = s["x"].float(), s["dy"].float()
        E, R, N = s["a"].shape[0], s["a"].shape[1], s["b"].shape[1]
        dT = (dy @ B.T) * _mask(s, R)
        dx = (s["dx"].float() + dT @ A).to(s["dx"].dtype)
        db = (T.T @ dy).view(E, R, N).transpose(1, 2).contiguous()
        return dict(dx=dx, da=(dT.T @ x).view(E, R, -1), db=db)
    if s["op"] == "qlinear_backward":
        return (s["dy"].float() @ _dequant(s)).to(s["dx"])
    [_adamw_plain(s, i, s["t"]) for i in range(len(s["p"]))]
    return _adamw_outputs(s)


def _mask(s, R):
    """[M, E*R]: the scale of the row's adapter in that adapter's R columns, 0 elsewhere."""
    E = s["scale"].shape[0]
    hot = (s["ids"][:, None] == torch.arange(E, device=DEV, dtype=torch.int32)[None, :]).float() * s["scale"][None, :]
    return hot.repeat_interleave(R, dim=1)


def _adapter_terms(s):
    """All adapters side by side: T [M, E*R] masked and scaled, A [E*R, K], B [E*R, N]."""
    E, R, K = s["a"].shape
    A = s["a"].float().view(E * R, K)
    B = s["b"].float().transpose(1, 2).reshape(E * R, -1)
    return (s["x"].float() @ A.T) * _mask(s, R), A, B


def _dequant(s):
    if s["fmt"] == "fp8":
        return s["w"].view(torch.float8_e4m3fn).float() * s["scale"][:, None]
    N, nb, _ = s["w"].shape
    d = s["w"][:, :, :4].contiguous().view(torch.float8_e4m3fn).float()
    qs = s["w"][:, :, 4:]
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=DEV)
    q = table[torch.stack([qs & 15, qs >> 4], dim=3).view(N, nb, 4, 16).int()]
    return ((q * d[..., None]) * (1.0 / s["gs"])).view(N, nb * 64)


MASK32 = 0xFFFFFFFF


def _mix(h):
    """32-bit integer mix (int64 tensors or ints holding 32-bit values): two rounds of multiply and xor-shift."""
    h = h ^ (h >> 16)
    h = (h * 0x7FEB352D) & MASK32
    h = h ^ (h >> 15)
    h = (h * 0x846CA68B) & MASK32
    return h ^ (h >> 16)


def _key(seed, step, tensor):
    return _mix((_mix((seed + 0x9E3779B9 * (int(step) & MASK32)) & MASK32) + tensor) & MASK32)


def _block_scale(x, half):
    """Power-of-two scale of each block: the smallest 2^e with max |x| <= 0.875 * 2^half * 2^e."""
    f, p = torch.frexp(x.abs().amax(dim=1))
    e = (p - half + (f > 0.875).to(p.dtype)).clamp(-100, 100)
    return torch.where(f > 0, torch.ldexp(torch.ones_like(f), e), torch.ones_like(f))


def _round8(x, rnd, mant, emin):
    """x rounded to `mant` mantissa bits (exponent at least emin) by adding 16 random bits below the kept ones."""
    drop = 23 - mant
    mag = x.abs()
    up = ((mag.view(torch.int32) + (rnd << (drop - 16))) >> drop) << drop
    sub = (((mag.clamp(max=2.0 ** emin) * 2.0 ** (mant - emin + 16)).to(torch.int32) + rnd) >> 16).float() * 2.0 ** (emin - mant)
    return torch.copysign(torch.where(mag < 2.0 ** emin, sub, up.view(torch.float32)), x)


def _adamw_plain(s, i, t):
    p, g, n = s["p"][i], s["g"][i].float(), s["p"][i].numel()
    if s["bits"] == 8:
        pad = lambda x: torch.nn.functional.pad(x, (0, -n % BLOCK)).view(-1, BLOCK)
        m = (pad(s["m"][i].float()) * s["ms"][i][:, None]).view(-1)[:n]
        v = (pad(s["v"][i].float()) * s["vs"][i][:, None]).view(-1)[:n]
    else:
        m, v = s["m"][i], s["v"][i]
    m = m * BETA1 + g * (1 - BETA1)
    v = v * BETA2 + (g * g) * (1 - BETA2)
    lr = s["lr"]
    step = (m / (1 - BETA1 ** t)) / (torch.sqrt(v / (1 - BETA2 ** t)) + EPS)
    p.copy_(p * (1 - lr * DECAY) - lr * step)
    if s["copy"]:
        s["copy"][i].copy_(p)
    if s["bits"] != 8:
        s["m"][i].copy_(m)
        s["v"][i].copy_(v)
        return
    at = torch.arange(n, device=DEV, dtype=torch.int64)
    h = _mix((_key(s["seed"], t, i) + at * 0x9E3779B9) & MASK32)
    for x, rnd, half, mant, emin, codes, scales in ((m, h & 0xFFFF, 9, 3, -6, s["m"][i], s["ms"][i]),
                                                    (v, h >> 16, 16, 2, -14, s["v"][i], s["vs"][i])):
        xb = pad(x)
        sc = _block_scale(xb, half)
        q = _round8((xb / sc[:, None]).view(-1)[:n], rnd.int(), mant, emin)
        codes.copy_(q.to(codes.dtype))
        scales.copy_(sc)


# ---- counts and exact results -----------------------------------------------------------------------------------
def work(case):
    c = case
    if c["op"] in ("lora", "lora_backward"):
        M, K, N, R = c["M"], c["K"], c["N"], c["R"]
        used = min(c["E"], c["requests"])
        w = used * R * (K + N)
        if c["op"] == "lora":
            return dict(bytes=M * K * SIZE[c["x"]] + w * SIZE[c["w"]] + 8 * M * N + 4 * M, flops=2 * M * R * (K + N))
        return dict(bytes=M * K * (SIZE[c["x"]] + 2 * SIZE[c["dx"]]) + M * N * SIZE[c["dy"]] + w * SIZE[c["w"]]
                    + c["E"] * R * (K + N) * 4 + 4 * M, flops=2 * M * R * (3 * K + 2 * N))
    if c["op"] == "qlinear_backward":
        M, N, K = c["M"], c["N"], c["K"]
        wb = N * K + 4 * N if c["fmt"] == "fp8" else N * (K // 64) * 36
        return dict(bytes=M * N * SIZE[c["dy"]] + wb + M * K * SIZE[c["dx"]], flops=2 * M * N * K)
    n = sum(int(v) for v in c["sizes"].split(","))
    each = 8 + SIZE[c["g"]] + (4 if c["bits"] == 8 else 16) + (0 if c["copy"] == "none" else 2)
    return dict(bytes=n * each + (n // BLOCK * 16 if c["bits"] == 8 else 0), flops=16 * n)


def exact(case, seed):
    global own
    was, own = own, False
    s = prepare(case, seed)
    own = was
    D = torch.float64
    if s["op"] in ("lora", "lora_backward"):
        x, a, b, sc = s["x"].to(D), s["a"].to(D), s["b"].to(D), s["scale"].to(D)
        rows = [torch.nonzero(s["ids"] == e).flatten() for e in range(a.shape[0])]
        if s["op"] == "lora":
            out = s["y"].to(D)
            for e, at in enumerate(rows):
                out[at] += sc[e] * ((x[at] @ a[e].T.contiguous()) @ b[e].T.contiguous())
            return out
        dy, dx, da, db = s["dy"].to(D), s["dx"].to(D), torch.zeros_like(a), torch.zeros_like(b)
        for e, at in enumerate(rows):
            t, dt = x[at] @ a[e].T.contiguous(), sc[e] * (dy[at] @ b[e])
            db[e], da[e] = sc[e] * (dy[at].T.contiguous() @ t), dt.T.contiguous() @ x[at]
            dx[at] += dt @ a[e]
        return dict(dx=dx, da=da, db=db)
    if s["op"] == "qlinear_backward":
        if s["fmt"] == "fp8":
            w = s["w"].view(torch.float8_e4m3fn).to(D) * s["scale"].to(D)[:, None]
        else:
            rec = s["w"]
            N, nb = rec.shape[:2]
            code = torch.empty((N, nb, 64), dtype=torch.uint8, device=DEV)
            code[..., 0::2], code[..., 1::2] = rec[..., 4:] & 15, rec[..., 4:] >> 4
            mag = (code & 7).to(D)
            mag = torch.where(mag < 5, mag / 2, torch.where(mag < 6, mag - 2, torch.where(mag < 7, mag - 2, mag - 1)))
            mag = torch.where(code >= 8, -mag, mag)
            d = rec[..., :4].contiguous().view(torch.float8_e4m3fn).to(D)
            w = (mag.view(N, nb, 4, 16) * d[..., None] / s["gs"]).view(N, nb * 64)
        return s["dy"].to(D) @ w
    t, out = s["t"], dict(p=[], m=[], v=[], ms=[], vs=[], copy=[])
    at = sorted({x.numel(): i for i, x in reversed(list(enumerate(s["p"])))}.values())[:9]
    lr = s["lr"].to(D)
    for i in at:
        p, g, m, v = s["p"][i].to(D), s["g"][i].to(D), s["m"][i].to(D), s["v"][i].to(D)
        if s["bits"] == 8:
            each = torch.arange(p.numel(), device=DEV) // BLOCK
            m, v = m * s["ms"][i].to(D)[each], v * s["vs"][i].to(D)[each]
        m, v = BETA1 * m + (1 - BETA1) * g, BETA2 * v + (1 - BETA2) * g ** 2
        p = p - lr * DECAY * p - lr * (m / (1 - BETA1 ** t)) / ((v / (1 - BETA2 ** t)).sqrt() + EPS)
        for key, value in (("p", p), ("m", m), ("v", v), ("copy", p)):
            out[key].append(None if s["bits"] == 8 and key in "mv" else value)
        for key in ("ms", "vs"):
            out[key].append(None)
    if s["bits"] != 8:
        out["ms"], out["vs"] = [], []
    if not s["copy"]:
        out["copy"] = []
    return out
