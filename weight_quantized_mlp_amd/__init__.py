"""Python binding of libwqmlp (the C ABI declared in include/wqmlp.h, include/wqmlp_adapters.h and include/wqmlp_blocks.h).

Argument marshalling only: torch tensors provide device memory and the
current HIP stream; every step of the computation runs in the library's
gfx950 kernels.  Functions carry the C entry points' names.  A missing or
unloadable library raises at first use; nothing falls back to another path.

Outputs and workspaces that the caller does not pass are allocated with
torch on the input's device (the library itself never allocates).
"""
import ctypes
import os

import torch

__all__ = [
    "WQError", "lib", "lib_path", "WQ_F32", "WQ_BF16", "WQ_F16", "WQ_FMT_FP8W", "WQ_FMT_NVFP4",
    "WQ_PATH_AUTO", "WQ_PATH_GEMV", "WQ_PATH_MFMA", "WQ_STAGE_GATEUP_ONLY", "WQ_STAGE_DOWN_ONLY", "WQ_ACT_E4M3",
    "wq_abi_version", "wq_strerror",
    "WQ_STATIC_SCRATCH_BYTES", "mlp_workspace_bytes", "mlp_fp8w_run", "mlp_fp8w_run_noalloc", "mlp_nvfp4_run", "awq_bank_bytes", "moe_awq_m1_run",
    "nvfp4_pack_block64", "awq_pack_bank", "fp8w_dequant_f32", "nvfp4_dequant_f32", "awq_dequant_f16",
    "qlinear_workspace_bytes", "qlinear_run", "wq_read_probe",
    "WQ_LORA_MAX_RANK", "WQ_ADAMW_BLOCK", "WQ_ADAMW_KEEP_V", "lora_workspace_bytes", "lora_run", "lora_backward",
    "qlinear_backward_workspace_bytes", "qlinear_backward", "adamw_table_bytes", "AdamWTable", "adamw_table", "adamw_run",
    "awq_linear_workspace_bytes", "awq_linear_run", "awq_linear_backward_workspace_bytes", "awq_linear_backward",
    "WQ_MOE_MAX_TOKENS", "WQ_MOE_RENORM", "moe_awq_workspace_bytes", "moe_awq_run",
    "block_norm_run", "block_norm_backward_workspace_bytes", "block_norm_backward",
]

WQ_F32, WQ_BF16, WQ_F16 = 0, 1, 2
WQ_FMT_FP8W, WQ_FMT_NVFP4 = 0, 1
WQ_PATH_AUTO, WQ_PATH_GEMV, WQ_PATH_MFMA = 0, 1, 2
WQ_STAGE_GATEUP_ONLY, WQ_STAGE_DOWN_ONLY = 4, 8
WQ_ACT_E4M3 = 16
WQ_STATIC_SCRATCH_BYTES = 32 << 20
WQ_LORA_MAX_RANK = 256
WQ_ADAMW_BLOCK = 256
WQ_ADAMW_KEEP_V = 256
WQ_MOE_MAX_TOKENS = 256
WQ_MOE_RENORM = 1
_PATHS = {"auto": WQ_PATH_AUTO, "gemv": WQ_PATH_GEMV, "mfma": WQ_PATH_MFMA}
_STAGES = {None: 0, "gateup": WQ_STAGE_GATEUP_ONLY, "down": WQ_STAGE_DOWN_ONLY}
_ACTS = {None: 0, "e4m3": WQ_ACT_E4M3}

# The in-tree library; WQMLP_LIBRARY names another build of it (the host-sanitizer build of the CPU tests).
lib_path = os.environ.get("WQMLP_LIBRARY") or os.path.join(os.path.dirname(os.path.abspath(__file__)), "libwqmlp.so")
_lib = None

_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_INT = ctypes.c_int
_F = ctypes.c_float
_SZ = ctypes.c_size_t
_D = ctypes.c_double
_SIGS = {
    "wq_abi_version": (_INT, []),
    "wq_strerror": (ctypes.c_char_p, [_INT]),
    "wq_last_hip_error": (_INT, []),
    "mlp_workspace_bytes": (_SZ, [_INT, _I64, _I64, _I64, _INT]),
    "mlp_fp8w_run": (_INT, [_I64, _I64, _I64, _P, _INT, _P, _P, _P, _P, _P, _P, _P, _SZ, _P, _INT, _P]),
    "mlp_fp8w_run_noalloc": (_INT, [_I64, _I64, _I64, _P, _INT, _P, _P, _P, _P, _P, _P, _P, _INT, _P]),
    "mlp_nvfp4_run": (_INT, [_I64, _I64, _I64, _P, _INT, _P, _F, _P, _F, _P, _F, _P, _SZ, _P, _INT, _P]),
    "awq_bank_bytes": (_SZ, [_I64, _I64, _I64, _INT]),
    "moe_awq_m1_run": (_INT, [_I64, _I64, _I64, _I64, _P, _P, _P, _P, _P, _INT, _P, _P, _P]),
    "nvfp4_pack_block64": (_INT, [_I64, _I64, _P, _P, _P, _P]),
    "awq_pack_bank": (_INT, [_I64, _I64, _I64, _P, _P, _P, _INT, _P, _P]),
    "fp8w_dequant_f32": (_INT, [_I64, _I64, _P, _P, _P, _P]),
    "nvfp4_dequant_f32": (_INT, [_I64, _I64, _P, _F, _P, _P]),
    "awq_dequant_f16": (_INT, [_I64, _I64, _I64, _P, _INT, _P, _P]),
    "qlinear_workspace_bytes": (_SZ, [_INT, _I64, _I64, _I64, _INT]),
    "qlinear_run": (_INT, [_INT, _I64, _I64, _I64, _P, _INT, _P, _P, _F, _P, _SZ, _P, _INT, _P]),
    "wq_read_probe": (_INT, [_P, _SZ, _P, _INT, _P]),
    "lora_workspace_bytes": (_SZ, [_I64, _I64, _I64, _I64, _I64, _INT]),
    "lora_run": (_INT, [_I64, _I64, _I64, _I64, _I64, _P, _INT, _P, _P, _INT, _P, _P, _P, _P, _SZ, _P, _P]),
    "lora_backward": (_INT, [_I64, _I64, _I64, _I64, _I64, _P, _INT, _P, _INT, _P, _P, _INT, _P, _P, _P, _INT, _P, _SZ,
                             _P, _P, _P, _P]),
    "qlinear_backward_workspace_bytes": (_SZ, [_INT, _I64, _I64, _I64, _INT]),
    "qlinear_backward": (_INT, [_INT, _I64, _I64, _I64, _P, _INT, _P, _P, _F, _P, _SZ, _P, _INT, _P]),
    "adamw_table_bytes": (_SZ, [_I64]),
    "adamw_table_build": (_INT, [_I64, _P, _INT, _P, _SZ, _P]),
    "adamw_run": (_INT, [_I64, _I64, _INT, _P, _P, _P, _D, _D, _D, _D, _F, ctypes.c_uint32, _P]),
    "awq_linear_workspace_bytes": (_SZ, [_I64, _I64, _I64, _INT]),
    "awq_linear_run": (_INT, [_I64, _I64, _I64, _P, _INT, _P, _INT, _P, _SZ, _P, _P]),
    "awq_linear_backward_workspace_bytes": (_SZ, [_I64, _I64, _I64, _INT, _INT]),
    "awq_linear_backward": (_INT, [_I64, _I64, _I64, _P, _INT, _P, _INT, _P, _SZ, _P, _INT, _P]),
    "moe_awq_workspace_bytes": (_SZ, [_I64, _I64, _I64, _I64, _I64]),
    "moe_awq_run": (_INT, [_I64, _I64, _I64, _I64, _I64, _P, _INT, _P, _INT, _P, _P, _P, _P, _INT, _P, _SZ, _P, _INT, _INT, _P]),
    "block_norm_run": (_INT, [_I64, _I64, _P, _INT, _P, _INT, _P, _P, _INT, _P, _I64, _INT, _F, _F, _F, _P, _P, _INT, _P]),
    "block_norm_backward_workspace_bytes": (_SZ, [_I64, _I64, _I64]),
    "block_norm_backward": (_INT, [_I64, _I64, _P, _INT, _P, _INT, _P, _P, _INT, _P, _P, _INT, _P, _I64, _INT, _F, _F, _F,
                                   _P, _SZ, _P, _P, _P, _P, _P, _P]),
}


class _AdamWTensor(ctypes.Structure):   # wq_adamw_tensor
    _fields_ = [("n", _I64), ("p", _P), ("g", _P), ("m", _P), ("v", _P), ("m_scale", _P), ("v_scale", _P), ("copy", _P),
                ("g_dtype", ctypes.c_int32), ("copy_dtype", ctypes.c_int32)]


class WQError(RuntimeError):
    def __init__(self, fn, rc):
        self.rc = rc
        msg = lib().wq_strerror(rc).decode()
        extra = ""
        if rc in (-4, -7):
            extra = f" (hipError {lib().wq_last_hip_error()})"
        super().__init__(f"{fn}: rc={rc}: {msg}{extra}")


def lib():
    """Load the in-tree libwqmlp.so once; raise if it is missing."""
    global _lib
    if _lib is None:
        if not os.path.exists(lib_path):
            raise RuntimeError(f"{lib_path} is not built: run __graft_entry__.build() first")
        so = ctypes.CDLL(lib_path)
        for name, (res, args) in _SIGS.items():
            f = getattr(so, name)
            f.restype = res
            f.argtypes = args
        _lib = so
    return _lib


def _check(fn, rc):
    if rc != 0:
        raise WQError(fn, rc)


def _ptr(t):
    return None if t is None else t.data_ptr()


# The current stream's handle; torch's own accessor of the raw handle spares 2 us of object making where it exists.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(dev):
    if _raw_stream is not None and dev.index is not None:
        return _raw_stream(dev.index)
    return torch.cuda.current_stream(dev).cuda_stream


def _need(t, name, dtype, dev=None, numel=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if not t.is_cuda or (dev is not None and t.device != dev):
        raise ValueError(f"{name} must live on {dev or 'a GPU'}")
    if numel is not None and t.numel() != numel:
        raise ValueError(f"{name} must have {numel} elements, has {t.numel()}")
    return t


def _xdtype(x, allow_f16=False):
    if x.dtype == torch.float32:
        return WQ_F32
    if x.dtype == torch.bfloat16:
        return WQ_BF16
    if allow_f16 and x.dtype == torch.float16:
        return WQ_F16
    raise TypeError("x must be float32 or bfloat16" + (" (or float16 for NVFP4)" if allow_f16 else ""))


def wq_abi_version():
    return lib().wq_abi_version()


def wq_strerror(rc):
    return lib().wq_strerror(rc).decode()


def mlp_workspace_bytes(fmt, M, H, I, path="auto", act=None):
    return lib().mlp_workspace_bytes(fmt, M, H, I, _PATHS[path] | _ACTS[act])


def _workspace(nbytes, dev, workspace):
    if workspace is None:
        return torch.empty(max(nbytes, 1), dtype=torch.uint8, device=dev)
    _need(workspace, "workspace", torch.uint8, dev)
    return workspace


def _stage_flags(stage, workspace):
    """Stage bits; a one-stage call must bring the workspace that carries act between the two stages."""
    if stage not in _STAGES:
        raise ValueError(f"stage must be one of {list(_STAGES)}")
    if stage is not None and workspace is None:
        raise ValueError("stage='gateup' or 'down' needs the caller's workspace: act is handed from the "
                         "gate/up stage to the down stage through it")
    return _STAGES[stage]


def mlp_fp8w_run(x, w_gate, s_gate, w_up, s_up, w_down, s_down, out=None, workspace=None, path="auto",
                 stage=None):
    """FP8 E4M3 per-channel SwiGLU MLP.  x [M,H] f32/bf16; w_gate/w_up [I,H] u8; w_down [H,I] u8; s_* f32."""
    sflags = _stage_flags(stage, workspace)
    dev = x.device
    M, H = x.shape
    I = w_gate.shape[0]
    _need(x, "x", x.dtype, dev)
    for n, t, k in (("w_gate", w_gate, I * H), ("w_up", w_up, I * H), ("w_down", w_down, H * I)):
        _need(t, n, torch.uint8, dev, k)
    for n, t, k in (("s_gate", s_gate, I), ("s_up", s_up, I), ("s_down", s_down, H)):
        _need(t, n, torch.float32, dev, k)
    if out is None:
        out = torch.empty((M, H), dtype=torch.float32, device=dev)
    _need(out, "out", torch.float32, dev, M * H)
    nb = mlp_workspace_bytes(WQ_FMT_FP8W, M, H, I, path)
    ws = _workspace(nb, dev, workspace)
    rc = lib().mlp_fp8w_run(M, H, I, _ptr(x), _xdtype(x), _ptr(w_gate), _ptr(s_gate), _ptr(w_up), _ptr(s_up),
                            _ptr(w_down), _ptr(s_down), _ptr(ws), ws.numel(), _ptr(out),
                            _PATHS[path] | sflags, _stream(dev))
    _check("mlp_fp8w_run", rc)
    return out


def mlp_fp8w_run_noalloc(x, w_gate, s_gate, w_up, s_up, w_down, s_down, out, path="auto"):
    """mlp_fp8w_run on the library's static scratch: no workspace, and the caller passes out (nothing is
    allocated, here or in the library).  Calls needing more than WQ_STATIC_SCRATCH_BYTES raise (WQ_ESCRATCH)."""
    dev = x.device
    M, H = x.shape
    I = w_gate.shape[0]
    _need(x, "x", x.dtype, dev)
    for n, t, k in (("w_gate", w_gate, I * H), ("w_up", w_up, I * H), ("w_down", w_down, H * I)):
        _need(t, n, torch.uint8, dev, k)
    for n, t, k in (("s_gate", s_gate, I), ("s_up", s_up, I), ("s_down", s_down, H)):
        _need(t, n, torch.float32, dev, k)
    _need(out, "out", torch.float32, dev, M * H)
    rc = lib().mlp_fp8w_run_noalloc(M, H, I, _ptr(x), _xdtype(x), _ptr(w_gate), _ptr(s_gate), _ptr(w_up),
                                    _ptr(s_up), _ptr(w_down), _ptr(s_down), _ptr(out), _PATHS[path], _stream(dev))
    _check("mlp_fp8w_run_noalloc", rc)
    return out


def mlp_nvfp4_run(x, gate_blk, gate_gs, up_blk, up_gs, down_blk, down_gs, out=None, workspace=None, path="auto",
                  stage=None, act=None):
    """NVFP4 Block64 SwiGLU MLP.  x [M,H]; gate/up_blk [I,H/64,36] u8; down_blk [H,I/64,36] u8; gs floats.
    act="e4m3": the W4A8 variant (activations quantized per row to E4M3; MFMA path)."""
    sflags = _stage_flags(stage, workspace)
    dev = x.device
    M, H = x.shape
    I = gate_blk.shape[0]
    _need(x, "x", x.dtype, dev)
    for n, t, k in (("gate_blk", gate_blk, I * H // 64 * 36), ("up_blk", up_blk, I * H // 64 * 36),
                    ("down_blk", down_blk, H * I // 64 * 36)):
        _need(t, n, torch.uint8, dev, k)
    if out is None:
        out = torch.empty((M, H), dtype=torch.float32, device=dev)
    _need(out, "out", torch.float32, dev, M * H)
    nb = mlp_workspace_bytes(WQ_FMT_NVFP4, M, H, I, path, act)
    ws = _workspace(nb, dev, workspace)
    rc = lib().mlp_nvfp4_run(M, H, I, _ptr(x), _xdtype(x), _ptr(gate_blk), float(gate_gs), _ptr(up_blk),
                             float(up_gs), _ptr(down_blk), float(down_gs), _ptr(ws), ws.numel(), _ptr(out),
                             _PATHS[path] | sflags | _ACTS[act], _stream(dev))
    _check("mlp_nvfp4_run", rc)
    return out


def awq_bank_bytes(E, N, K, meta_layout=3):
    return lib().awq_bank_bytes(E, N, K, meta_layout)


def moe_awq_m1_run(x, expert_ids, router_w, w13_bank, w2_bank, E, I, meta_layout=3, act=None, out=None):
    """AWQ routed-expert M=1 step.  x f16-bits [H] (int16/uint16 view or float16); ids int32; weights f32."""
    dev = x.device
    H = x.numel()
    topk = expert_ids.numel()
    xb = x.view(torch.int16) if x.dtype in (torch.float16, torch.int16) else None
    if xb is None:
        raise TypeError("x must be float16 (or its int16 bits)")
    _need(xb, "x", torch.int16, dev)
    _need(expert_ids, "expert_ids", torch.int32, dev)
    _need(router_w, "router_w", torch.float32, dev, topk)
    _need(w13_bank, "w13_bank", torch.uint8, dev, awq_bank_bytes(E, 2 * I, H, meta_layout))
    _need(w2_bank, "w2_bank", torch.uint8, dev, awq_bank_bytes(E, H, I, meta_layout))
    if act is None:
        act = torch.empty((topk, I), dtype=torch.float16, device=dev)
    if out is None:
        out = torch.empty((H,), dtype=torch.float16, device=dev)
    _need(act, "act", torch.float16, dev, topk * I)
    _need(out, "out", torch.float16, dev, H)
    rc = lib().moe_awq_m1_run(E, topk, H, I, _ptr(xb), _ptr(expert_ids), _ptr(router_w), _ptr(w13_bank),
                              _ptr(w2_bank), meta_layout, _ptr(act), _ptr(out), _stream(dev))
    _check("moe_awq_m1_run", rc)
    return out, act


def nvfp4_pack_block64(weight_packed, weight_scale, blk=None):
    """[N,K/2] u8 + [N,K/16] u8 (device) -> Block64 records [N,K/64,36] u8."""
    dev = weight_packed.device
    N, Kh = weight_packed.shape
    K = 2 * Kh
    _need(weight_packed, "weight_packed", torch.uint8, dev)
    _need(weight_scale, "weight_scale", torch.uint8, dev, N * K // 16)
    if blk is None:
        blk = torch.empty((N, K // 64, 36), dtype=torch.uint8, device=dev)
    _need(blk, "blk", torch.uint8, dev, N * K // 64 * 36)
    _check("nvfp4_pack_block64", lib().nvfp4_pack_block64(N, K, _ptr(weight_packed), _ptr(weight_scale),
                                                          _ptr(blk), _stream(dev)))
    return blk


def awq_pack_bank(codes, scales, zeros, meta_layout=3, bank=None):
    """codes [E,N,K] u8 (0..15), scales [E,N,K/32] f16 (or int16 bits), zeros [E,N,K/32] u8 -> bank u8."""
    dev = codes.device
    E, N, K = codes.shape
    _need(codes, "codes", torch.uint8, dev)
    sb = scales.view(torch.int16)
    _need(sb, "scales", torch.int16, dev, E * N * K // 32)
    _need(zeros, "zeros", torch.uint8, dev, E * N * K // 32)
    nb = awq_bank_bytes(E, N, K, meta_layout)
    if bank is None:
        bank = torch.empty(nb, dtype=torch.uint8, device=dev)
    _need(bank, "bank", torch.uint8, dev, nb)
    _check("awq_pack_bank", lib().awq_pack_bank(E, N, K, _ptr(codes), _ptr(sb), _ptr(zeros), meta_layout,
                                                _ptr(bank), _stream(dev)))
    return bank


def fp8w_dequant_f32(w, s):
    dev = w.device
    N, K = w.shape
    _need(w, "w", torch.uint8, dev)
    _need(s, "s", torch.float32, dev, N)
    out = torch.empty((N, K), dtype=torch.float32, device=dev)
    _check("fp8w_dequant_f32", lib().fp8w_dequant_f32(N, K, _ptr(w), _ptr(s), _ptr(out), _stream(dev)))
    return out


def nvfp4_dequant_f32(blk, global_scale):
    dev = blk.device
    N, nb, rb = blk.shape
    _need(blk, "blk", torch.uint8, dev)
    out = torch.empty((N, nb * 64), dtype=torch.float32, device=dev)
    _check("nvfp4_dequant_f32", lib().nvfp4_dequant_f32(N, nb * 64, _ptr(blk), float(global_scale), _ptr(out),
                                                        _stream(dev)))
    return out


def awq_dequant_f16(bank, E, N, K, meta_layout=3):
    dev = bank.device
    _need(bank, "bank", torch.uint8, dev)
    out = torch.empty((E, N, K), dtype=torch.float16, device=dev)
    _check("awq_dequant_f16", lib().awq_dequant_f16(E, N, K, _ptr(bank), meta_layout, _ptr(out), _stream(dev)))
    return out


def qlinear_workspace_bytes(fmt, M, N, K, path="auto", act=None):
    return lib().qlinear_workspace_bytes(fmt, M, N, K, _PATHS[path] | _ACTS[act])


def qlinear_run(fmt, x, w, scale=None, global_scale=1.0, N=None, path="auto", out=None, workspace=None, act=None):
    """y = x dq(W)^T.  FP8: w [N,K] u8 + scale [N] f32; NVFP4: w Block64 [N,K/64,36] + global_scale.
    act="e4m3" (NVFP4): x quantized per row to E4M3 first (the W4A8 variant; MFMA path)."""
    dev = x.device
    M, K = x.shape
    N = w.shape[0] if N is None else N
    _need(x, "x", x.dtype, dev)
    _need(w, "w", torch.uint8, dev)
    if scale is not None:
        _need(scale, "scale", torch.float32, dev, N)
    if out is None:
        out = torch.empty((M, N), dtype=torch.float32, device=dev)
    _need(out, "out", torch.float32, dev, M * N)
    nb = 0 if x.dtype == torch.float16 else qlinear_workspace_bytes(fmt, M, N, K, path, act)
    ws = _workspace(nb, dev, workspace) if nb else None
    rc = lib().qlinear_run(fmt, M, N, K, _ptr(x), _xdtype(x, allow_f16=True), _ptr(w), _ptr(scale), float(global_scale), _ptr(ws),
                           0 if ws is None else ws.numel(), _ptr(out), _PATHS[path] | _ACTS[act], _stream(dev))
    _check("qlinear_run", rc)
    return out


def wq_read_probe(src, sink, nbytes=None, grid=None):
    """Streaming read of nbytes (default: all) of the device tensor src; sink: int32 tensor of >= grid words."""
    dev = src.device
    nbytes = src.numel() * src.element_size() if nbytes is None else nbytes
    grid = sink.numel() if grid is None else grid
    _need(sink, "sink", torch.int32, dev)
    if grid > sink.numel() or nbytes > src.numel() * src.element_size():
        raise ValueError("grid exceeds sink or nbytes exceeds src")
    _check("wq_read_probe", lib().wq_read_probe(_ptr(src), nbytes, _ptr(sink), grid, _stream(dev)))


_FLOATS = {torch.float32: WQ_F32, torch.bfloat16: WQ_BF16, torch.float16: WQ_F16}


def _float_code(dtype, name, allowed=(torch.float32, torch.bfloat16, torch.float16)):
    if dtype not in allowed:
        raise TypeError(f"{name} must be one of {[str(d) for d in allowed]}, got {dtype}")
    return _FLOATS[dtype]


def lora_workspace_bytes(M, K, N, E, R, backward=False):
    return lib().lora_workspace_bytes(M, K, N, E, R, int(backward))


def _want(t, name, dtype, dev, numel):
    """_need for the hot calls: one cheap test, and _need's own errors where it fails."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == dev.index and t.numel() == numel
            and t.is_contiguous()):
        _need(t, name, dtype, dev, numel)
    return t


def _lora_args(x, a, b, scale, ids):
    """Checks shared by the forward and the backward call; (M, K, N, E, R, x code, weight code)."""
    dev, xs, as_, bs = x.device, x.shape, a.shape, b.shape
    if len(xs) != 2 or len(as_) != 3 or len(bs) != 3:
        raise ValueError("x must be [M, K], a [E, R, K] and b [E, N, R]")
    M, K = xs
    E, R, Ka = as_
    N = bs[1]
    if Ka != K or bs[0] != E or bs[2] != R:
        raise ValueError(f"a must be [E, R, {K}] and b [E, N, R], got {tuple(as_)} and {tuple(bs)}")
    xt, wt = _float_code(x.dtype, "x"), _float_code(a.dtype, "a")
    _want(x, "x", x.dtype, dev, M * K)
    _want(a, "a", a.dtype, dev, E * R * K)
    _want(b, "b", a.dtype, dev, E * N * R)
    _want(scale, "scale", torch.float32, dev, E)
    _want(ids, "ids", torch.int32, dev, M)
    return M, K, N, E, R, xt, wt


def lora_run(x, a, b, scale, ids, y, out=None, workspace=None):
    """out[m] = y[m] + scale[e] * (x[m] a[e]^T) b[e]^T with e = ids[m]; out[m] = y[m] where ids[m] is outside [0, E).

    x [M,K] f32/bf16/f16; a [E,R,K] and b [E,N,R] f32/bf16/f16; scale [E] f32; ids [M] int32; y [M,N] f32 (a
    projection's result) or None for zeros.  out [M,N] f32 (may be y: in place)."""
    M, K, N, E, R, xt, wt = _lora_args(x, a, b, scale, ids)
    dev = x.device
    if y is not None:
        _want(y, "y", torch.float32, dev, M * N)
    if out is None:
        out = torch.empty((M, N), dtype=torch.float32, device=dev)
    else:
        _want(out, "out", torch.float32, dev, M * N)
    nb = lora_workspace_bytes(M, K, N, E, R)
    ws = _workspace(nb, dev, workspace) if nb else None
    rc = lib().lora_run(M, K, N, E, R, _ptr(x), xt, _ptr(a), _ptr(b), wt, _ptr(scale), _ptr(ids), _ptr(y), _ptr(ws),
                        0 if ws is None else ws.numel(), _ptr(out), _stream(dev))
    _check("lora_run", rc)
    return out


def _result_dtype(name, asked, default, **given):
    """The result's type: that of the given tensors, else the one asked for by name, else the default; TypeError where they differ."""
    want = asked
    for key, t in given.items():
        if t is not None:
            if want is not None and t.dtype != want:
                raise TypeError(f"{key} is {t.dtype}, where {name} or another tensor says {want}")
            want = t.dtype
    return default if want is None else want


def lora_backward(dy, x, a, b, scale, ids, dx0=None, dx=None, da=None, db=None, workspace=None, dx_dtype=None,
                  need=(True, True, True)):
    """Gradients of lora_run: (dx, da, db).  dx = dx0 (None: zeros) + the adapters' part, of dx0's type (or dx_dtype,
    default x's; a TypeError where they differ); da, db float32, summed over each adapter's rows.  need: which of
    (dx, da, db) to compute (others None).  dx may be dx0 (in place)."""
    want = _result_dtype("dx_dtype", dx_dtype, x.dtype, dx=dx, dx0=dx0)
    M, K, N, E, R, xt, wt = _lora_args(x, a, b, scale, ids)
    dev = x.device
    dyt = _float_code(dy.dtype, "dy", (torch.float32, torch.bfloat16))
    _want(dy, "dy", dy.dtype, dev, M * N)
    dxt = _float_code(want, "dx")
    if dx0 is not None:
        _want(dx0, "dx0", want, dev, M * K)
    outs = []
    for t, name, shape, dtype, wanted in ((dx, "dx", (M, K), want, need[0]), (da, "da", (E, R, K), torch.float32, need[1]),
                                          (db, "db", (E, N, R), torch.float32, need[2])):
        if not wanted:
            outs.append(None)
            continue
        if t is None:
            t = torch.empty(shape, dtype=dtype, device=dev)
        else:
            _want(t, name, dtype, dev, shape[0] * shape[1] * (shape[2] if len(shape) == 3 else 1))
        outs.append(t)
    ws = _workspace(lora_workspace_bytes(M, K, N, E, R, True), dev, workspace)
    rc = lib().lora_backward(M, K, N, E, R, _ptr(dy), dyt, _ptr(x), xt, _ptr(a), _ptr(b), wt, _ptr(scale), _ptr(ids),
                             _ptr(dx0), dxt, _ptr(ws), ws.numel(), _ptr(outs[0]), _ptr(outs[1]), _ptr(outs[2]), _stream(dev))
    _check("lora_backward", rc)
    return tuple(outs)


def qlinear_backward_workspace_bytes(fmt, M, N, K, dx_dtype=torch.float32):
    return lib().qlinear_backward_workspace_bytes(fmt, M, N, K, _FLOATS[dx_dtype])


def qlinear_backward(fmt, dy, w, scale=None, global_scale=1.0, dtype=None, out=None, workspace=None):
    """dx = dy dq(W): the gradient of qlinear_run with respect to its input.  dy [M,N] f32/bf16; w, scale and
    global_scale as for qlinear_run; dx [M,K] f32/bf16 (out's type, or dtype, default dy's;
    a TypeError where they differ)."""
    want = _result_dtype("dtype", dtype, dy.dtype, out=out)
    dev = dy.device
    M, N = dy.shape
    if N == 0:
        raise ValueError("dy must have at least one column")
    dyt = _float_code(dy.dtype, "dy", (torch.float32, torch.bfloat16))
    _want(dy, "dy", dy.dtype, dev, M * N)
    if w.shape[0] != N:
        raise ValueError(f"w must have {N} rows, has {w.shape[0]}")
    K = w.numel() // 36 * 64 // N if fmt == WQ_FMT_NVFP4 else w.numel() // N
    _want(w, "w", torch.uint8, dev, N * (K // 64) * 36 if fmt == WQ_FMT_NVFP4 else N * K)
    if scale is not None:
        _want(scale, "scale", torch.float32, dev, N)
    dxt = _float_code(want, "dx", (torch.float32, torch.bfloat16))
    if out is None:
        out = torch.empty((M, K), dtype=want, device=dev)
    else:
        _want(out, "out", want, dev, M * K)
    nb = qlinear_backward_workspace_bytes(fmt, M, N, K, want)
    ws = _workspace(nb, dev, workspace) if nb else None
    rc = lib().qlinear_backward(fmt, M, N, K, _ptr(dy), dyt, _ptr(w), _ptr(scale), float(global_scale), _ptr(ws),
                                0 if ws is None else ws.numel(), _ptr(out), dxt, _stream(dev))
    _check("qlinear_backward", rc)
    return out


def adamw_table_bytes(count):
    return lib().adamw_table_bytes(count)


class AdamWTable:
    """A built AdamW table: the device buffer and references to the tensors whose addresses it holds."""

    def __init__(self, table, count, elems, bits, tensors):
        self.table, self.count, self.elems, self.bits, self.tensors = table, count, elems, bits, tensors


def adamw_table(params, grads, m, v, copies=None, m_scales=None, v_scales=None, keep_v=False):
    """Table of the tensors adamw_run steps over (lists of equal length): params f32, grads f32/bf16, states m and v
    f32, or, with m_scales and v_scales (f32, one per WQ_ADAMW_BLOCK elements), 8-bit codes (float8_e4m3fn and
    float8_e5m2, or their uint8 views); copies: bf16/f16 tensors that receive the rounded parameters (entries may be
    None).  keep_v (8-bit states): a positive v keeps a positive code, for blocks whose gradients lie further apart than
    2^16.  The table holds addresses: rebuild it when a tensor is replaced.  Waits for the current stream."""
    count = len(params)
    bits = 8 if m_scales is not None else 32
    if (m_scales is None) != (v_scales is None):
        raise ValueError("m_scales and v_scales come together")
    if keep_v and bits != 8:
        raise ValueError("keep_v is for 8-bit states")
    lists = {"grads": grads, "m": m, "v": v, "copies": copies, "m_scales": m_scales, "v_scales": v_scales}
    for name, ts in lists.items():
        if ts is not None and len(ts) != count:
            raise ValueError(f"{name} must have {count} entries, has {len(ts)}")
    if count == 0:
        raise ValueError("no tensors")
    dev = params[0].device
    kinds = {"m": (torch.float8_e4m3fn, torch.uint8), "v": (torch.float8_e5m2, torch.uint8)}
    arr = (_AdamWTensor * count)()
    for i, p in enumerate(params):
        n = p.numel()
        _need(p, f"params[{i}]", torch.float32, dev)
        t = arr[i]
        t.n, t.p = n, _ptr(p)
        t.g_dtype = _float_code(grads[i].dtype, f"grads[{i}]", (torch.float32, torch.bfloat16))
        t.g = _ptr(_need(grads[i], f"grads[{i}]", grads[i].dtype, dev, n))
        for name, s in (("m", m[i]), ("v", v[i])):
            if bits == 8 and s.dtype not in kinds[name]:
                raise TypeError(f"{name}[{i}] must be {kinds[name][0]} or torch.uint8, got {s.dtype}")
            setattr(t, name, _ptr(_need(s, f"{name}[{i}]", s.dtype if bits == 8 else torch.float32, dev, n)))
        if bits == 8:
            blocks = (n + WQ_ADAMW_BLOCK - 1) // WQ_ADAMW_BLOCK
            t.m_scale = _ptr(_need(m_scales[i], f"m_scales[{i}]", torch.float32, dev, blocks))
            t.v_scale = _ptr(_need(v_scales[i], f"v_scales[{i}]", torch.float32, dev, blocks))
        c = copies[i] if copies is not None else None
        if c is not None:
            t.copy_dtype = _float_code(c.dtype, f"copies[{i}]", (torch.bfloat16, torch.float16))
            t.copy = _ptr(_need(c, f"copies[{i}]", c.dtype, dev, n))
    table = torch.empty(max(adamw_table_bytes(count), 1), dtype=torch.uint8, device=dev)
    _check("adamw_table_build", lib().adamw_table_build(count, arr, bits | (WQ_ADAMW_KEEP_V if keep_v else 0), _ptr(table), table.numel(), _stream(dev)))
    torch.cuda.current_stream(dev).synchronize()      # built once: steps on any stream may follow
    keep = (list(params), list(grads), list(m), list(v), copies and list(copies), m_scales and list(m_scales),
            v_scales and list(v_scales))
    return AdamWTable(table, count, sum(p.numel() for p in params), bits, keep)


def adamw_run(table, step, lr, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01, grad_scale=1.0, seed=0):
    """One AdamW step over the table's tensors, in place.  step: int64 device tensor holding t >= 1; lr: float32
    device tensor (both read on the device when the step runs); seed: of the 8-bit states' stochastic rounding."""
    dev = table.table.device
    _want(step, "step", torch.int64, dev, 1)
    _want(lr, "lr", torch.float32, dev, 1)
    rc = lib().adamw_run(table.count, table.elems, table.bits, _ptr(table.table), _ptr(step), _ptr(lr), beta1, beta2, eps,
                         weight_decay, grad_scale, seed & 0xFFFFFFFF, _stream(dev))
    _check("adamw_run", rc)


def _empty_as(t, dtype):
    """A new tensor of t's shape (t dense); empty_like spares half a microsecond where the types agree."""
    return torch.empty_like(t) if t.dtype is dtype else torch.empty(t.shape, dtype=dtype, device=t.device)


def awq_linear_workspace_bytes(M, N, K, x_dtype=torch.float32):
    return lib().awq_linear_workspace_bytes(M, N, K, _FLOATS[x_dtype])


def awq_linear_run(x, bank, N, meta_layout=3, out=None, workspace=None):
    """y = x dq(W)^T with AWQ int4 group-32 weights.  x [M,K] f32/bf16/f16; bank: the [N,K] weights as awq_pack_bank lays
    them out (E = 1); y [M,N] f32."""
    dev = x.device
    if x.dim() != 2:
        raise ValueError("x must be [M, K]")
    M, K = x.shape
    xt = _float_code(x.dtype, "x")
    _want(x, "x", x.dtype, dev, M * K)
    _want(bank, "bank", torch.uint8, dev, awq_bank_bytes(1, N, K, meta_layout))
    if out is None:
        out = torch.empty((M, N), dtype=torch.float32, device=dev)
    else:
        _want(out, "out", torch.float32, dev, M * N)
    nb = awq_linear_workspace_bytes(M, N, K, x.dtype)
    ws = _workspace(nb, dev, workspace) if nb else None
    rc = lib().awq_linear_run(M, N, K, _ptr(x), xt, _ptr(bank), meta_layout, _ptr(ws), 0 if ws is None else ws.numel(),
                              _ptr(out), _stream(dev))
    _check("awq_linear_run", rc)
    return out


def awq_linear_backward_workspace_bytes(M, N, K, dy_dtype=torch.float32, dx_dtype=torch.float32):
    return lib().awq_linear_backward_workspace_bytes(M, N, K, _FLOATS[dy_dtype], _FLOATS[dx_dtype])


def awq_linear_backward(dy, bank, K, meta_layout=3, dtype=None, out=None, workspace=None):
    """dx = dy dq(W): the gradient of awq_linear_run with respect to its input.  dy [M,N] f32/bf16; bank as for
    awq_linear_run; dx [M,K] f32/bf16 (out's type, or dtype, default dy's; a TypeError where they differ)."""
    want = _result_dtype("dtype", dtype, dy.dtype, out=out)
    dev = dy.device
    if dy.dim() != 2:
        raise ValueError("dy must be [M, N]")
    M, N = dy.shape
    dyt = _float_code(dy.dtype, "dy", (torch.float32, torch.bfloat16))
    dxt = _float_code(want, "dx", (torch.float32, torch.bfloat16))
    _want(dy, "dy", dy.dtype, dev, M * N)
    _want(bank, "bank", torch.uint8, dev, awq_bank_bytes(1, N, K, meta_layout))
    if out is None:
        out = torch.empty((M, K), dtype=want, device=dev)
    else:
        _want(out, "out", want, dev, M * K)
    nb = awq_linear_backward_workspace_bytes(M, N, K, dy.dtype, want)
    ws = _workspace(nb, dev, workspace) if nb else None
    rc = lib().awq_linear_backward(M, N, K, _ptr(dy), dyt, _ptr(bank), meta_layout, _ptr(ws), 0 if ws is None else ws.numel(),
                                   _ptr(out), dxt, _stream(dev))
    _check("awq_linear_backward", rc)
    return out


def moe_awq_workspace_bytes(M, E, topk, H, I):
    return lib().moe_awq_workspace_bytes(M, E, topk, H, I)


def moe_awq_run(x, w13_bank, w2_bank, E, I, topk=None, router=None, ids=None, weights=None, renorm=True, meta_layout=3,
                dtype=None, out=None, workspace=None):
    """A mixture-of-experts layer for the M <= WQ_MOE_MAX_TOKENS rows of x [M,H] f32/bf16/f16: the router's topk experts of
    each row, their SwiGLU MLPs with AWQ weights (banks as for moe_awq_m1_run), their weighted sum.

    With router [E,H] f32/bf16/f16 the call chooses: ids and weights [M,topk] (int32, f32) are written (allocated where not
    given), the weights a softmax over the chosen logits, or with renorm=False their share in the softmax over all.  Without
    router, ids and weights are inputs; ids outside [0, E) contribute nothing.  out [M,H] of `dtype` (default x's type, or
    out's).  Returns (out, ids, weights)."""
    dev = x.device
    if x.dim() != 2:
        raise ValueError("x must be [M, H]")
    M, H = x.shape
    xt = _float_code(x.dtype, "x")
    _want(x, "x", x.dtype, dev, M * H)
    want = _result_dtype("dtype", dtype, x.dtype, out=out)
    ot = _float_code(want, "out")
    rt = 0
    if router is not None:
        rt = _float_code(router.dtype, "router")
        _want(router, "router", router.dtype, dev, E * H)
        if topk is None:
            raise ValueError("topk must be given with router")
        if ids is None:
            ids = torch.empty((M, topk), dtype=torch.int32, device=dev)
        if weights is None:
            weights = torch.empty((M, topk), dtype=torch.float32, device=dev)
    elif ids is None or weights is None:
        raise ValueError("without router, ids and weights must be given")
    elif topk is None:
        if ids.dim() != 2:
            raise ValueError("ids must be [M, topk]")
        topk = ids.shape[1]
    _want(ids, "ids", torch.int32, dev, M * topk)
    _want(weights, "weights", torch.float32, dev, M * topk)
    _want(w13_bank, "w13_bank", torch.uint8, dev, awq_bank_bytes(E, 2 * I, H, meta_layout))
    _want(w2_bank, "w2_bank", torch.uint8, dev, awq_bank_bytes(E, H, I, meta_layout))
    if out is None:
        out = _empty_as(x, want)
    else:
        _want(out, "out", want, dev, M * H)
    nb = moe_awq_workspace_bytes(M, E, topk, H, I)
    ws = _workspace(nb, dev, workspace) if nb else None
    rc = lib().moe_awq_run(M, E, topk, H, I, _ptr(x), xt, _ptr(router), rt, _ptr(ids), _ptr(weights), _ptr(w13_bank),
                           _ptr(w2_bank), meta_layout, _ptr(ws), 0 if ws is None else ws.numel(), _ptr(out), ot,
                           WQ_MOE_RENORM if router is not None and renorm else 0, _stream(dev))
    _check("moe_awq_run", rc)
    return out, ids, weights


def _norm_args(h, y, post, gate, pre):
    """Checks shared by block_norm_run and its backward call; (M, H, G, h code, y code, weight code, gate code)."""
    dev = h.device
    if h.dim() != 2:
        raise ValueError("h must be [M, H]")
    M, H = h.shape
    ht = _float_code(h.dtype, "h")
    _want(h, "h", h.dtype, dev, M * H)
    yt = wt = gt = 0
    G = 1
    if y is None:
        if post is not None or gate is not None:
            raise ValueError("post and gate need y")
        if pre is None:
            raise ValueError("neither y nor pre: nothing to do")
    else:
        yt = _float_code(y.dtype, "y")
        _want(y, "y", y.dtype, dev, M * H)
    if post is not None or pre is not None:
        first = post if post is not None else pre
        wt = _float_code(first.dtype, "post and pre")
        for t, name in ((post, "post"), (pre, "pre")):
            if t is not None:
                _want(t, name, first.dtype, dev, H)
    if gate is not None:
        gt = _float_code(gate.dtype, "gate")
        if gate.dim() == 2:
            G = gate.shape[0]
        if M % G if G else M:
            raise ValueError(f"gate must be [G, H] with G a divisor of the {M} rows, has {G} rows")
        _want(gate, "gate", gate.dtype, dev, G * H)
    return M, H, G, ht, yt, wt, gt


def block_norm_run(h, y=None, post=None, gate=None, alpha=1.0, pre=None, eps=1e-6, offset=0.0, x_dtype=None, h_out=None,
                   x=None):
    """h_out = h + alpha * gate * norm(y; post) and x = norm(h_out; pre), what stands between one block and the next;
    norm(t; w) = t / sqrt(mean(t^2) + eps) * (offset + w).

    h [M,H] (the residual stream) and y [M,H] (a block's result) f32/bf16/f16; post and pre [H] of one float type; gate
    [G,H], G a divisor of M (row j for the M/G rows from j M/G on), or [H].  Without post, y enters as it is; without y
    only the norm before a block is taken (h_out is h); without pre no x (None).  x of x_dtype (default h's type), h_out of
    h's type (may be h: in place).  Returns (h_out, x)."""
    M, H, G, ht, yt, wt, gt = _norm_args(h, y, post, gate, pre)
    dev = h.device
    xt = 0
    if pre is not None:
        want = _result_dtype("x_dtype", x_dtype, h.dtype, x=x)
        xt = _float_code(want, "x")
        if x is None:
            x = _empty_as(h, want)
        else:
            _want(x, "x", want, dev, M * H)
    elif x is not None or x_dtype is not None:
        raise ValueError("x and x_dtype need pre")
    if y is not None:
        if h_out is None:
            h_out = torch.empty_like(h)
        else:
            _want(h_out, "h_out", h.dtype, dev, M * H)
    elif h_out is not None:
        raise ValueError("h_out needs y")
    rc = lib().block_norm_run(M, H, _ptr(h), ht, _ptr(y), yt, _ptr(post), _ptr(pre), wt, _ptr(gate), G, gt, alpha, offset, eps,
                              _ptr(h_out), _ptr(x), xt, _stream(dev))
    _check("block_norm_run", rc)
    return (h if y is None else h_out), x


def block_norm_backward_workspace_bytes(M, H, G=1):
    return lib().block_norm_backward_workspace_bytes(M, H, G)


def block_norm_backward(h, y=None, dh=None, dx=None, post=None, gate=None, alpha=1.0, pre=None, eps=1e-6, offset=0.0,
                        dh_in=None, dy=None, dpost=None, dgate=None, dpre=None, workspace=None,
                        need=(True, True, True, True, True)):
    """Gradients of block_norm_run: (dh, dy, dpost, dgate, dpre).  h: the stream after the block (h_out of the forward call,
    or h itself without y); dh: the gradient of h_out from its later uses (None: zeros), of h's type; dx: that of x (with
    pre).  The first result is the gradient of the stream before the block, of h's type (dh_in may be dh: in place); dy of
    y's type; dpost, dpre [H] and dgate [G,H] (or [H] like gate) float32.  need: which of them to compute, where their
    inputs are there (others None)."""
    M, H, G, ht, yt, wt, gt = _norm_args(h, y, post, gate, pre)
    dev = h.device
    if dh is not None:
        _want(dh, "dh", h.dtype, dev, M * H)
    if (dx is None) != (pre is None):
        raise ValueError("dx and pre come together")
    xt = 0
    if dx is not None:
        xt = _float_code(dx.dtype, "dx")
        _want(dx, "dx", dx.dtype, dev, M * H)
    f32 = torch.float32
    outs = []
    for t, name, src, dtype, wanted in ((dh_in, "dh_in", h, h.dtype, need[0]), (dy, "dy", y, y is not None and y.dtype, need[1]),
                                        (dpost, "dpost", post, f32, need[2]), (dgate, "dgate", gate, f32, need[3]),
                                        (dpre, "dpre", pre, f32, need[4])):
        if src is None or not wanted:
            if t is not None:
                raise ValueError(f"{name} is given, but not computed")
            outs.append(None)
            continue
        if t is None:
            t = _empty_as(src, dtype)
        else:
            _want(t, name, dtype, dev, src.numel())
        outs.append(t)
    nb = block_norm_backward_workspace_bytes(M, H, G)
    ws = _workspace(nb, dev, workspace) if nb else None
    rc = lib().block_norm_backward(M, H, _ptr(h), ht, _ptr(y), yt, _ptr(dh), _ptr(dx), xt, _ptr(post), _ptr(pre), wt,
                                   _ptr(gate), G, gt, alpha, offset, eps, _ptr(ws), 0 if ws is None else ws.numel(),
                                   *(_ptr(t) for t in outs), _stream(dev))
    _check("block_norm_backward", rc)
    return tuple(outs)
