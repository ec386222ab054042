"""Host-only checks of the adapter, input-gradient and AdamW entry points: symbols, sizes and refusals.

Every refusal here comes from the pure-arithmetic phase, before any HIP call, so these run without a GPU; pointers
are made-up addresses that are never read.
"""
import ctypes
import os
import re
import shutil
import subprocess

import pytest

import weight_quantized_mlp_amd as wq

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
EINVAL, EALIGN, EOVERLAP, EWORKSPACE = -1, -2, -3, -6
A = 1 << 32
MB = 1 << 20


@pytest.fixture(scope="module")
def L():
    return wq.lib()


def test_every_declared_symbol_is_exported(L):
    text = open(os.path.join(ROOT, "include", "wqmlp_adapters.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = set(re.findall(r"^\s*(?:size_t|int)\s+(\w+)\(", text, flags=re.M))
    assert names == {"lora_workspace_bytes", "lora_run", "lora_backward", "qlinear_backward_workspace_bytes",
                     "qlinear_backward", "adamw_table_bytes", "adamw_table_build", "adamw_run"}
    for n in names:
        assert hasattr(L, n) and (n in wq.__all__ or n == "adamw_table_build")


def lora_args(**kw):
    a = dict(M=4, K=2048, N=48, E=2, R=8, x=A, xt=1, a=A + MB, b=A + 2 * MB, wt=1, sc=A + 3 * MB, ids=A + 4 * MB,
             y=A + 5 * MB, ws=A + 6 * MB, wsb=MB, out=A + 7 * MB)
    a.update(kw)
    return [a[k] for k in ("M", "K", "N", "E", "R", "x", "xt", "a", "b", "wt", "sc", "ids", "y", "ws", "wsb", "out")] + [None]


@pytest.mark.parametrize("kw,rc", [
    (dict(x=None), EINVAL), (dict(a=None), EINVAL), (dict(b=None), EINVAL), (dict(sc=None), EINVAL),
    (dict(ids=None), EINVAL), (dict(out=None), EINVAL), (dict(xt=3), EINVAL), (dict(wt=-1), EINVAL),
    (dict(M=-1), EINVAL), (dict(M=(1 << 23) + 1), EINVAL), (dict(K=0), EINVAL), (dict(K=72), EINVAL), (dict(N=0), EINVAL),
    (dict(E=0), EINVAL), (dict(R=0), EINVAL), (dict(R=4), EINVAL), (dict(R=12), EINVAL), (dict(R=264), EINVAL),
    (dict(M=1 << 23, N=1 << 14), EINVAL), (dict(E=1 << 23, N=1 << 14), EINVAL),
    (dict(x=A + 8), EALIGN), (dict(ids=A + 4 * MB + 4), EALIGN), (dict(y=A + 5 * MB + 2), EALIGN), (dict(ws=A + 6 * MB + 1), EALIGN),
    (dict(ws=None), EWORKSPACE), (dict(wsb=0), EWORKSPACE),
    (dict(out=A), EOVERLAP), (dict(out=A + MB), EOVERLAP), (dict(out=A + 5 * MB + 16), EOVERLAP), (dict(ws=A + 5 * MB), EOVERLAP),
    (dict(ws=A + 7 * MB), EOVERLAP), (dict(out=A + 4 * MB), EOVERLAP),
])
def test_lora_refusals(L, kw, rc):
    assert L.lora_run(*lora_args(**kw)) == rc


def test_lora_empty_calls(L):
    assert L.lora_run(*lora_args(M=0, x=None, ids=None, y=None, out=None, ws=None, wsb=0)) == 0
    assert L.lora_run(*lora_args(M=0, a=None)) == EINVAL
    assert L.lora_workspace_bytes(0, 64, 48, 2, 9, 0) == 0
    assert L.lora_workspace_bytes(4, 64, 48, 2, 8, 2) == 0
    assert L.lora_workspace_bytes(4, 2048, 48, 2, 8, 0) >= 4 * 8 * 4
    assert L.lora_workspace_bytes(4, 64, 48, 2, 8, 0) == 0              # a small adapter: one launch, no intermediate
    assert L.lora_workspace_bytes(4, 64, 48, 2, 8, 1) >= 2 * 4 * 8 * 4


def back_args(**kw):
    a = dict(M=4, K=64, N=48, E=2, R=8, dy=A, dyt=0, x=A + MB, xt=1, a=A + 2 * MB, b=A + 3 * MB, wt=1, sc=A + 4 * MB,
             ids=A + 5 * MB, dx0=A + 6 * MB, dxt=1, ws=A + 7 * MB, wsb=MB, dx=A + 8 * MB, da=A + 9 * MB, db=A + 10 * MB)
    a.update(kw)
    return [a[k] for k in ("M", "K", "N", "E", "R", "dy", "dyt", "x", "xt", "a", "b", "wt", "sc", "ids", "dx0", "dxt", "ws",
                           "wsb", "dx", "da", "db")] + [None]


@pytest.mark.parametrize("kw,rc", [
    (dict(dy=None), EINVAL), (dict(x=None), EINVAL), (dict(ids=None), EINVAL), (dict(sc=None), EINVAL),
    (dict(dyt=2), EINVAL), (dict(dxt=3), EINVAL), (dict(xt=5), EINVAL), (dict(R=260), EINVAL), (dict(K=8), EINVAL),
    (dict(dx=None, da=None, db=None), EINVAL), (dict(dx=A + 8 * MB + 8), EALIGN), (dict(dx0=A + 6 * MB + 2), EALIGN),
    (dict(ws=None), EWORKSPACE), (dict(dx=A + MB), EOVERLAP), (dict(da=A + 2 * MB), EOVERLAP),
    (dict(da=A + 10 * MB), EOVERLAP), (dict(dx0=A + 8 * MB + 16), EOVERLAP), (dict(db=A), EOVERLAP),
])
def test_lora_backward_refusals(L, kw, rc):
    assert L.lora_backward(*back_args(**kw)) == rc


def test_lora_backward_empty(L):
    assert L.lora_backward(*back_args(M=0, dy=None, x=None, ids=None, dx0=None, da=None, db=None, ws=None, wsb=0)) == 0


def grad_args(fmt, **kw):
    a = dict(fmt=fmt, M=4, N=48, K=64, dy=A, dyt=0, w=A + MB, sc=A + 2 * MB, gs=1.0, ws=A + 3 * MB, wsb=MB, dx=A + 4 * MB, dxt=1)
    a.update(kw)
    return [a[k] for k in ("fmt", "M", "N", "K", "dy", "dyt", "w", "sc", "gs", "ws", "wsb", "dx", "dxt")] + [None]


@pytest.mark.parametrize("fmt,kw,rc", [
    (2, {}, EINVAL), (0, dict(dy=None), EINVAL), (0, dict(w=None), EINVAL), (0, dict(sc=None), EINVAL), (0, dict(dx=None), EINVAL),
    (0, dict(dyt=2), EINVAL), (1, dict(dxt=2), EINVAL), (0, dict(K=40), EINVAL), (1, dict(K=96), EINVAL), (0, dict(N=0), EINVAL),
    (1, dict(gs=0.0), EINVAL), (1, dict(gs=float("inf")), EINVAL), (0, dict(M=-1), EINVAL),
    (0, dict(dy=A + 4), EALIGN), (0, dict(sc=A + 2 * MB + 4), EALIGN),
    (0, dict(dx=A), EOVERLAP), (1, dict(dx=A + MB), EOVERLAP), (0, dict(dx=A + 2 * MB), EOVERLAP),
])
def test_qlinear_backward_refusals(L, fmt, kw, rc):
    assert L.qlinear_backward(*grad_args(fmt, **kw)) == rc


def test_qlinear_backward_workspace(L):
    assert L.qlinear_backward(*grad_args(0, M=0, dy=None, dx=None, ws=None, wsb=0)) == 0
    need = L.qlinear_backward_workspace_bytes(0, 4, 48, 64, 0)
    if need:
        assert L.qlinear_backward(*grad_args(0, dxt=0, wsb=need - 1)) == EWORKSPACE
        assert L.qlinear_backward(*grad_args(0, dxt=0, ws=A + 4 * MB)) == EOVERLAP
    assert L.qlinear_backward_workspace_bytes(0, 4, 48, 64, 2) == 0


def tensor(i=0, **kw):
    base = A + 64 * MB * i
    t = dict(n=1000, p=base, g=base + MB, m=base + 2 * MB, v=base + 3 * MB, m_scale=base + 4 * MB, v_scale=base + 5 * MB,
             copy=base + 6 * MB, g_dtype=0, copy_dtype=1)
    t.update(kw)
    return wq._AdamWTensor(*[t[f[0]] for f in wq._AdamWTensor._fields_])


def build(L, ts, bits=8, table=A - 64 * MB, nbytes=None):
    arr = (wq._AdamWTensor * max(len(ts), 1))(*ts)
    n = L.adamw_table_bytes(len(ts)) if nbytes is None else nbytes
    return L.adamw_table_build(len(ts), arr, bits, table, n, None)


@pytest.mark.parametrize("kw,rc", [
    (dict(n=-1), EINVAL), (dict(p=None), EINVAL), (dict(g=None), EINVAL), (dict(m=None), EINVAL), (dict(v=None), EINVAL),
    (dict(m_scale=None), EINVAL), (dict(v_scale=None), EINVAL), (dict(g_dtype=2), EINVAL), (dict(copy_dtype=0), EINVAL),
    (dict(p=A + 4), EALIGN), (dict(copy=A + 6 * MB + 2), EALIGN), (dict(m=A + 2 * MB + 8), EALIGN),
    (dict(m=A), EOVERLAP), (dict(g=A + 16), EOVERLAP), (dict(v=A + 2 * MB + 992), EOVERLAP), (dict(copy=A + MB), EOVERLAP),
    (dict(p=A - 64 * MB), EOVERLAP), (dict(g=A - 64 * MB), EOVERLAP), (dict(v_scale=A + 4 * MB), EOVERLAP),
])
def test_adamw_table_refusals(L, kw, rc):
    assert build(L, [tensor(**kw)]) == rc
    assert build(L, [tensor(1), tensor(**kw)]) == rc


def test_adamw_table_refusals_between_tensors(L):
    assert build(L, [tensor(0), tensor(1, p=A)]) == EOVERLAP                       # the same parameter twice
    assert build(L, [tensor(0), tensor(1, g=A + 2 * MB)]) == EOVERLAP              # a gradient that is another's state
    assert build(L, [tensor(0)], bits=16) == EINVAL
    assert build(L, [tensor(0)], table=None) == EINVAL
    assert build(L, [tensor(0)], nbytes=8) == EWORKSPACE
    assert build(L, [tensor(0)], table=A - 64 * MB + 8) == EALIGN
    assert L.adamw_table_build(1, None, 8, A, 1 << 20, None) == EINVAL
    assert L.adamw_table_bytes(0) == 0 and L.adamw_table_bytes((1 << 20) + 1) == 0
    assert L.adamw_table_bytes(3) >= 3 * 80


@pytest.mark.parametrize("kw", [dict(count=0), dict(elems=-1), dict(bits=4), dict(table=None), dict(step=None), dict(lr=None),
                                dict(b1=1.0), dict(b1=-0.1), dict(b2=float("nan")), dict(eps=-1.0), dict(eps=float("inf")),
                                dict(wd=-0.1)])
def test_adamw_run_refusals(L, kw):
    a = dict(count=1, elems=10, bits=32, table=A, step=A + MB, lr=A + 2 * MB, b1=0.9, b2=0.999, eps=1e-8, wd=0.0, gs=1.0, seed=0)
    a.update(kw)
    assert L.adamw_run(*a.values(), None) == EINVAL
    a = dict(a, **{k: v for k, v in dict(count=1, elems=10, bits=32, table=A, step=A + MB + 8, lr=A, b1=0.9, b2=0.9, eps=0.0, wd=0.0).items()})
    assert L.adamw_run(*a.values(), None) == EALIGN


def test_python_refusals():
    import torch
    x = torch.zeros(4, 64)
    a, b = torch.zeros(2, 8, 64), torch.zeros(2, 48, 8)
    sc, ids = torch.zeros(2), torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        wq.lora_run(x, a, b, sc, ids, None)                         # host tensors
    with pytest.raises(ValueError):
        wq.lora_run(x, a[:, :, :32], b, sc, ids, None)
    with pytest.raises(ValueError):
        wq.lora_run(x, a, torch.zeros(2, 48, 16), sc, ids, None)
    with pytest.raises(TypeError):
        wq.lora_run(x.double(), a, b, sc, ids, None)
    with pytest.raises(ValueError):
        wq.adamw_table([], [], [], [])
    with pytest.raises(ValueError):
        wq.adamw_table([x], [x], [x], [x], m_scales=[x])
    with pytest.raises(ValueError):
        wq.adamw_table([x], [x, x], [x], [x])


def test_header_is_strict_c(L, tmp_path):
    gcc = shutil.which("gcc")
    if gcc is None or os.environ.get("WQMLP_LIBRARY"):
        pytest.skip("no C compiler, or another build of the library is loaded")
    src = tmp_path / "c.c"
    src.write_text('#include "wqmlp_adapters.h"\n#include <stdio.h>\nint main(void) {\n'
                   "  if (lora_run(1, 16, 1, 1, 8, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0) != WQ_EINVAL) return 1;\n"
                   "  if (adamw_table_bytes(1) < sizeof(wq_adamw_tensor)) return 2;\n"
                   "  printf(\"%zu\\n\", sizeof(wq_adamw_tensor));\n  return 0;\n}\n")
    d = os.path.dirname(os.path.abspath(wq.lib_path))
    exe = str(tmp_path / "c")
    r = subprocess.run([gcc, "-std=c99", "-Wall", "-Wextra", "-pedantic", "-Werror", "-I", os.path.join(ROOT, "include"),
                        str(src), "-L", d, "-l:libwqmlp.so", "-Wl,-rpath," + d, "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and int(r.stdout) == ctypes.sizeof(wq._AdamWTensor)
