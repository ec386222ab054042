"""Host-only checks of the block entry points: symbols, sizes and refusals.

Every refusal here comes from the pure-arithmetic phase, before any HIP call, so these run without a GPU; pointers
are made-up addresses that are never read.
"""
import os
import re

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
    text = open(os.path.join(ROOT, "include", "wqmlp_blocks.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = set(re.findall(r"^\s*(?:size_t|int)\s+(\w+)\(", text, flags=re.M))
    assert names
    for n in names:
        assert hasattr(L, n) and n in wq.__all__


NORM = ("M", "H", "h", "ht", "y", "yt", "post", "pre", "wt", "gate", "G", "gt", "alpha", "offset", "eps", "ho", "x", "xt")


def norm_args(**kw):
    a = dict(M=12, H=64, h=A, ht=0, y=A + MB, yt=1, post=A + 2 * MB, pre=A + 3 * MB, wt=2, gate=A + 4 * MB, G=3, gt=0, alpha=1.0,
             offset=0.0, eps=1e-6, ho=A + 5 * MB, x=A + 6 * MB, xt=1)
    a.update(kw)
    return [a[k] for k in NORM] + [None]


@pytest.mark.parametrize("kw,rc", [
    (dict(h=None), EINVAL), (dict(y=None), EINVAL), (dict(ho=None), EINVAL), (dict(x=None), EINVAL), (dict(pre=None), EINVAL),
    (dict(ht=3), EINVAL), (dict(yt=-1), EINVAL), (dict(xt=3), EINVAL), (dict(wt=4), EINVAL), (dict(gt=3), EINVAL),
    (dict(M=-1), EINVAL), (dict(M=(1 << 23) + 3), EINVAL), (dict(H=0), EINVAL), (dict(H=60), EINVAL), (dict(H=(1 << 23) + 8), EINVAL),
    (dict(M=1 << 23, H=1 << 14, G=1), EINVAL), (dict(G=0), EINVAL), (dict(G=5), EINVAL), (dict(G=-3), EINVAL), (dict(gate=None), EINVAL),
    (dict(eps=-1.0), EINVAL), (dict(eps=float("nan")), EINVAL), (dict(alpha=float("inf")), EINVAL), (dict(offset=float("nan")), EINVAL),
    (dict(y=None, post=None, gate=None, G=1, ho=None, pre=None, x=None), EINVAL),
    (dict(y=None, post=None, gate=None, G=1), EINVAL), (dict(y=None, ho=None, gate=None, G=1), EINVAL),
    (dict(h=A + 8), EALIGN), (dict(x=A + 6 * MB + 2), EALIGN), (dict(gate=A + 4 * MB + 4), EALIGN), (dict(post=A + 2 * MB + 2), EALIGN),
    (dict(x=A), EOVERLAP), (dict(ho=A + MB), EOVERLAP), (dict(ho=A + 16), EOVERLAP), (dict(x=A + 5 * MB + 64), EOVERLAP),
    (dict(x=A + 4 * MB), EOVERLAP), (dict(ho=A + 3 * MB), EOVERLAP), (dict(x=A + 2 * MB + 16), EOVERLAP),
])
def test_norm_refusals(L, kw, rc):
    assert L.block_norm_run(*norm_args(**kw)) == rc


def test_norm_empty_calls(L):
    assert L.block_norm_run(*norm_args(M=0, h=None, y=None, ho=None, x=None)) == 0
    assert L.block_norm_run(*norm_args(M=0, H=60)) == EINVAL
    assert L.block_norm_backward_workspace_bytes(0, 64, 1) == 0
    assert L.block_norm_backward_workspace_bytes(12, 60, 1) == 0
    assert L.block_norm_backward_workspace_bytes(12, 64, 5) == 0
    assert L.block_norm_backward_workspace_bytes(12, 64, 3) == 3 * 12 * 64 * 4


NGRAD = ("M", "H", "h", "ht", "y", "yt", "dh", "dx", "xt", "post", "pre", "wt", "gate", "G", "gt", "alpha", "offset", "eps", "ws", "wsb",
         "dhi", "dy", "dpost", "dgate", "dpre")


def ngrad_args(**kw):
    a = dict(M=12, H=64, h=A, ht=0, y=A + MB, yt=1, dh=A + 2 * MB, dx=A + 3 * MB, xt=1, post=A + 4 * MB, pre=A + 5 * MB, wt=2,
             gate=A + 6 * MB, G=3, gt=0, alpha=1.0, offset=0.0, eps=1e-6, ws=A + 7 * MB, wsb=MB, dhi=A + 8 * MB, dy=A + 9 * MB,
             dpost=A + 10 * MB, dgate=A + 11 * MB, dpre=A + 12 * MB)
    a.update(kw)
    return [a[k] for k in NGRAD] + [None]


@pytest.mark.parametrize("kw,rc", [
    (dict(h=None), EINVAL), (dict(dx=None), EINVAL), (dict(pre=None), EINVAL), (dict(post=None), EINVAL), (dict(gate=None), EINVAL),
    (dict(gate=None, G=1), EINVAL), (dict(y=None), EINVAL), (dict(y=None, post=None, gate=None, G=1, dpost=None, dgate=None), EINVAL),
    (dict(dhi=None, dy=None, dpost=None, dgate=None, dpre=None), EINVAL), (dict(G=5), EINVAL), (dict(H=4), EINVAL), (dict(ht=7), EINVAL),
    (dict(xt=-1), EINVAL), (dict(eps=-1e-9), EINVAL),
    (dict(dh=A + 2 * MB + 8), EALIGN), (dict(dgate=A + 11 * MB + 4), EALIGN), (dict(ws=A + 7 * MB + 1), EALIGN),
    (dict(ws=None), EWORKSPACE), (dict(wsb=3 * 12 * 64 * 4 - 1), EWORKSPACE),
    (dict(dhi=A), EOVERLAP), (dict(dhi=A + 2 * MB + 16), EOVERLAP), (dict(dy=A + MB), EOVERLAP), (dict(dy=A + 8 * MB), EOVERLAP),
    (dict(dpost=A + 4 * MB), EOVERLAP), (dict(dgate=A + 7 * MB), EOVERLAP), (dict(dpre=A + 3 * MB), EOVERLAP),
])
def test_norm_backward_refusals(L, kw, rc):
    assert L.block_norm_backward(*ngrad_args(**kw)) == rc


def test_norm_backward_without_rows(L):
    none = dict(M=0, h=None, y=None, dh=None, dx=None, dhi=None, dy=None, ws=None, wsb=0)
    assert L.block_norm_backward(*ngrad_args(**none, dpost=None, dgate=None, dpre=None)) == 0
    assert L.block_norm_backward(*ngrad_args(**none, pre=None)) == EINVAL


LIN = ("M", "N", "K", "x", "xt", "bank", "layout", "ws", "wsb", "y")


def lin_args(**kw):
    a = dict(M=40, N=48, K=64, x=A, xt=1, bank=A + MB, layout=3, ws=A + 2 * MB, wsb=MB, y=A + 3 * MB)
    a.update(kw)
    return [a[k] for k in LIN] + [None]


@pytest.mark.parametrize("kw,rc", [
    (dict(x=None), EINVAL), (dict(bank=None), EINVAL), (dict(y=None), EINVAL), (dict(xt=3), EINVAL), (dict(xt=-1), EINVAL),
    (dict(layout=2), EINVAL), (dict(M=-1), EINVAL), (dict(N=0), EINVAL), (dict(K=48), EINVAL), (dict(K=0), EINVAL),
    (dict(M=(1 << 23) + 1), EINVAL), (dict(N=(1 << 23) + 1), EINVAL), (dict(M=1 << 23, N=1 << 14), EINVAL),
    (dict(x=A + 8), EALIGN), (dict(bank=A + MB + 4), EALIGN), (dict(y=A + 3 * MB + 4), EALIGN), (dict(ws=A + 2 * MB + 1), EALIGN),
    (dict(ws=None), EWORKSPACE), (dict(wsb=64), EWORKSPACE),
    (dict(y=A), EOVERLAP), (dict(y=A + MB + 1024), EOVERLAP), (dict(ws=A), EOVERLAP), (dict(ws=A + 3 * MB), EOVERLAP),
])
def test_awq_linear_refusals(L, kw, rc):
    assert L.awq_linear_run(*lin_args(**kw)) == rc


def test_awq_linear_empty_calls(L):
    assert L.awq_linear_run(*lin_args(M=0, x=None, y=None, ws=None, wsb=0)) == 0
    assert L.awq_linear_run(*lin_args(M=0, bank=None)) == EINVAL
    assert L.awq_linear_workspace_bytes(0, 48, 64, 0) == 0
    assert L.awq_linear_workspace_bytes(4, 48, 48, 0) == 0
    assert L.awq_linear_workspace_bytes(4, 48, 64, 3) == 0


LGRAD = ("M", "N", "K", "dy", "dyt", "bank", "layout", "ws", "wsb", "dx", "dxt")


def lgrad_args(**kw):
    a = dict(M=4, N=48, K=64, dy=A, dyt=1, bank=A + MB, layout=3, ws=A + 2 * MB, wsb=MB, dx=A + 3 * MB, dxt=0)
    a.update(kw)
    return [a[k] for k in LGRAD] + [None]


@pytest.mark.parametrize("kw,rc", [
    (dict(dy=None), EINVAL), (dict(bank=None), EINVAL), (dict(dx=None), EINVAL), (dict(dyt=2), EINVAL), (dict(dxt=2), EINVAL),
    (dict(layout=5), EINVAL), (dict(M=-1), EINVAL), (dict(N=0), EINVAL), (dict(K=48), EINVAL), (dict(K=0), EINVAL),
    (dict(M=(1 << 23) + 1), EINVAL), (dict(N=(1 << 23) + 1), EINVAL), (dict(M=1 << 23, K=1 << 14), EINVAL),
    (dict(dy=A + 8), EALIGN), (dict(bank=A + MB + 4), EALIGN), (dict(dx=A + 3 * MB + 4), EALIGN), (dict(ws=A + 2 * MB + 1), EALIGN),
    (dict(ws=None), EWORKSPACE), (dict(wsb=64), EWORKSPACE),
    (dict(dx=A), EOVERLAP), (dict(dx=A + MB + 1024), EOVERLAP), (dict(ws=A), EOVERLAP), (dict(ws=A + 3 * MB), EOVERLAP),
])
def test_awq_linear_backward_refusals(L, kw, rc):
    assert L.awq_linear_backward(*lgrad_args(**kw)) == rc


def test_awq_linear_backward_empty_calls(L):
    assert L.awq_linear_backward(*lgrad_args(M=0, dy=None, dx=None, ws=None, wsb=0)) == 0
    assert L.awq_linear_backward(*lgrad_args(M=0, bank=None)) == EINVAL
    assert L.awq_linear_backward_workspace_bytes(0, 48, 64, 0, 0) == 0
    assert L.awq_linear_backward_workspace_bytes(4, 48, 48, 0, 0) == 0
    assert L.awq_linear_backward_workspace_bytes(4, 48, 64, 2, 0) == 0


MOE = ("M", "E", "topk", "H", "I", "x", "xt", "router", "rt", "ids", "w", "w13", "w2", "layout", "ws", "wsb", "out", "ot", "flags")


def moe_args(**kw):
    a = dict(M=4, E=8, topk=2, H=64, I=32, x=A, xt=1, router=A + MB, rt=0, ids=A + 2 * MB, w=A + 3 * MB, w13=A + 4 * MB, w2=A + 5 * MB, layout=3,
             ws=A + 6 * MB, wsb=MB, out=A + 7 * MB, ot=2, flags=1)
    a.update(kw)
    return [a[k] for k in MOE] + [None]


@pytest.mark.parametrize("kw,rc", [
    (dict(x=None), EINVAL), (dict(ids=None), EINVAL), (dict(w=None), EINVAL), (dict(w13=None), EINVAL), (dict(w2=None), EINVAL),
    (dict(out=None), EINVAL), (dict(xt=3), EINVAL), (dict(rt=3), EINVAL), (dict(ot=-1), EINVAL), (dict(layout=5), EINVAL),
    (dict(M=-1), EINVAL), (dict(M=257), EINVAL), (dict(E=0), EINVAL), (dict(topk=0), EINVAL), (dict(topk=17, E=32), EINVAL),
    (dict(topk=9), EINVAL), (dict(H=48), EINVAL), (dict(I=16), EINVAL), (dict(H=0), EINVAL), (dict(I=16416), EINVAL), (dict(H=16416), EINVAL),
    (dict(E=1 << 23, H=1 << 14), EINVAL), (dict(flags=2), EINVAL), (dict(router=None), EINVAL), (dict(router=None, flags=4), EINVAL),
    (dict(x=A + 8), EALIGN), (dict(ids=A + 2 * MB + 4), EALIGN), (dict(w2=A + 5 * MB + 8), EALIGN), (dict(router=A + MB + 2), EALIGN),
    (dict(ws=None), EWORKSPACE), (dict(wsb=256), EWORKSPACE),
    (dict(out=A), EOVERLAP), (dict(out=A + 4 * MB), EOVERLAP), (dict(ids=A + 3 * MB), EOVERLAP), (dict(ids=A + 7 * MB), EOVERLAP),
    (dict(w=A + 6 * MB), EOVERLAP), (dict(ws=A + MB), EOVERLAP), (dict(router=None, flags=0, out=A + 2 * MB), EOVERLAP),
    (dict(router=None, flags=0, ws=A + 3 * MB), EOVERLAP),
])
def test_moe_refusals(L, kw, rc):
    assert L.moe_awq_run(*moe_args(**kw)) == rc


def test_moe_empty_calls(L):
    assert L.moe_awq_run(*moe_args(M=0, x=None, ids=None, w=None, out=None, ws=None, wsb=0)) == 0
    assert L.moe_awq_run(*moe_args(M=0, w13=None)) == EINVAL
    assert L.moe_awq_workspace_bytes(0, 8, 2, 64, 32) == 0
    assert L.moe_awq_workspace_bytes(257, 8, 2, 64, 32) == 0
    assert L.moe_awq_workspace_bytes(4, 8, 2, 48, 32) == 0
