"""moe_awq_run in every plan of its products: contractions split over the waves of a workgroup and not, for both matrices, one pass and
several, up to the widest layers; a token's bits in plans that differ; both banks past 4 GiB.

Bounds are those of test_moe_layer.py.  Wide banks with many experts hold a few different ones over and over.
"""
import numpy as np
import pytest
import torch

import weight_quantized_mlp_amd as wq
from adapter_common import DEV, host, randn
from test_moe_layer import check, layer, layer_ref, route_ref

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
pytestmark = pytest.mark.gpu


def split(M, E, topk, K, rows, per):
    """Whether a product's blocks of 512 k are split over waves: where whole pairs of tiles would be too few."""
    return K > 512 and min(M * topk, E) * (rows // per) < 512


def plans(M, E, topk, H, I):
    return split(M, E, topk, H, I, 16), split(M, E, topk, I, H, 32)


def repeated(E0, E, H, I, layout):
    """Banks of E experts, the E0 of a small bank over and over, and the small one's weights."""
    b13, w13, b2, w2 = layer(E0, H, I, layout)
    many = lambda b: b.view(E0, -1).repeat(E // E0, 1).view(-1)
    return many(b13), w13, many(b2), w2


# M, E, different ones, topk, H, I, (W13 split, W2 split)
SHAPES = [(1, 8, 8, 2, 256, 704, (False, True)), (3, 16, 16, 4, 96, 1056, (False, True)), (40, 1, 1, 1, 64, 544, (False, True)),
          (19, 2, 2, 2, 1056, 1568, (True, True)), (45, 3, 3, 3, 576, 96, (True, False)), (16, 64, 8, 4, 640, 608, (False, False)),
          (2, 4, 4, 2, 16384, 64, (True, False)), (3, 4, 4, 2, 64, 16384, (False, True)), (18, 1, 1, 1, 16384, 32, (True, False)),
          (18, 1, 1, 1, 32, 16384, (False, True)),
          (26, 256, 4, 10, 16384, 32, (False, False)), (52, 512, 4, 10, 32, 16384, (False, False))]


@pytest.mark.parametrize("layout", [3, 4])
@pytest.mark.parametrize("xt", [F32, BF16, F16])
@pytest.mark.parametrize("M,E,E0,topk,H,I,want", SHAPES)
def test_plans(M, E, E0, topk, H, I, want, xt, layout):
    print("[moe plan]", M, E, topk, H, I, xt, layout, flush=True)
    assert plans(M, E, topk, H, I) == want
    b13, w13, b2, w2 = repeated(E0, E, H, I, layout)
    x, xd = randn(M + H, (M, H), xt)
    router, rd = randn(E + 1, (E, H), F32, 2 * H ** -0.5)
    guard = torch.full((M * H + 64,), 7.0, device=DEV)
    out, ids, weights = wq.moe_awq_run(x, b13, b2, E, I, topk, router=router, meta_layout=layout, dtype=F32, out=guard[: M * H].view(M, H))
    assert (guard[M * H:] == 7.0).all()
    ref_ids, ref_w = route_ref(xd, rd, topk, True)
    assert np.array_equal(host(ids), ref_ids)
    ref, bound = layer_ref(xd, xt, ref_ids % E0, ref_w, w13, w2)
    check(out, ref, bound, F32, H + I, 64)


@pytest.mark.parametrize("layout", [3, 4])
@pytest.mark.parametrize("xt", [F32, BF16, F16])
def test_a_token_is_the_same_in_plans_that_differ(xt, layout):
    """Alone both products are split over waves; in batches neither is, with one pass and with several; in between one of them is."""
    E, topk, H, I = 64, 8, 1056, 544
    assert plans(1, E, topk, H, I) == (True, True) and plans(2, E, topk, H, I) == plans(200, E, topk, H, I) == (False, False)
    b13, _, b2, _ = repeated(8, E, H, I, layout)
    x, _ = randn(5, (200, H), xt)
    router, _ = randn(6, (E, H), F32, H ** -0.5)
    run = lambda rows: wq.moe_awq_run(x[rows].contiguous(), b13, b2, E, I, topk, router=router, meta_layout=layout, dtype=F32)
    out, ids, w = run(list(range(200)))
    for rows in [[m] for m in (0, 7, 39, 101, 199)] + [[3, 39], list(range(40)), list(range(199, -1, -1))]:
        o, i, ww = run(rows)
        assert torch.equal(o, out[rows]) and torch.equal(i, ids[rows]) and torch.equal(ww, w[rows]), rows


def test_one_product_split_and_the_other_not():
    """Batches of the same tokens: both split up to 8, W2 alone up to 14, neither above."""
    E, topk, H, I = 40, 1, 1152, 928
    assert [plans(n, E, topk, H, I) for n in (8, 9, 14, 15)] == [(True, True), (False, True), (False, True), (False, False)]
    b13, _, b2, _ = repeated(4, E, H, I, 3)
    x, _ = randn(5, (40, H), BF16)
    ids = (torch.arange(40, device=DEV, dtype=torch.int32) * 7 % E)[:, None].contiguous()
    w = torch.rand((40, 1), device=DEV)
    run = lambda n: wq.moe_awq_run(x[:n].contiguous(), b13, b2, E, I, ids=ids[:n].contiguous(), weights=w[:n].contiguous(), dtype=F32)[0]
    out = run(40)
    for n in (1, 8, 9, 14, 15, 17, 29, 39):
        assert torch.equal(run(n), out[:n]), n


def test_both_banks_past_4_GiB():
    """The last experts of banks that both pass 2^32 bytes give what a small bank of just them gives, on either side of the boundary."""
    topk, H, I, M = 2, 2560, 160, 3
    n13, n2 = wq.awq_bank_bytes(1, 2 * I, H), wq.awq_bank_bytes(1, H, I)
    E = (1 << 32) // n2 + 3
    assert (E - 2) * n13 > 1 << 32 and (E - 2) * n2 > 1 << 32
    s13, _, s2, _ = layer(2, H, I, 3)
    b13, b2 = (torch.zeros((E, n), dtype=torch.uint8, device=DEV) for n in (n13, n2))
    x, _ = randn(1, (M, H), BF16)
    ids = torch.tensor([[0, 1], [1, 0], [1, 1]], dtype=torch.int32, device=DEV)
    w = torch.tensor([[0.3, 0.7], [0.5, 0.5], [1.0, -0.5]], device=DEV)
    small, _, _ = wq.moe_awq_run(x, s13, s2, 2, I, ids=ids, weights=w)
    for first in (E - 2, (1 << 32) // n2 - 1, (1 << 32) // n13 - 1):
        b13[first:first + 2] = s13.view(2, n13)
        b2[first:first + 2] = s2.view(2, n2)
        large, _, _ = wq.moe_awq_run(x, b13.view(-1), b2.view(-1), E, I, ids=ids + first, weights=w)
        assert torch.equal(small, large), first
