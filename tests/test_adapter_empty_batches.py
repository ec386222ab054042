"""Batches of no rows at the sizes of real projections: size queries, lora_run, lora_backward, qlinear_backward."""
import pytest

import weight_quantized_mlp_amd as wq

SIZES = [(5120, 17408, 1, 16), (17408, 5120, 6, 32), (16384, 64, 2, 8), (64, 16384, 2, 256), (1 << 20, 1 << 20, 3, 64)]


@pytest.mark.parametrize("K,N,E,R", SIZES)
def test_size_queries_of_no_rows(K, N, E, R):
    for backward in (False, True):
        assert wq.lora_workspace_bytes(0, K, N, E, R, backward) <= wq.lora_workspace_bytes(1, K, N, E, R, backward)
    assert wq.lora_workspace_bytes(0, K, N, E, R) == 0             # no intermediate, no parts


@pytest.mark.parametrize("K,N,E,R", SIZES)
def test_calls_of_no_rows_on_the_host(K, N, E, R):
    """Without weight gradients nothing is enqueued, so these return before any device is asked for."""
    A, MB = 1 << 40, 1 << 34
    L = wq.lib()
    assert L.lora_run(0, K, N, E, R, None, 1, A, A + MB, 1, A + 2 * MB, None, None, None, 0, None, None) == 0
    assert L.lora_backward(0, K, N, E, R, None, 1, None, 1, A, A + MB, 1, A + 2 * MB, None, None, 1, None, 0, A + 3 * MB, None,
                           None, None) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("K,N,E,R", SIZES[:4])
def test_calls_of_no_rows(K, N, E, R):
    import torch
    dev = torch.device("cuda:0")
    x, y = torch.empty((0, K), dtype=torch.bfloat16, device=dev), torch.empty((0, N), device=dev)
    a = torch.randn((E, R, K), device=dev).to(torch.bfloat16)
    b = torch.randn((E, N, R), device=dev).to(torch.bfloat16)
    scale, ids = torch.ones(E, device=dev), torch.empty(0, dtype=torch.int32, device=dev)
    assert wq.lora_run(x, a, b, scale, ids, y).shape == (0, N)
    da, db = torch.full((E, R, K), 7.0, device=dev), torch.full((E, N, R), 7.0, device=dev)
    dx, da, db = wq.lora_backward(y, x, a, b, scale, ids, da=da, db=db)
    assert dx.shape == (0, K) and not da.any() and not db.any()


def test_empty_dx_alone_on_the_host():
    """An empty dx may be NULL, so a call that asks for dx alone passes no output at all."""
    A, MB = 1 << 40, 1 << 20
    for M, rc in ((0, 0), (1, -1)):
        x = None if M == 0 else A + 4 * MB
        assert wq.lib().lora_backward(M, 64, 48, 2, 8, x, 1, x, 1, A, A + MB, 1, A + 2 * MB, x, None, 1, None, 0, None, None, None,
                                      None) == rc


@pytest.mark.gpu
def test_empty_dx_alone():
    import torch
    dev = torch.device("cuda:0")
    a, b, scale = torch.ones((2, 8, 64), device=dev), torch.ones((2, 48, 8), device=dev), torch.ones(2, device=dev)
    dx, da, db = wq.lora_backward(torch.empty((0, 48), device=dev), torch.empty((0, 64), device=dev), a, b, scale,
                                  torch.empty(0, dtype=torch.int32, device=dev), need=(True, False, False))
    assert dx.shape == (0, 64) and da is None and db is None
