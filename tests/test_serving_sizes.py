"""Workspace sizes of the serving ops (no GPU): what a call may ask for."""
import pytest
import torch

from zeroth_order_fine_b200 import zo


@pytest.fixture(scope="module", autouse=True)
def built():
    from zeroth_order_fine_b200 import build
    build.build()


MB = 1 << 20


@pytest.mark.parametrize("M", [65, 301, 1000, 4093, 16384, 100000])
@pytest.mark.parametrize("N,K", [(2048, 2048), (20480, 5120), (8192, 2048), (5120, 20480), (1 << 21, 64)])
def test_fp32_adapters_ask_for_bounded_slices(M, N, K):
    """The K splits' slices: 64 MB at most where there is more than one, and one pass's rows, 256 MB at
    most (one tile's 64 rows at least); behind them 4 bytes a row and rank."""
    n, r = 8, 64
    got = zo.zo_op_linear_adapters_workspace(M, N, K, n, r, torch.float32)
    one = min(M, 64) * N * 4
    assert got <= M * r * 4 + max(256 * MB, one) + 1024
    assert got >= M * r * 4 + min(M * N * 4, 192 * MB)                   # whole tiles of rows


@pytest.mark.parametrize("M,N,K,splits", [(301, 2048, 2048, 8), (64, 4096, 4096, 2), (1000, 4096, 4096, 1),
                                          (4093, 20480, 5120, 1), (4096, 8192, 2048, 1)])
def test_fp32_adapters_split_only_where_rounds_are_few(M, N, K, splits):
    got = zo.zo_op_linear_adapters_workspace(M, N, K, 1, 1, torch.float32)
    rows = min(M, 256 * MB // 4 // N // 64 * 64)
    assert abs(got - splits * rows * N * 4 - M * 4) < 1024, got
