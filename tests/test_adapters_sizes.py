"""Sizes of the adapters' calls, checked before any device is touched: each direction refuses what
its own launches cannot take."""
import ctypes
import os

import pytest

from two_sided_gptq_amd import bakron

F = ctypes.c_void_p(4096)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(bakron.LIB_PATH):
        from two_sided_gptq_amd import build
        build.build()
    return bakron.load()


# rows, N, K, groups whose forward launch has less than 2^32 threads, and whose sums over places have more
FORWARD_ONLY = [(600000, 1 << 18, 64, 4096), (530000, 300000, 128, 4096), (140000, 1 << 20, 64, 1024), (600000, 64, 1 << 18, 4096)]


@pytest.mark.parametrize("rows,N,K,groups", FORWARD_ONLY)
def test_forward_is_not_held_to_the_gradients_launches(lib, rows, N, K, groups):
    assert (rows // 64 + 1 + groups + 1) * -(-max(N, K) // 256) * 256 < 1 << 32 <= groups * max(N, K) * 4
    assert lib.bakron_adapter_matmul_workspace_size(rows, N, K, 1, groups) > 0
    rc = lib.bakron_adapter_matmul(F, 1, K, F, F, rows, N, K, 1, groups, F, None, None, None, 0, F, 1, N, None, None, 0, None)
    assert rc == 2 and b"workspace" in lib.bakron_last_error()  # nothing but the missing workspace
    assert lib.bakron_adapter_matmul_grad_workspace_size(rows, N, K, 1, groups) == 0
    rc = lib.bakron_adapter_matmul_grad(F, N, F, 1, K, F, F, rows, N, K, 1, groups, F, None, None, None, 0, F, 1, K, F, F, 0,
                                        None, F, 1 << 60, None)
    assert rc == 1 and b"too many tiles" in lib.bakron_last_error()


@pytest.mark.parametrize("rows,N,K,groups", [(1 << 24, 1 << 14, 64, 4096), (16, 1 << 20, 64, 4096), (16, 64, 1 << 20, 4096)])
def test_forward_refuses_what_its_own_launch_cannot_take(lib, rows, N, K, groups):
    high = 64 if rows >= 64 * (groups + 1) else 16
    assert (-(-rows // high) + groups + 1) * -(-max(N, K) // 256) * 256 >= 1 << 32
    assert lib.bakron_adapter_matmul_workspace_size(rows, N, K, 1, groups) == 0
    rc = lib.bakron_adapter_matmul(F, 1, K, F, F, rows, N, K, 1, groups, F, None, None, None, 0, F, 1, N, None, F, 1 << 60, None)
    assert rc == 1 and b"too many tiles" in lib.bakron_last_error()
