"""Products whose launches would need 2^32 threads or more are refused before any device
is touched; a little below they are not."""
import ctypes
import os

import pytest

from two_sided_gptq_amd import bakron

F = ctypes.c_void_p(4096)
GROUPS = 4096


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(bakron.LIB_PATH):
        from two_sided_gptq_amd import build
        build.build()
    return bakron.load()


def run(lib, name, rows, N, K, less=0):
    lda, ldb, ldy = {"_grad_x": (N, K, K), "_grad_w": (N, K, K)}.get(name, (K, K, N))
    if name == "fp8":
        return lib.bakron_fp8_matmul(F, lda - less, F, F, ldb, F, 0, rows, N, K, GROUPS, F, F, 1, ldy, None, F, 1 << 40, None)
    call = getattr(lib, "bakron_grouped_matmul" + name)
    return call(F, 1, lda - less, F, ldb, rows, N, K, GROUPS, F, F, 1, ldy, None, F, 1 << 40, None)


# Workgroups of 256 threads: one for 64 rows of W and each of 4096 groups, the rows
# after them and the 16 rows' own tile (few rows: 4098 row tiles); tiles of 128 x 128
# otherwise, with a row tile for each group beside the rows' own.
REFUSED = [("fp8", 1, 1 << 18, 16), ("", 1, 1 << 18, 16), ("_grad_x", 1, 16, 1 << 19), ("_grad_w", 1, 1 << 18, 1 << 9),
           ("", 1 << 20, 1 << 18, 16)]


@pytest.mark.parametrize("name,rows,N,K", REFUSED)
def test_launches_beyond_the_limit(lib, name, rows, N, K):
    assert run(lib, name, rows, N, K) == 1
    assert b"too many tiles" in lib.bakron_last_error()


# A row stride that is too small ends these calls after the sizes have been accepted.
@pytest.mark.parametrize("name,rows,N,K", [("fp8", 1, (1 << 18) - 1024, 16), ("", 1, (1 << 18) - 1024, 16),
                                           ("_grad_x", 1, 16, (1 << 19) - 4096), ("_grad_w", 1, 1 << 18, 128)])
def test_launches_within_the_limit(lib, name, rows, N, K):
    assert run(lib, name, rows, N, K, less=1) == 1
    assert b"bad row stride" in lib.bakron_last_error()
