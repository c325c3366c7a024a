"""Offsets that fall, overlap or leave the rows, in every form of the products: they are
reported and nothing outside the output and the workspace is written.  The calls go
through the C ABI with a workspace of exactly the size that it asks for, in the middle of
a larger buffer of known bytes, and an output with known rows around it.

Tolerances, fixed before the first run, for good offsets: one rounding of the output to
bf16 (2^-8 of the value) and sums in fp32 ((R + 8) 2^-23 of the sum of magnitudes; fp8
products 2^-12 of it)."""
import ctypes

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

GUARD = 0x5a
BEHIND = 48 << 20  # more than all tiles of the overlapping groups below would need
P = ctypes.c_void_p


@pytest.fixture(scope="module")
def bk():
    from two_sided_gptq_amd import bakron
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    bakron.load()
    return bakron


def bad_offsets(groups, rows):
    """All rows again and again, back to front, and beyond both ends."""
    over = [0 if g % 2 == 0 else rows for g in range(groups + 1)]
    back = [rows - rows * g // groups for g in range(groups + 1)]
    wild = [(-1) ** g * (rows + 7 * g) for g in range(groups + 1)]
    far = [(2 ** 31 - 1 if g % 2 else -2 ** 31) for g in range(groups + 1)]
    return over, back, wild, far


# form, rows, N, K, groups: reductions that are split, large tiles with a tail, few rows,
# rows off 16 bytes, and small tiles
SHAPES = [("split", 1500, 256, 4096, 5), ("large", 4100, 4216, 264, 3), ("few", 40, 200, 512, 12),
          ("odd", 700, 301, 259, 6), ("small", 600, 520, 128, 9)]


@pytest.mark.parametrize("form,rows,N,K,groups", SHAPES, ids=[s[0] for s in SHAPES])
@pytest.mark.parametrize("call", ["forward", "grad_x", "grad_w", "fp8 row", "fp8 block"])
def test_bad_offsets_stay_inside(bk, call, form, rows, N, K, groups):
    lib = bk.load()
    if call == "grad_x":
        N, K = K, N  # the reduction runs over N
    fp8 = call.startswith("fp8")
    g = torch.Generator().manual_seed(rows + N + K)
    size = lib.bakron_fp8_matmul_workspace_size if fp8 else lib.bakron_grouped_matmul_workspace_size
    need = size(rows, N, K, groups)
    if form == "split":
        assert need > 0
    if fp8:
        A = torch.randint(0, 120, (rows, K), generator=g, dtype=torch.uint8).cuda()
        B = torch.randint(0, 120, (groups, N, K), generator=g, dtype=torch.uint8).cuda()
        kb, nb = -(-K // 128), -(-N // 128)
        sx = torch.ones(kb, rows, device="cuda")
        sw = torch.ones(groups, N, device="cuda") if call == "fp8 row" else torch.ones(groups, kb, nb, device="cuda")
        shape = (rows, N)
    else:
        left, right = {"forward": ((rows, K), (groups, N, K)), "grad_x": ((rows, N), (groups, N, K)),
                       "grad_w": ((rows, N), (rows, K))}[call]
        A = torch.randn(left, generator=g).bfloat16().cuda()
        B = torch.randn(right, generator=g).bfloat16().cuda()
        shape = {"forward": (rows, N), "grad_x": (rows, K), "grad_w": (groups * N, K)}[call]
    around = torch.full((shape[0] + 256, shape[1]), 7.0, dtype=torch.bfloat16, device="cuda")
    Y = around[128:-128]
    space = torch.full((need + BEHIND,), GUARD, dtype=torch.uint8, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def run(offsets):
        off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
        tail = (rows, N, K, groups, P(off.data_ptr()), P(Y.data_ptr()), bk.T_BF16, shape[1], P(status.data_ptr()),
                P(space.data_ptr()), need, P(torch.cuda.current_stream().cuda_stream))
        if fp8:
            rc = lib.bakron_fp8_matmul(P(A.data_ptr()), K, P(sx.data_ptr()), P(B.data_ptr()), K, P(sw.data_ptr()),
                                       bk.SCALE_ROW if call == "fp8 row" else bk.SCALE_BLOCK, *tail)
        else:
            name = "bakron_grouped_matmul" + {"forward": "", "grad_x": "_grad_x", "grad_w": "_grad_w"}[call]
            rc = getattr(lib, name)(P(A.data_ptr()), bk.T_BF16, A.shape[-1], P(B.data_ptr()), B.shape[-1], *tail)
        assert rc == 0, lib.bakron_last_error()
        torch.cuda.synchronize()
        assert bool((space[need:] == GUARD).all()), offsets
        assert bool((around[:128] == 7).all()) and bool((around[-128:] == 7).all()), offsets

    for bad in bad_offsets(groups, rows):
        status.zero_()
        run(bad)
        assert int(status) == bk.DEV_BAD_INDEX, bad
    # and good ones are right afterwards
    status.zero_()
    at = np.linspace(0, rows, groups + 1).astype(int).tolist()
    run(at)
    assert int(status) == 0
    a, b = (t.view(torch.float8_e4m3fn).double().cpu() if fp8 else t.double().cpu() for t in (A, B))
    form = {"grad_x": lambda x, w: x @ w, "grad_w": lambda x, w: x.T @ w}.get(call, lambda x, w: x @ w.T)
    length = {"grad_x": N, "grad_w": rows}.get(call, K)
    share = 2.0 ** -12 if fp8 else (length + 8) * 2.0 ** -23
    for e in range(groups):
        x, w = a[at[e]:at[e + 1]], b[at[e]:at[e + 1]] if call == "grad_w" else b[e]
        want, mass = form(x, w), form(x.abs(), w.abs())
        got = Y[e * N:(e + 1) * N] if call == "grad_w" else Y[at[e]:at[e + 1]]
        assert bool(((got.double().cpu() - want).abs() <= 2.0 ** -8 * want.abs() + share * mass + 2.0 ** -24).all()), e


@pytest.mark.parametrize("form,rows,N,K,groups", SHAPES, ids=[s[0] for s in SHAPES])
@pytest.mark.parametrize("call", ["forward", "grad_x", "fp8 row", "fp8 block"])
@pytest.mark.parametrize("left", [1, 0.6])
def test_rows_of_no_group(bk, call, form, rows, N, K, groups, left):
    """Rows after the last group's get 0, in every form; the others are as without them."""
    if call == "grad_x":
        N, K = K, N
    rest = 1 if left == 1 else int(rows * left)
    g = torch.Generator().manual_seed(rows + N * K)
    at = np.linspace(0, rows - rest, groups + 1).astype(int)
    at[1] = at[2] if groups > 2 else at[1]  # an empty group
    off = torch.tensor(at, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    w = torch.randn(groups, N, K, generator=g).mul_(0.1).bfloat16().cuda()
    x = torch.randn(rows, N if call == "grad_x" else K, generator=g).bfloat16().cuda()
    Y = torch.full((rows, K if call == "grad_x" else N), 7.0, dtype=torch.bfloat16, device="cuda")
    a, b = x.double().cpu(), w.double().cpu()
    if call == "forward":
        bk.grouped_matmul(x, w, off, out=Y, dev_status=status)
    elif call == "grad_x":
        Y, _ = bk.grouped_matmul_grad(x, Y, w, off, want_w=False, dev_status=status)
    else:
        x8, sx = bk.fp8_quantize(x)
        w8, sw = bk.fp8_quantize(w.view(-1, K))
        w8 = w8.view(groups, N, K)
        if call == "fp8 row":
            sw = torch.rand(groups, N, generator=g).add_(0.5).cuda()
            scale = sw.double().cpu()[..., None]
        else:
            sw = torch.rand(groups, -(-K // 128), -(-N // 128), generator=g).add_(0.5).cuda()
            scale = sw.double().cpu().transpose(1, 2).repeat_interleave(128, 1).repeat_interleave(128, 2)[:, :N, :K]
        bk.fp8_matmul(x8, sx, w8, sw, off, out=Y, dev_status=status)
        a = x8.double().cpu() * sx.double().cpu().t().repeat_interleave(128, 1)[:, :K]
        b = w8.double().cpu() * scale
    assert int(status) == 0
    y = Y.double().cpu()
    assert bool((y[rows - rest:] == 0).all())
    length = N if call == "grad_x" else K
    share = 2.0 ** -12 if call.startswith("fp8") else (length + 8) * 2.0 ** -23
    for e in range(groups):
        v, m = a[at[e]:at[e + 1]], b[e] if call == "grad_x" else b[e].T
        want, mass = v @ m, v.abs() @ m.abs()
        assert bool(((y[at[e]:at[e + 1]] - want).abs() <= 2.0 ** -8 * want.abs() + share * mass + 2.0 ** -24).all()), e
