"""The operators for rounded layers against plain 64-bit implementations.

Tolerances, fixed before the kernels first ran:
  16-bit products: inputs are exact, products exact in fp32; a sum of R of them is
    off by at most (R + 8) 2^-23 sum |p q| (one truncation a step), and the output
    is rounded once (bf16 2^-8, fp16 2^-11 of |y|, fp16 also 2^-24; fp32 2^-23).
  fp8 products: the matrix cores' sums of fp8 products keep about 13 bits of the
    largest term: 2^-12 sum |s x w|, and the output's rounding.
  fp8 codes and scales: exact, from the same fp32 steps.
  log probabilities: 2^-20 (1 + |lse| + max |x|) for values (fp32 sums of e^d with
    d rounded once, error at most 2^-24 |d| each); tokens exact.
  gradients of log probabilities: p carries the relative error 2^-20 (1 + |x| + |lse|).
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

U = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -23}
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


@pytest.fixture(scope="module")
def bk():
    from two_sided_gptq_amd import bakron
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    bakron.load()
    return bakron


def gen(seed):
    return torch.Generator().manual_seed(seed)


def strided(t, pad, shift=0):
    """t on the GPU with rows `pad` elements further apart, `shift` elements into the storage."""
    *lead, n, k = t.shape
    count = int(np.prod(lead, dtype=int)) * n * (k + pad) + shift
    full = torch.zeros(count, dtype=t.dtype, device="cuda")
    strides = [1, k + pad]
    for d in reversed([*lead, n][1:]):
        strides.append(strides[-1] * d)
    v = full.as_strided(tuple(t.shape), tuple(reversed(strides)), shift)
    v.copy_(t)
    return v


# ---------------------------------------------------------------- fp8 quantisation

def e4m3_values():
    c = np.arange(127)
    e, m = c >> 3, c & 7
    return np.where(e > 0, (8.0 + m) * 2.0 ** (e - 10.0), m * 2.0 ** -9)


def e4m3_round(x):
    """Codes of |x| <= 448 (64-bit): nearest, ties to the even code."""
    v = e4m3_values()
    mid = (v[1:] + v[:-1]) / 2
    a = np.abs(x)
    lo = np.searchsorted(mid, a, side="left")
    tie = (lo < 126) & (a == mid[np.minimum(lo, 125)]) & (lo % 2 == 1)
    code = lo + tie
    return (code | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def quantize64(x, br):
    rows, cols = x.shape
    nb, kb = -(-rows // br), -(-cols // 128)
    full = np.zeros((nb * br, kb * 128), np.float32)
    full[:rows, :cols] = x
    amax = np.abs(full.reshape(nb, br, kb, 128)).max(axis=(1, 3))
    amax = np.where(amax > 0, np.maximum(amax, np.float32(2.0 ** -100)), np.float32(448))
    inv = (np.float32(448) / amax).astype(np.float32)
    y = (full.reshape(nb, br, kb, 128) * inv[:, None, :, None]).astype(np.float32)
    y = np.clip(y, -448, 448).reshape(nb * br, kb * 128)[:rows, :cols]
    return e4m3_round(y.astype(np.float64)), (amax / np.float32(448)).T


@pytest.mark.parametrize("rows,cols,dtype,br,pad,shift", [
    (1, 1, "f32", 1, 0, 0), (1, 14336, "bf16", 1, 0, 0), (5, 127, "f16", 1, 0, 0), (17, 128, "bf16", 1, 3, 1),
    (33, 129, "f32", 1, 1, 0), (300, 1000, "bf16", 1, 0, 0), (7, 4096, "f16", 1, 8, 0),
    (1, 1, "bf16", 128, 0, 0), (127, 129, "f32", 128, 0, 0), (128, 128, "bf16", 128, 5, 3),
    (257, 500, "f16", 128, 0, 0), (1024, 1024, "bf16", 128, 0, 0)])
def test_fp8_quantize(bk, rows, cols, dtype, br, pad, shift):
    x = torch.randn(rows, cols, generator=gen(rows * 31 + cols))
    x[:, ::97] *= 20
    if cols > 200:
        x[0, :128] = 0            # a block of zeros
        x[-1, 128:256] *= 1e-6
    x = x.to(DT[dtype])
    xd = strided(x, pad, shift)
    q, s = bk.fp8_quantize(xd, block_rows=br)
    qs = strided(torch.zeros(rows, cols, dtype=torch.uint8), 3, 1).view(torch.float8_e4m3fn)
    q2, s2 = bk.fp8_quantize(xd, block_rows=br, out=qs)
    want_q, want_s = quantize64(x.float().numpy(), br)
    assert np.array_equal(s.cpu().numpy(), want_s)
    assert np.array_equal(q.view(torch.uint8).cpu().numpy(), want_q)
    assert torch.equal(q2.contiguous().view(torch.uint8), q.view(torch.uint8)) and torch.equal(s, s2)


def test_fp8_quantize_limits(bk):
    """Blocks of the smallest and the largest values, and blocks that hold a NaN or an infinity."""
    x = torch.zeros(4, 512)
    x[0, :128] = 1e-44
    x[0, 128:256] = torch.linspace(-1, 1, 128) * 3.4e38
    x[1, 5] = float("inf")
    x[2, 200] = float("nan")
    x[3, 384:] = torch.linspace(-448, 448, 128)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    q, s = bk.fp8_quantize(x[[0, 3]].contiguous().cuda(), dev_status=status)
    want_q, want_s = quantize64(x[[0, 3]].numpy(), 1)
    assert int(status) == 0
    assert np.array_equal(s.cpu().numpy(), want_s) and np.array_equal(q.view(torch.uint8).cpu().numpy(), want_q)
    q, s = bk.fp8_quantize(x.cuda(), dev_status=status)
    assert int(status) == bk.DEV_NONFINITE
    bad = torch.zeros(4, 4, dtype=torch.bool)
    bad[0, 1] = bad[1, 2] = True                      # (block of columns, row)
    assert torch.equal(torch.isnan(s).cpu(), bad)
    assert torch.equal(torch.isnan(q.float()).cpu(), bad.t().repeat_interleave(128, 1))


@pytest.mark.parametrize("kind,bits,m,n,pad", [(0, 4, 65, 127, 0), (0, 2, 64, 64, 16), (1, 4, 200, 70, 1),
                                               (1, 2, 3, 300, 0), (0, 3, 1, 1, 0)])
def test_fp8_from_codes(bk, kind, bits, m, n, pad):
    g = gen(m + n)
    lo, hi = (-2 ** (bits - 1), 2 ** (bits - 1)) if kind == 0 else (0, 2 ** bits)
    codes = torch.randint(lo, hi, (m, n), generator=g, dtype=torch.int8)
    zeros = torch.randint(0, 2 ** bits, (m,), generator=g).float() if kind == 1 else None
    out = strided(torch.zeros(m, n, dtype=torch.uint8), pad).view(torch.float8_e4m3fn)
    q = bk.fp8_from_codes(codes.cuda(), None if zeros is None else zeros.cuda(), kind=kind, bits=bits, out=out)
    want = codes.double() - (zeros[:, None].double() if zeros is not None else 0)
    assert torch.equal(q.double().cpu(), want)


# ---------------------------------------------------------------- products

def offsets_of(counts):
    return torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32)


def counts_of(rows, groups, seed, skew=1.0):
    """Ragged counts with empty groups among them."""
    r = np.random.default_rng(seed)
    share = (1.0 + np.arange(groups)) ** -skew
    share[r.permutation(groups)[:groups // 4]] = 0
    share = r.permutation(share)
    return r.multinomial(rows, share / share.sum())


FP8_CASES = [
    # rows, n, k, groups, scale, out, pad of X and W
    (1, 1, 1, 1, "row", "bf16", 0), (1, 64, 128, 1, "block", "f16", 0), (3, 65, 127, 1, "row", "bf16", 0),
    (16, 200, 70, 1, "block", "bf16", 1), (17, 128, 256, 1, "row", "f16", 16), (33, 300, 1000, 1, "block", "bf16", 8),
    (65, 257, 513, 1, "row", "bf16", 0), (128, 128, 1024, 1, "block", "bf16", 0), (300, 1000, 400, 1, "block", "f16", 0),
    (515, 520, 528, 1, "row", "bf16", 16), (1, 1024, 4096, 1, "row", "bf16", 0), (1025, 1032, 272, 1, "block", "bf16", 0),
    (40, 96, 160, 8, "row", "bf16", 0), (333, 200, 144, 7, "block", "bf16", 0), (1000, 384, 512, 70, "row", "f16", 0),
    (64, 130, 77, 5, "block", "bf16", 3), (2500, 300, 256, 3, "row", "bf16", 0), (4200, 1100, 640, 2, "block", "bf16", 0),
    # enough tiles for the large ones
    (4100, 2120, 656, 3, "row", "bf16", 0), (4100, 2120, 912, 1, "block", "f16", 16), (4100, 2125, 144, 1, "block", "bf16", 0),
    # a little over one round of large tiles: the rest in small ones
    (4100, 4216, 272, 1, "block", "bf16", 0), (4100, 4200, 400, 3, "row", "f16", 8),
    # few rows: the form for single tokens, its widths and ends
    (1, 4096, 1040, 1, "block", "bf16", 0), (2, 40, 2500, 1, "row", "f16", 1), (20, 1000, 384, 1, "block", "bf16", 0),
    (50, 333, 640, 1, "row", "bf16", 0), (64, 512, 129, 1, "block", "f16", 0), (30, 272, 400, 16, "row", "bf16", 0),
    # and rows that begin off whole dwords
    (3, 200, 3077, 1, "row", "bf16", 0), (9, 130, 1500, 5, "block", "f16", 2), (1, 90, 2999, 1, "block", "bf16", 3),
    (150, 100, 256, 9, "block", "bf16", 0),
    # few tiles and a long reduction, which is split
    (40, 260, 4200, 1, "block", "bf16", 0), (130, 100, 6416, 1, "row", "f16", 0), (200, 130, 4112, 3, "block", "bf16", 0)]
SPLIT_CASES = [(40, 260, 4200, 1), (130, 100, 6416, 1), (200, 130, 4112, 3)]


def test_long_reductions_are_split(bk):
    """The cases above that stand for split reductions have a workspace, the others' sizes none."""
    for rows, n, k, groups in SPLIT_CASES:
        assert bk.load().bakron_fp8_matmul_workspace_size(rows, n, k, groups) > 0
    for rows, n, k, groups in ((300, 136, 2104, 3), (100, 2201, 130, 2), (6000, 130, 70, 2), (5000, 136, 72, 3)):
        assert bk.load().bakron_grouped_matmul_workspace_size(rows, n, k, groups) > 0
    assert bk.load().bakron_fp8_matmul_workspace_size(1, 4096, 4096, 1) == 0
    assert bk.load().bakron_fp8_matmul_workspace_size(8192, 4096, 4096, 1) == 0


@pytest.mark.parametrize("rows,n,k,groups,scale,out,pad", FP8_CASES)
def test_fp8_matmul(bk, rows, n, k, groups, scale, out, pad):
    g = gen(rows + 7 * n + 13 * k)
    kb, nb = -(-k // 128), -(-n // 128)
    lead = (groups,) if groups > 1 else ()
    x = torch.randn(rows, k, generator=g).mul_(100).clamp_(-448, 448).to(torch.float8_e4m3fn)
    w = torch.randn(*lead, n, k, generator=g).mul_(60).clamp_(-448, 448).to(torch.float8_e4m3fn)
    sx = torch.rand(kb, rows, generator=g) + 0.1
    sw = torch.rand(*lead, n, generator=g) + 0.1 if scale == "row" else torch.rand(*lead, kb, nb, generator=g) + 0.1
    counts = counts_of(rows, groups, rows) if groups > 1 else [rows]
    at = np.concatenate([[0], np.cumsum(counts)])
    col, row = torch.arange(k) // 128, torch.arange(n) // 128
    xs = x.double() * sx.double()[col].t()
    wd, sd = w.double().reshape(groups, n, k), sw.double().reshape(groups, *sw.shape[len(lead):])
    want, mass = torch.zeros(rows, n, dtype=torch.float64), torch.zeros(rows, n, dtype=torch.float64)
    for e in range(groups):
        ws = wd[e] * (sd[e][:, None] if scale == "row" else sd[e][col][:, row].t())
        want[at[e]:at[e + 1]] = xs[at[e]:at[e + 1]] @ ws.t()
        mass[at[e]:at[e + 1]] = xs[at[e]:at[e + 1]].abs() @ ws.abs().t()
    xd = strided(x.view(torch.uint8), pad).view(torch.float8_e4m3fn)
    wdv = strided(w.view(torch.uint8), pad).view(torch.float8_e4m3fn)
    off = offsets_of(counts).cuda() if groups > 1 else None
    scale_out = 1.0 if out == "bf16" else float(30000 / max(1.0, want.abs().max()))  # fp16's range
    sxd = (sx * scale_out).cuda()
    want, mass = want * scale_out, mass * scale_out
    y = bk.fp8_matmul(xd, sxd, wdv, sw.cuda(), offsets=off, out_dtype=DT[out])
    err = (y.double().cpu() - want).abs()
    tol = U[out] * want.abs() + 2.0 ** -12 * mass + 2.0 ** -24
    assert bool((err <= tol).all()), float((err / tol).max())
    y2 = bk.fp8_matmul(xd, sxd, wdv, sw.cuda(), offsets=off, out_dtype=DT[out])
    assert torch.equal(y, y2)


GROUPED_CASES = [
    # rows, n, k, groups, dtype, out, pad, shift
    (1, 1, 1, 1, "bf16", None, 0, 0), (1, 64, 64, 4, "f16", None, 0, 0), (2, 65, 127, 3, "bf16", "f32", 0, 0),
    (37, 130, 70, 5, "f16", "f32", 1, 1), (64, 256, 128, 64, "bf16", None, 0, 0), (100, 72, 200, 9, "bf16", None, 8, 8),
    (257, 264, 136, 2, "f16", None, 0, 0), (300, 520, 520, 24, "f16", None, 0, 0), (513, 128, 1000, 3, "bf16", "f32", 0, 0),
    (1000, 384, 256, 130, "bf16", None, 0, 0), (1500, 1000, 328, 4, "bf16", None, 0, 0), (2050, 301, 259, 3, "f16", None, 0, 0),
    (4300, 560, 328, 3, "bf16", "f32", 8, 0),
    # enough tiles for the large ones: forward, gradient of X, gradient of W
    (4100, 2120, 328, 3, "bf16", None, 0, 0), (4100, 328, 2120, 2, "f16", "f32", 8, 8), (700, 2056, 1416, 3, "bf16", None, 0, 0),
    (4100, 2128, 264, 1, "f16", "f32", 0, 0),
    # a little over one round of large tiles, the rest in small ones: forward, gradient of X, gradient of W
    (4100, 4216, 200, 3, "bf16", None, 0, 0), (4100, 200, 4216, 1, "f16", None, 0, 0), (4100, 136, 4300, 2, "bf16", "f32", 0, 0),
    (400, 2616, 2632, 3, "bf16", None, 0, 0),
    # few rows
    (1, 300, 1000, 1, "bf16", None, 0, 0), (2, 33, 2050, 1, "f16", "f32", 1, 1), (60, 1000, 200, 1, "bf16", None, 0, 0),
    (3, 130, 3077, 1, "bf16", None, 0, 1), (40, 70, 1111, 20, "f16", None, 2, 3), (1, 48, 2304, 1, "bf16", "f32", 1, 0),
    (90, 130, 520, 7, "bf16", "f32", 0, 0), (33, 272, 264, 40, "f16", None, 0, 0),
    # few tiles and a long reduction, which is split: forward, gradients
    (300, 136, 2104, 3, "bf16", None, 0, 0), (100, 2201, 130, 2, "f16", "f32", 0, 0), (6000, 130, 70, 2, "bf16", "f32", 0, 0),
    (5000, 136, 72, 3, "f16", None, 0, 0)]


def product_inputs(rows, n, k, groups, dtype, seed):
    g = gen(seed)
    x = torch.randn(rows, k, generator=g).to(DT[dtype])
    w = torch.randn(groups, n, k, generator=g).mul_(0.05).to(DT[dtype])
    dy = torch.randn(rows, n, generator=g).mul_(0.1).to(DT[dtype])
    counts = counts_of(rows, groups, seed) if groups > 1 else [rows]
    return x, w, dy, counts, np.concatenate([[0], np.cumsum(counts)])


def within(y, want, mass, r, out):
    err = (y.double().cpu() - want).abs()
    tol = U[out] * want.abs() + (r + 8) * 2.0 ** -23 * mass + 2.0 ** -24
    assert bool((err <= tol).all()), float((err / tol).max())


@pytest.mark.parametrize("rows,n,k,groups,dtype,out,pad,shift", GROUPED_CASES)
def test_grouped_matmul(bk, rows, n, k, groups, dtype, out, pad, shift):
    x, w, dy, counts, at = product_inputs(rows, n, k, groups, dtype, rows + n + k)
    xd, wd = strided(x, pad, shift), strided(w, pad, shift)
    off = offsets_of(counts).cuda() if groups > 1 else None
    y = bk.grouped_matmul(xd, wd, off, out_dtype=DT[out] if out else None)
    want, mass = torch.zeros(rows, n, dtype=torch.float64), torch.zeros(rows, n, dtype=torch.float64)
    for e in range(groups):
        a, b = at[e], at[e + 1]
        want[a:b] = x[a:b].double() @ w[e].double().t()
        mass[a:b] = x[a:b].double().abs() @ w[e].double().abs().t()
    within(y, want, mass, k, out or dtype)
    assert torch.equal(y, bk.grouped_matmul(xd, wd, off, out_dtype=DT[out] if out else None))


@pytest.mark.parametrize("rows,n,k,groups,dtype,out,pad,shift", GROUPED_CASES)
def test_grouped_matmul_grad(bk, rows, n, k, groups, dtype, out, pad, shift):
    x, w, dy, counts, at = product_inputs(rows, n, k, groups, dtype, rows + n + k)
    xd, wd, dyd = strided(x, pad, shift), strided(w, pad, shift), strided(dy, pad, shift)
    off = offsets_of(counts).cuda() if groups > 1 else None
    dx, dw = bk.grouped_matmul_grad(dyd, xd, wd, off, w_dtype=DT[out] if out else None)
    X, W, G = x.double(), w.double(), dy.double()
    want, mass = torch.zeros_like(X), torch.zeros_like(X)
    for e in range(groups):
        a, b = at[e], at[e + 1]
        want[a:b], mass[a:b] = G[a:b] @ W[e], G[a:b].abs() @ W[e].abs()
    within(dx, want, mass, n, dtype)
    wantw, massw = torch.zeros_like(W), torch.zeros_like(W)
    for e in range(groups):
        a, b = at[e], at[e + 1]
        wantw[e], massw[e] = G[a:b].t() @ X[a:b], G[a:b].abs().t() @ X[a:b].abs()
    within(dw, wantw, massw, rows, out or dtype)
    # against differences of the loss sum(dY Y(X, W)) in 64 bits, along random directions
    g, eps = gen(5), 1e-4
    U1, U2 = torch.randn(X.shape, generator=g, dtype=torch.float64), torch.randn(W.shape, generator=g, dtype=torch.float64)

    def loss(X, W):
        return sum(float((G[at[e]:at[e + 1]] * (X[at[e]:at[e + 1]] @ W[e].t())).sum()) for e in range(groups))

    for d, u, v, m, r, o in ((dx, U1, lambda t: (X + t * U1, W), mass, n, dtype),
                             (dw, U2, lambda t: (X, W + t * U2), massw, rows, out or dtype)):
        slope = (loss(*v(eps)) - loss(*v(-eps))) / (2 * eps)
        got = float((d.double().cpu() * u).sum())
        tol = float(((U[o] * d.double().cpu().abs() + (r + 8) * 2.0 ** -23 * m + 2.0 ** -24) * u.abs()).sum())
        tol += 1e-9 * float((m * u.abs()).sum()) / eps  # the differences' own rounding
        assert abs(got - slope) <= tol, (got, slope, tol)


def test_rows_of_no_group_and_bad_offsets(bk):
    """Rows after the last group get 0; offsets that fall or leave the rows are
    reported, and write nothing outside the output."""
    x, w, dy, _, _ = product_inputs(300, 96, 64, 3, "bf16", 1)
    off = torch.tensor([0, 100, 100, 180], dtype=torch.int32, device="cuda")
    full = torch.full((302, 96), 7.0, dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = bk.grouped_matmul(x.cuda(), w.cuda(), off, out=full[1:301], dev_status=status)
    assert int(status) == 0 and bool((y[180:] == 0).all()) and bool((y[:180].abs().sum(1) > 0).all())
    dx, dw = bk.grouped_matmul_grad(dy.cuda(), x.cuda(), w.cuda(), off, dev_status=status)
    assert bool((dx[180:] == 0).all()) and bool((dw[1] == 0).all()) and int(status) == 0
    for bad in ([0, 200, 100, 300], [0, 100, 200, 400], [-5, 0, 100, 300], [3, 5, 100, 300]):
        status.zero_()
        off = torch.tensor(bad, dtype=torch.int32, device="cuda")
        bk.grouped_matmul(x.cuda(), w.cuda(), off, out=full[1:301], dev_status=status)
        assert int(status) == bk.DEV_BAD_INDEX, bad
        assert bool((full[0] == 7).all()) and bool((full[301] == 7).all())


def test_non_finite_stays_in_its_row(bk):
    x, w, dy, counts, at = product_inputs(300, 200, 136, 3, "bf16", 9)
    off = offsets_of(counts).cuda()
    x[7, 3], x[100, 5] = float("nan"), float("inf")
    y = bk.grouped_matmul(x.cuda(), w.cuda(), off).float().cpu()
    fine = torch.ones(300, dtype=torch.bool)
    fine[[7, 100]] = False
    assert bool(torch.isfinite(y[fine]).all()) and not bool(torch.isfinite(y[~fine]).any())


# ---------------------------------------------------------------- token log probabilities

def logits_of(rows, vocab, dtype, seed, masked):
    g = gen(seed)
    x = torch.randn(rows, vocab, generator=g).mul_(3)
    x[torch.arange(rows), torch.randint(0, vocab, (rows,), generator=g)] += 8
    x = x.to(DT[dtype])
    t = torch.randint(0, vocab, (rows,), generator=g)
    if masked:
        low = torch.finfo(DT[dtype]).min
        x[0] = -torch.inf                              # nothing left
        if rows > 1:
            x[1] = low                                 # uniform
        if rows > 2:
            x[2, : vocab - 1] = -torch.inf             # one token left
            t[2] = vocab - 1
        if rows > 3:
            x[3, ::2] = low
            t[3] = min(1, vocab - 1)
        if rows > 4:
            x[4] = 1.5                                 # all equal
        if rows > 5:
            t[5] = -100
    return x, t


def stats64(x):
    x = x.double()
    m = x.amax(1, keepdim=True)
    none = torch.isinf(m)
    d = torch.where(none, -torch.inf, x - torch.where(none, 0, m))
    e = d.exp()
    s = e.sum(1, keepdim=True)
    lse = torch.where(none, -torch.inf, m + s.log())
    ent = torch.where(none, 0, s.log() - torch.where(e > 0, e * d, 0).sum(1, keepdim=True) / s)
    return lse[:, 0], ent[:, 0]


def near(got, want, tol):
    got, want = got.double().cpu(), want.double()
    inf = torch.isinf(want)
    assert torch.equal(torch.isinf(got), inf) and torch.equal(got[inf], want[inf])
    err = (got - want).abs()[~inf]
    tol = tol.expand_as(want)[~inf]
    assert bool((err <= tol).all()), float((err / tol).max())


LOGIT_CASES = [
    (1, 1, "f32", 1, False), (3, 2, "bf16", 2, True), (7, 17, "f16", 5, True), (5, 100, "f32", 64, True),
    (9, 1000, "bf16", 20, True), (1, 5000, "f32", 0, False), (6, 8192, "bf16", 64, True), (2, 32768, "f16", 7, True),
    (8, 100003, "bf16", 20, True), (4, 131072, "f32", 64, True), (3, 200001, "bf16", 1, True), (600, 1027, "f32", 5, True),
    (700, 131073, "bf16", 20, True), (1, 2 ** 21, "bf16", 64, False)]


@pytest.mark.parametrize("rows,vocab,dtype,k,masked", LOGIT_CASES)
def test_token_logprobs(bk, rows, vocab, dtype, k, masked):
    x, t = logits_of(rows, vocab, dtype, rows + vocab, masked)
    for pad, shift in ((0, 0), (3, 1)):
        if pad and rows * vocab > 1 << 24:
            continue
        out = bk.token_logprobs(strided(x, pad, shift), t.cuda(), top=k)
        lse, ent = stats64(x)
        fin = torch.where(torch.isinf(lse), 0, lse)
        mag = torch.where(torch.isinf(x.float()), 0, x.float()).abs()
        mag = torch.where(mag > 1e30, 0, mag).amax(1).double()
        tol = 2.0 ** -20 * (1 + torch.where(fin.abs() > 1e30, fin.abs(), fin.abs() + mag))
        near(out["lse"], lse, tol)
        near(out["entropy"], ent, 2.0 ** -20 * (1 + mag + ent.abs()))
        xt = x.double().gather(1, t.clamp(min=0)[:, None])[:, 0]
        lp = torch.where(t < 0, 0.0, torch.where(torch.isinf(lse), -torch.inf, xt - lse))
        near(out["logprob"], lp, tol)
        if k == 0:
            assert out["top_ids"] is None
            continue
        v, i = torch.sort(x.double(), dim=1, descending=True, stable=True)
        assert torch.equal(out["top_ids"].cpu(), i[:, :k])
        want = torch.where(torch.isinf(lse)[:, None], -torch.inf, v[:, :k] - lse[:, None])
        near(out["top_logprob"], want, torch.where(want.abs() > 1e30, want.abs() * 2.0 ** -20, tol[:, None]))


def test_token_logprobs_ties_and_orders(bk):
    """Rows whose chunks all reach the bound (more candidates than are held at
    once), rising and falling rows, both zeros, few distinct values."""
    vocab, k = 65536, 64
    rows = [torch.arange(vocab).float(), -torch.arange(vocab).float(), torch.zeros(vocab),
            torch.where(torch.arange(vocab) % 3 == 0, -0.0, 0.0), (torch.arange(vocab) % 7).float(),
            torch.where(torch.arange(vocab) // 16 % 8 == 0, 5.0, 1.0), torch.full((vocab,), -torch.inf)]
    # one group of 8 threads holds all large chunks, all of them tied with others far off
    r = torch.zeros(vocab)
    c = torch.arange(vocab) // 16
    r[(c % 512) < 200] = 3.0
    rows.append(r)
    for dtype in ("f32", "bf16"):
        x = torch.stack(rows).to(DT[dtype])
        t = torch.zeros(len(rows), dtype=torch.int64)
        v, i = torch.sort(x.double(), dim=1, descending=True, stable=True)
        for kk in (1, 20, k):
            out = bk.token_logprobs(x.cuda(), t.cuda(), top=kk)
            assert torch.equal(out["top_ids"].cpu(), i[:, :kk]), (dtype, kk)
        # the same rows, one workgroup each
        y = x.repeat(80, 1)
        out = bk.token_logprobs(y.cuda(), torch.zeros(len(y), dtype=torch.int64, device="cuda"), top=k)
        assert torch.equal(out["top_ids"].cpu(), i[:, :k].repeat(80, 1))


def test_token_logprobs_non_finite(bk):
    x = torch.randn(5, 3000, generator=gen(3))
    x[1, 77], x[2, 2999], x[3, 5] = float("nan"), float("inf"), float("nan")
    t = torch.tensor([0, 1, 2, 3, 4])
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = bk.token_logprobs(x.cuda(), t.cuda(), top=4, dev_status=status)
    assert int(status) == bk.DEV_NONFINITE
    bad = torch.tensor([False, True, True, True, False])
    for name in ("logprob", "lse", "entropy"):
        assert torch.equal(torch.isnan(out[name]).cpu(), bad)
    assert bool(((out["top_ids"] >= 0) & (out["top_ids"] < 3000)).all())
    status.zero_()
    t[0] = 3000
    out = bk.token_logprobs(x[:1].cuda(), t[:1].cuda(), dev_status=status)
    assert int(status) == bk.DEV_BAD_INDEX and bool(torch.isnan(out["logprob"][0])) and bool(torch.isfinite(out["lse"][0]))


@pytest.mark.parametrize("rows,vocab,dtype,masked", [(1, 1, "f32", False), (6, 17, "f32", True), (7, 1000, "bf16", True),
                                                     (9, 8193, "f16", True), (600, 3001, "bf16", True),
                                                     (6, 100003, "f32", True)])
@pytest.mark.parametrize("entropy", [False, True])
def test_token_logprobs_grad(bk, rows, vocab, dtype, masked, entropy):
    x, t = logits_of(rows, vocab, dtype, 3 * rows + vocab, masked)
    g, gh = torch.randn(rows, generator=gen(1)), torch.randn(rows, generator=gen(2))
    for pad, shift in ((0, 0), (3, 1)):
        xd = strided(x, pad, shift)
        f = bk.token_logprobs(xd, t.cuda())
        d = bk.token_logprobs_grad(xd, t.cuda(), f["lse"], f["entropy"] if entropy else None, g.cuda(),
                                   gh.cuda() if entropy else None)
        lse, ent = stats64(x)
        none = torch.isinf(lse)
        lp = x.double() - torch.where(none, 0, lse)[:, None]
        p = torch.where(none[:, None], 0, lp.exp())
        hit = torch.zeros_like(p)
        hit[torch.arange(rows)[t >= 0], t[t >= 0]] = 1
        gd = torch.where((t >= 0) & ~none, g.double(), 0)[:, None]
        hd = gh.double()[:, None] if entropy else torch.zeros(rows, 1, dtype=torch.float64)
        plp = torch.where(p > 0, p * (lp + ent[:, None]), 0)
        want = gd * (hit - p) - hd * plp
        rel = 2.0 ** -20 * (1 + torch.where(p > 0, x.double().abs() + torch.where(none, 0, lse).abs()[:, None], 0))
        rel = torch.where(p > 1e-38, rel.clamp(max=1), 0)
        tol = U[dtype] * want.abs() + rel * p * (gd.abs() + hd.abs() * (2 + lp.abs().clamp(max=200) + ent[:, None])) + 2.0 ** -24
        err = (d.double().cpu() - want).abs()
        assert bool((err <= tol).all()), float((err / tol).max())


def test_token_logprobs_grad_against_differences(bk):
    """The fp32 gradient against central differences of the 64-bit scores."""
    rows, vocab = 4, 50
    x, t = logits_of(rows, vocab, "f32", 11, False)
    g, gh = torch.randn(rows, generator=gen(1)).double(), torch.randn(rows, generator=gen(2)).double()
    f = bk.token_logprobs(x.cuda(), t.cuda())
    d = bk.token_logprobs_grad(x.cuda(), t.cuda(), f["lse"], f["entropy"], g.float().cuda(), gh.float().cuda())

    def score(x):
        lse, ent = stats64(x)
        return float((g * (x.gather(1, t[:, None])[:, 0] - lse) + gh * ent).sum())

    eps = 1e-5
    for r in range(rows):
        for j in range(vocab):
            e = torch.zeros(rows, vocab, dtype=torch.float64)
            e[r, j] = eps
            slope = (score(x.double() + e) - score(x.double() - e)) / (2 * eps)
            assert abs(float(d[r, j]) - slope) <= 1e-5 * (1 + abs(slope)) * 4


# ---------------------------------------------------------------- streams, graphs

def test_other_stream_and_graph(bk):
    """Every operator on a stream that is not torch's current one, then captured
    into a graph and replayed with eager work between; all results equal."""
    x, w, dy, counts, _ = product_inputs(300, 264, 256, 4, "bf16", 21)
    x, w, dy, off = x.cuda(), w.cuda(), dy.cuda(), offsets_of(counts).cuda()
    logits, t = logits_of(6, 40000, "bf16", 4, True)
    logits, t = logits.cuda(), t.cuda()
    g = torch.randn(6, device="cuda")

    def all_of(stream=None):
        q, s = bk.fp8_quantize(x, stream=stream)
        qw, sw = bk.fp8_quantize(w.view(-1, 256), block_rows=128, stream=stream)
        y8 = bk.fp8_matmul(q, s, qw[:264], sw[:, :3].contiguous() if stream is None else sw_first, stream=stream)
        y = bk.grouped_matmul(x, w, off, stream=stream)
        dx, dw = bk.grouped_matmul_grad(dy, x, w, off, stream=stream)
        f = bk.token_logprobs(logits, t, top=20, stream=stream)
        d = bk.token_logprobs_grad(logits, t, f["lse"], f["entropy"], g, g, stream=stream)
        return [q.view(torch.uint8), s, y8, y, dx, dw, *f.values(), d]

    _, sw_all = bk.fp8_quantize(w.view(-1, 256), block_rows=128)
    sw_first = sw_all[:, :3].contiguous()
    want = [v.clone() for v in all_of()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = all_of(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    same = lambda a, b: torch.equal(torch.nan_to_num(a.float(), nan=1e9), torch.nan_to_num(b.float(), nan=1e9))
    assert all(same(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        all_of()
    torch.cuda.current_stream().wait_stream(side)
    with torch.cuda.graph(graph):
        kept = all_of()
    for _ in range(3):
        for v in kept:
            v.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(same(a, b) for a, b in zip(want, kept))
        assert all(same(a, b) for a, b in zip(want, all_of()))


# ---------------------------------------------------------------- together

@pytest.mark.parametrize("kind,bits", [(0, 4), (1, 3)])
def test_rounded_experts(bk, kind, bits):
    """The example: experts rounded, multiplied in fp8 and scored.  The fp8 weights are
    the solve's V exactly, the product is theirs with the activations as quantised,
    and the scores are those of the logits."""
    from two_sided_gptq_amd import experts
    X, W, head, offsets, targets = experts.example(experts=4, tokens=500, width=192, vocab=1000)
    r = experts.round_experts(X, W, head, offsets, targets, kind=kind, bits=bits)
    assert int(r["status"]) == 0
    at = offsets.tolist()
    assert at[-1] == 500 and at[-2] == 500  # the last expert has no tokens
    Vd = r["W8"].double() * r["scales"].double()[:, :, None]
    err = (Vd - r["V"].double()).abs()
    assert bool((err <= 2.0 ** -23 * Vd.abs()).all())
    col = torch.arange(192, device="cuda") // 128
    Xd = r["X8"].double() * r["sx"].double()[col].t()
    for e in range(4):
        a, b = at[e], at[e + 1]
        want, mass = Xd[a:b] @ Vd[e].t(), Xd[a:b].abs() @ Vd[e].abs().t()
        assert bool(((r["Y8"][a:b].double() - want).abs() <= U["bf16"] * want.abs() + 2.0 ** -12 * mass).all())
    # rounding to 4 bits costs little of the scores, to 3 more, and both change them
    loss = float((r["before"]["logprob"] - r["after"]["logprob"]).mean())
    assert loss != 0.0 and abs(loss) < (0.5 if bits == 4 else 2.0), loss
