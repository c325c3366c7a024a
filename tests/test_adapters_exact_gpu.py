"""Results of the adapters in fp32, exactly.

All values are whole numbers, of up to 7 bits in the inputs and so few or so sparse that every sum
of magnitudes stays below 2^24.  Then P, U and the results are whole numbers that fp32 holds, and
so are all partial sums in any order; the products that the matrix cores add are exact.  There
is no rounding anywhere, so results have to be equal.  P and U go beyond 2^17: kept with
16 bits they would not be.
"""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module")
def bk():
    from two_sided_gptq_amd import bakron
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    bakron.load()
    return bakron


class Whole:
    """rows, N, K, rank, adapters; which of the matrices are dense, the others have +-1 in a few places."""

    def __init__(self, rows, N, K, rank, groups, dense, seed, high=63):
        g = torch.Generator().manual_seed(seed)

        def values(name, *shape):
            if name in dense:
                return torch.randint(0, high + 1, shape, generator=g).double()
            # at most one in a row and in a column, or one in a row of few columns
            t = torch.zeros(shape, dtype=torch.float64).view(-1, *shape[-2:])
            for m in t:
                n, k = m.shape
                at = torch.randperm(max(n, k), generator=g)[:n] % k if name in ("A", "B") else torch.arange(n) % k
                some = torch.arange(n) if name in ("A", "B") else torch.randperm(n, generator=g)[:max(1, min(n, k) // 2)]
                m[some, at[some]] = torch.randint(0, 2, (len(some),), generator=g).double() * 2 - 1
            return t.view(shape)
        self.X, self.dY = values("X", rows, K), values("dY", rows, N)
        self.A, self.B = values("A", groups, rank, K), values("B", groups, N, rank)
        self.ids = torch.randint(-1, groups, (rows,), generator=g)
        self.ids[rows // 2] = 0
        self.scale = torch.randint(0, 2, (groups,), generator=g).float() + 1.0
        self.base = {w: torch.randint(-100, 101, (rows, w), generator=g).float() for w in {N, K}}

    def wanted(self):
        """(out, dX, dA, dB, the largest of P or U), and that no sum of magnitudes leaves fp32."""
        groups, rank, K = self.A.shape
        out, dX = self.base[self.B.shape[1]].double(), self.base[K].double()
        dA, dB, most, between = torch.zeros_like(self.A), torch.zeros_like(self.B), 0.0, [0.0, 0.0]
        for g in range(groups):
            m = (self.ids == g).nonzero().squeeze(1)
            x, dy, a, b, s = self.X[m], self.dY[m], self.A[g], self.B[g], float(self.scale[g])
            p, u = s * (x @ a.t()), s * (dy @ b)
            out[m] += p @ b.t()
            dX[m] += u @ a
            dA[g], dB[g] = u.t() @ x, dy.t() @ p
            pm, um = s * (x.abs() @ a.abs().t()), s * (dy.abs() @ b.abs())
            for t in (pm, um, pm @ b.abs().t() + 100, um @ a.abs() + 100, um.t() @ x.abs(), dy.abs().t() @ pm):
                most = max(most, t.max().item() if t.numel() else 0.0)
            between = [max(v, t.abs().max().item() if t.numel() else 0.0) for v, t in zip(between, (p, u))]
        assert most < 2 ** 24
        return out, dX, dA, dB, *between


# rows, N, K, rank, adapters
SIZES = [(9, 300, 300, 16, 2), (40, 520, 260, 40, 3), (50, 257, 300, 12, 2), (33, 300, 264, 72, 2), (20, 264, 256, 200, 2),
         (1100, 300, 272, 16, 2), (1200, 260, 256, 64, 2), (1030, 256, 264, 100, 2), (1500, 256, 256, 256, 3),
         (2600, 300, 300, 32, 2), (300, 264, 72, 12, 1)]


def run(bk, c, dtype):
    t = DT[dtype]
    offsets, order, _ = bk.group_sort(c.ids.cuda(), c.A.shape[0])
    X, dY, A, B = (v.to(t).cuda() for v in (c.X, c.dY, c.A, c.B))
    N, K = B.shape[1], A.shape[2]
    out = bk.adapter_matmul(X, A, B, offsets, order, c.scale.cuda(), base=c.base[N].cuda())
    return (out, *bk.adapter_matmul_grad(dY, X, A, B, offsets, order, c.scale.cuda(), base=c.base[K].cuda(),
                                         w_dtype=torch.float32))


@pytest.mark.parametrize("sizes", SIZES, ids=str)
@pytest.mark.parametrize("dtype", list(DT))
def test_large_values_of_p(bk, sizes, dtype):
    """X and A dense: P is large, out and dB depend on all of its bits."""
    c = Whole(*sizes, ("X", "A"), 1, high=63 if sizes[2] >= 200 else 127)
    *want, p, u = c.wanted()
    assert p >= 2 ** 17
    for got, w in zip(run(bk, c, dtype), want):
        assert got.dtype == torch.float32 and torch.equal(got.cpu().double(), w)


@pytest.mark.parametrize("sizes", SIZES, ids=str)
@pytest.mark.parametrize("dtype", list(DT))
def test_large_values_of_u(bk, sizes, dtype):
    """dY and B dense: U is large, dX and dA depend on all of its bits."""
    c = Whole(*sizes, ("dY", "B"), 2)
    *want, p, u = c.wanted()
    assert u >= 2 ** 17
    for got, w in zip(run(bk, c, dtype), want):
        assert got.dtype == torch.float32 and torch.equal(got.cpu().double(), w)


@pytest.mark.parametrize("rows,K", [(1, 8200), (3, 8200), (8, 16400), (2, 4100)])
@pytest.mark.parametrize("dtype", list(DT))
def test_long_rows_shared_by_workgroups(bk, rows, K, dtype):
    c = Whole(rows, 300, K, 16, 2, ("X", "A"), 3, high=15)
    want, *_, p, u = c.wanted()
    assert p >= 2 ** 17
    assert torch.equal(run(bk, c, dtype)[0].cpu().double(), want)


@pytest.mark.parametrize("dtype", list(DT))
def test_results_of_both_types(bk, dtype):
    """dX in 16 bits beside dA and dB in fp32 and the other way round: each as without the other."""
    c = Whole(1200, 260, 256, 64, 2, ("dY", "B"), 4)
    t = DT[dtype]
    _, dX, dA, dB, *_ = c.wanted()
    offsets, order, _ = bk.group_sort(c.ids.cuda(), 2)
    args = (*(v.to(t).cuda() for v in (c.dY, c.X, c.A, c.B)), offsets, order, c.scale.cuda())
    narrow = bk.adapter_matmul_grad(*args)
    x, a, b = bk.adapter_matmul_grad(*args, w_dtype=torch.float32)
    assert torch.equal(x, narrow[0]) and torch.equal(a.cpu().double(), dA) and torch.equal(b.cpu().double(), dB)
    x, a, b = bk.adapter_matmul_grad(*args, base=c.base[256].cuda())
    assert torch.equal(x.cpu().double(), dX) and torch.equal(a, narrow[1]) and torch.equal(b, narrow[2])


@pytest.mark.parametrize("rows", [4, 1100])
@pytest.mark.parametrize("dtype,out_dtype", [("bf16", torch.bfloat16), ("bf16", torch.float32), ("f16", torch.float32)])
def test_values_of_p_and_u_just_below_the_largest(bk, rows, dtype, out_dtype):
    """P and U are 2^128 - 2^119, whose 9 bits bf16 would round to infinity.  The other matrix brings them
    back to 2^28 - 2^19 (2^114 - 2^105 from fp16): fp32 holds that, and bf16's nearest, a tie, is 2^28."""
    t, N, rank = DT[dtype], 300, 2
    # 2^64 (2^63 + .. + 2^55); from fp16 2^14 (2^13 + .. + 2^5) 2^100
    one, high, scale, back = (2.0 ** 64, 63, 1.0, 2.0 ** -100) if dtype == "bf16" else (2.0 ** 14, 13, 2.0 ** 100, 2.0 ** -14)
    powers = torch.zeros(N, dtype=torch.float64)
    powers[:9] = 2.0 ** (high - torch.arange(9, dtype=torch.float64))
    A, B = powers.expand(1, rank, N).to(t).cuda(), torch.zeros(1, N, rank, dtype=t, device="cuda")
    B[0, 5, 1] = back
    X = torch.full((rows, N), one, dtype=t, device="cuda")
    s = torch.full((1,), scale, device="cuda")
    want = torch.zeros(rows, N)
    want[:, 5] = (2.0 ** 128 - 2.0 ** 119) * back
    assert torch.equal(bk.adapter_matmul(X, A, B, scale=s, out_dtype=out_dtype).cpu(), want.to(out_dtype))
    # U: X in dY's place, A in that of B and B in that of A
    dX = bk.adapter_matmul_grad(X, X, B.transpose(1, 2).contiguous(), A.transpose(1, 2).contiguous(), scale=s,
                                x_dtype=out_dtype, want_w=False)[0]
    assert torch.equal(dX.cpu(), want.to(out_dtype))
