"""Low-rank adapters beside a shared projection against plain 64-bit implementations.

Tolerances, fixed before the kernels first ran.  h is half a step of a type (bf16 2^-8, fp16
2^-11, fp32 2^-24); the matrix cores' sums of R exact products are off by at most
(R + 8) 2^-23 sum |p q|.
  P = s X A^T:  E_P = s (K + 8) 2^-23 |X| |A|^T + (2^-16 + 2^-23) |P|  (kept as two bf16
    numbers: half a step of the second, 2^-8, of what the first left, 2^-8; and the scale's
    product and sum over the waves).  U = s dY B the same with N.
  out: E_P |B|^T + (4 rank + 8) 2^-23 |P| |B|^T for the sum (up to four products a term), 2^-24 of
    base and sum for their addition, and the output's rounding, h of it (fp16 also 2^-25).
  dX: the same from U and A.  dA, dB: E_U^T |X| + (4 m + 8) 2^-23 |U|^T |X| with m places of the
    group, and the output's rounding.
"""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


@pytest.fixture(scope="module")
def bk():
    from two_sided_gptq_amd import bakron
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    bakron.load()
    return bakron


def strided(t, pad, shift=0):
    """t on the GPU with rows `pad` elements further apart, `shift` elements into the storage."""
    n, k = t.shape
    full = torch.zeros(n * (k + pad) + shift, dtype=t.dtype, device="cuda")
    v = full.as_strided((n, k), (k + pad, 1), shift)
    v.copy_(t)
    return v


def adapters_of(rows, groups, run, seed, none=0.2):
    g = torch.Generator().manual_seed(seed)
    runs = -(-rows // run)
    ids = torch.randint(0, groups, (runs,), generator=g)
    ids[torch.rand(runs, generator=g) < none] = -1
    return ids.repeat_interleave(run)[:rows].to(torch.int32)


class Case:
    def __init__(self, rows, N, K, rank, groups, run, dtype, seed, none=0.2):
        g = torch.Generator().manual_seed(seed)
        t = DT[dtype]
        self.t, self.rank, self.N, self.K, self.groups = t, rank, N, K, groups
        self.ids = adapters_of(rows, groups, run, seed + 1, none)
        self.X = torch.randn(rows, K, generator=g).to(t)
        self.A = (torch.randn(groups, rank, K, generator=g) * K ** -0.5).to(t)
        self.B = (torch.randn(groups, N, rank, generator=g) * 0.1).to(t)
        self.dY = torch.randn(rows, N, generator=g).to(t)
        self.scale = torch.rand(groups, generator=g) + 0.5

    def parts(self, x, w, s):
        """s x w^T in 64 bits and how far it may be off."""
        p, size = s * (x @ w.t()), s * (x.abs() @ w.abs().t())
        return p, (x.shape[1] + 8) * 2.0 ** -23 * size + (2.0 ** -16 + 2.0 ** -23) * p.abs()

    def forward(self, base, scaled=True):
        want = torch.zeros(self.X.shape[0], self.N, dtype=torch.float64) if base is None else base.double().clone()
        error = torch.zeros_like(want)
        for g in range(self.groups):
            m = (self.ids == g).nonzero().squeeze(1)
            b = self.B[g].double()
            p, e = self.parts(self.X[m].double(), self.A[g].double(), float(self.scale[g]) if scaled else 1.0)
            term, size = p @ b.t(), p.abs() @ b.abs().t()
            error[m] = e @ b.abs().t() + (4 * self.rank + 8) * 2.0 ** -23 * size + 2.0 ** -24 * (want[m].abs() + size)
            want[m] += term
        return want, error

    def backward(self, base):
        want = torch.zeros(self.X.shape[0], self.K, dtype=torch.float64) if base is None else base.double().clone()
        error = torch.zeros_like(want)
        grads = [torch.zeros(t.shape, dtype=torch.float64) for t in (self.A, self.A, self.B, self.B)]
        for g in range(self.groups):
            m = (self.ids == g).nonzero().squeeze(1)
            x, dy, a, b, s = (*(t.double() for t in (self.X[m], self.dY[m], self.A[g], self.B[g])), float(self.scale[g]))
            u, eu = self.parts(dy, b.t(), s)
            p, ep = self.parts(x, a, s)
            term, size = u @ a, u.abs() @ a.abs()
            error[m] = eu @ a.abs() + (4 * self.rank + 8) * 2.0 ** -23 * size + 2.0 ** -24 * (want[m].abs() + size)
            want[m] += term
            k = (4 * len(m) + 8) * 2.0 ** -23
            grads[0][g], grads[1][g] = u.t() @ x, eu.t() @ x.abs() + k * (u.abs().t() @ x.abs())
            grads[2][g], grads[3][g] = dy.t() @ p, dy.abs().t() @ ep + k * (dy.abs().t() @ p.abs())
        return (want, error), tuple(grads[:2]), tuple(grads[2:])


def close(got, want, error):
    got = got.cpu()
    bound = error + HALF[got.dtype] * (want.abs() + error) + (2.0 ** -25 if got.dtype == torch.float16 else 0.0)
    off = (got.double() - want).abs()
    assert (off <= bound).all(), f"off by {(off / bound.clamp(min=1e-300)).max():.3g} of what is allowed"


# rows, N, K, rank, adapters, rows of a request, elements between rows, elements before the first
CASES = [(1, 1, 1, 1, 1, 1, 0, 0), (1, 4096, 4096, 16, 4, 1, 0, 0), (3, 7, 33, 5, 2, 1, 0, 0), (17, 65, 100, 12, 3, 1, 3, 1),
         (64, 130, 64, 16, 64, 1, 0, 0), (65, 520, 520, 17, 5, 9, 8, 8), (300, 1000, 136, 32, 2, 70, 0, 0),
         (300, 65, 1001, 33, 4, 11, 1, 3), (1100, 200, 264, 64, 3, 300, 0, 0), (1500, 70, 72, 65, 2, 1, 2, 0),
         (2500, 333, 200, 8, 1, 100, 0, 0), (1030, 129, 515, 128, 2, 128, 0, 5), (40, 96, 80, 200, 7, 3, 0, 0),
         (1200, 64, 128, 256, 2, 17, 0, 0), (9, 40, 4100, 100, 3, 2, 0, 0), (200, 2, 3, 4, 100, 1, 0, 0),
         (5000, 48, 56, 16, 40, 33, 0, 0), (513, 4100, 16, 3, 2, 513, 4, 0)]


@pytest.mark.parametrize("case", CASES, ids=str)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("otype", ["same", "f32"])
def test_forward(bk, case, dtype, otype):
    *sizes, pad, shift = case
    c = Case(*sizes, dtype, 1)
    ot = c.t if otype == "same" else torch.float32
    offsets, order, _ = bk.group_sort(c.ids.cuda(), c.groups)
    X, A, B, scale = strided(c.X, pad, shift), c.A.cuda(), c.B.cuda(), c.scale.cuda()
    base = torch.randn(len(c.ids), c.N, generator=torch.Generator().manual_seed(9)).to(ot)
    want, error = c.forward(base)
    b = strided(base, pad, shift)
    out = bk.adapter_matmul(X, A, B, offsets, order, scale, base=b)
    assert out.dtype == ot
    close(out, want, error)
    assert torch.equal(b.cpu(), base)
    # in place, and rows of no adapter bit for bit
    again = bk.adapter_matmul(X, A, B, offsets, order, scale, base=b, out=b)
    assert again is b and torch.equal(b, out)
    none = c.ids < 0
    assert torch.equal(out.cpu()[none], base[none])
    # without base and scale, into a given output
    want, error = c.forward(None, scaled=False)
    given = strided(torch.full(base.shape, 7.0).to(ot), pad, shift)
    assert bk.adapter_matmul(X, A, B, offsets, order, out=given) is given
    close(given, want, error)
    assert torch.equal(bk.adapter_matmul(X, A, B, offsets, order, out_dtype=ot), given)


@pytest.mark.parametrize("case", CASES, ids=str)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("otype", ["same", "f32"])
def test_gradients(bk, case, dtype, otype):
    *sizes, pad, shift = case
    c = Case(*sizes, dtype, 2)
    ot = c.t if otype == "same" else torch.float32
    offsets, order, _ = bk.group_sort(c.ids.cuda(), c.groups)
    X, dY, A, B, scale = strided(c.X, pad, shift), strided(c.dY, pad, shift), c.A.cuda(), c.B.cuda(), c.scale.cuda()
    base = torch.randn(len(c.ids), c.K, generator=torch.Generator().manual_seed(9)).to(ot)
    (dx, ex), (da, ea), (db, eb) = c.backward(base)
    b = strided(base, pad, shift)
    got = bk.adapter_matmul_grad(dY, X, A, B, offsets, order, scale, base=b, w_dtype=ot)
    assert [t.dtype for t in got] == [ot] * 3
    close(got[0], dx, ex), close(got[1], da, ea), close(got[2], db, eb)
    assert (got[1][(torch.bincount(c.ids.clamp(min=0)[c.ids >= 0].long(), minlength=c.groups) == 0).cuda()] == 0).all()
    # one without the other, in place
    only = bk.adapter_matmul_grad(dY, X, A, B, offsets, order, scale, base=b, out=b, want_w=False)
    assert only[0] is b and only[1:] == (None, None) and torch.equal(b, got[0])
    only = bk.adapter_matmul_grad(dY, X, A, B, offsets, order, scale, want_x=False, w_dtype=ot)
    assert only[0] is None and torch.equal(only[1], got[1]) and torch.equal(only[2], got[2])
    # dX alone
    (dx, ex), _, _ = c.backward(None)
    close(bk.adapter_matmul_grad(dY, X, A, B, offsets, order, scale, x_dtype=ot, want_w=False)[0], dx, ex)


# enough places for workgroups of 64 places by 64 ranks, ragged: of the gradients; of both
MANY = [(2000, 72, 136, 250, 2, 30, 0, 0), (8200, 131, 72, 48, 4, 100, 3, 1), (17000, 64, 200, 33, 3, 177, 0, 0),
        (4200, 300, 67, 256, 2, 1, 0, 0)]


@pytest.mark.parametrize("case", MANY, ids=str)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_many_rows_and_ranks(bk, case, dtype):
    test_forward(bk, case, dtype, "same")
    test_gradients(bk, case, dtype, "f32")


@pytest.mark.parametrize("rows", [5, 70, 1500])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_one_adapter_without_offsets(bk, rows, dtype):
    c = Case(rows, 100, 90, 16, 1, rows, dtype, 3, none=0.0)
    X, A, B = c.X.cuda(), c.A.cuda(), c.B.cuda()
    want = c.forward(None, scaled=False)
    out = bk.adapter_matmul(X, A[0], B[0])
    close(out, *want)
    assert torch.equal(bk.adapter_matmul(X, A, B), out)
    dx, da, db = bk.adapter_matmul_grad(c.dY.cuda(), X, A[0], B[0], scale=c.scale.cuda())
    want = c.backward(None)
    close(dx, *want[0]), close(da[None], *want[1]), close(db[None], *want[2])


def test_rows_that_lie_sorted(bk):
    c = Case(200, 80, 70, 16, 5, 7, "bf16", 4)
    c.ids = torch.cat([c.ids[c.ids >= 0].sort().values, c.ids[c.ids < 0]])
    offsets, order, _ = bk.group_sort(c.ids.cuda(), 5)
    assert torch.equal(order.cpu(), torch.arange(200, dtype=torch.int32))
    X, dY, A, B = c.X.cuda(), c.dY.cuda(), c.A.cuda(), c.B.cuda()
    assert torch.equal(bk.adapter_matmul(X, A, B, offsets), bk.adapter_matmul(X, A, B, offsets, order))
    for a, b in zip(bk.adapter_matmul_grad(dY, X, A, B, offsets), bk.adapter_matmul_grad(dY, X, A, B, offsets, order)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("rows", [30, 1500])
def test_all_rows_without_adapter(bk, rows):
    c = Case(rows, 100, 72, 16, 3, 1, "bf16", 5, none=1.1)
    offsets, order, _ = bk.group_sort(c.ids.cuda(), 3)
    X, dY, A, B = c.X.cuda(), c.dY.cuda(), c.A.cuda(), c.B.cuda()
    base = torch.randn(rows, 100, device="cuda").bfloat16()
    assert torch.equal(bk.adapter_matmul(X, A, B, offsets, order, base=base), base)
    assert (bk.adapter_matmul(X, A, B, offsets, order) == 0).all()
    dx, da, db = bk.adapter_matmul_grad(dY, X, A, B, offsets, order)
    assert (dx == 0).all() and (da == 0).all() and (db == 0).all()


@pytest.mark.parametrize("rows", [40, 1500])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_values_of_other_rows_and_adapters_do_not_leak(bk, rows, dtype):
    """NaN and infinities in rows without adapter, in adapters without rows and in one row."""
    c = Case(rows, 100, 72, 12, 4, 3, dtype, 6)
    c.ids[c.ids == 2] = -1
    offsets, order, _ = bk.group_sort(c.ids.cuda(), 4)
    base, gbase = torch.randn(rows, 100, device="cuda").to(c.t), torch.randn(rows, 72, device="cuda").to(c.t)

    def run():
        args = c.A.cuda(), c.B.cuda(), offsets, order, c.scale.cuda()
        return (bk.adapter_matmul(c.X.cuda(), *args, base=base),
                *bk.adapter_matmul_grad(c.dY.cuda(), c.X.cuda(), *args, base=gbase))
    clean = run()
    none = c.ids < 0
    c.X[none], c.dY[none] = float("nan"), float("inf")
    c.A[2], c.B[2] = float("nan"), float("-inf")
    for a, b in zip(run(), clean):
        assert torch.equal(a, b)
    victim = int((c.ids == 1).nonzero()[0])
    c.X[victim, 5] = float("nan")
    out, dx, da, db = run()
    rest = torch.arange(rows) != victim
    assert torch.equal(out.cpu()[rest], clean[0].cpu()[rest]) and out[victim].isnan().all()
    assert torch.equal(dx, clean[1])
    for got, was in ((da, clean[2]), (db, clean[3])):
        assert torch.equal(got[[0, 2, 3]], was[[0, 2, 3]]) and got[1].isnan().any()


@pytest.mark.parametrize("rows", [30, 1500])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_infinities_of_a_matrix(bk, rows, dtype):
    """Results that depend on a value that is not finite are not finite, all others as they were."""
    c = Case(rows, 300, 72, 16, 2, 3, dtype, 13)
    offsets, order, _ = bk.group_sort(c.ids.cuda(), 2)
    X, dY, args = c.X.cuda(), c.dY.cuda(), (offsets, order)
    clean = bk.adapter_matmul(X, c.A.cuda(), c.B.cuda(), *args)
    grads = bk.adapter_matmul_grad(dY, X, c.A.cuda(), c.B.cuda(), *args)
    c.B[1, 7, 3], c.B[1, 290, 15] = float("inf"), float("-inf")
    out = bk.adapter_matmul(X, c.A.cuda(), c.B.cuda(), *args)
    mine = (c.ids == 1).cuda()
    assert not out[mine][:, [7, 290]].isfinite().any()
    out[mine, 7], out[mine, 290] = clean[mine, 7], clean[mine, 290]
    assert torch.equal(out, clean)
    dx, da, db = bk.adapter_matmul_grad(dY, X, c.A.cuda(), c.B.cuda(), *args)
    assert torch.equal(dx[~mine], grads[0][~mine]) and not dx[mine].isfinite().any()
    assert not da[1, [3, 15]].isfinite().any() and torch.equal(da[0], grads[1][0]) and torch.equal(db, grads[2])


def test_values_between_beyond_fp16(bk):
    """Rank values far beyond fp16's range, and far below it, come through."""
    rows, N, K, rank = 48, 64, 128, 16
    g = torch.Generator().manual_seed(7)
    for size in (300.0, 1e-3):
        c = Case(rows, N, K, rank, 1, rows, "f16", 8, none=0.0)
        c.X = (torch.rand(rows, K, generator=g) * size).half()
        c.A = (torch.rand(1, rank, K, generator=g) * size).half()
        c.B = (torch.randn(1, N, rank, generator=g) * (1e-3 if size > 1 else 1.0)).half()
        out = bk.adapter_matmul(c.X.cuda(), c.A.cuda(), c.B.cuda(), out_dtype=torch.float32)
        close(out, *c.forward(None, scaled=False))
        c.dY = (torch.rand(rows, N, generator=g) * size).half()
        got = bk.adapter_matmul_grad(c.dY.cuda(), c.X.cuda(), c.A.cuda(), c.B.cuda(), x_dtype=torch.float32,
                                     w_dtype=torch.float32, scale=c.scale.cuda())
        for t, want in zip(got, c.backward(None)):
            close(t, *want)


def test_gradients_against_differences(bk):
    """Of L = sum(c * out): by the call in fp32, and by differences of the formula in 64 bits.
    The loss is linear in X, in A and in B, so differences are exact but for 64-bit rounding;
    the call's own error is a relative 2^-15 of the terms."""
    c = Case(7, 6, 5, 3, 2, 2, "bf16", 9)
    offsets, order, _ = bk.group_sort(c.ids.cuda(), 2)
    got = bk.adapter_matmul_grad(c.dY.cuda(), c.X.cuda(), c.A.cuda(), c.B.cuda(), offsets, order, c.scale.cuda(),
                                 x_dtype=torch.float32, w_dtype=torch.float32)

    def loss(x, a, b):
        total = 0.0
        for r, g in enumerate(c.ids.tolist()):
            if g >= 0:
                total = total + c.scale[g].double() * (c.dY[r].double() * (b[g] @ (a[g] @ x[r]))).sum()
        return total
    values = [t.double() for t in (c.X, c.A, c.B)]
    for i, grad in enumerate(got):
        for k in range(values[i].numel()):
            h = torch.zeros(values[i].numel(), dtype=torch.float64)
            h[k] = 1e-3
            up, down = list(values), list(values)
            up[i], down[i] = values[i] + h.view(values[i].shape), values[i] - h.view(values[i].shape)
            assert abs((loss(*up) - loss(*down)) / 2e-3 - grad.cpu().flatten()[k].double()) < 1e-3


@pytest.mark.parametrize("rows", [30, 1500])
def test_places_out_of_range(bk, rows):
    c = Case(rows, 70, 40, 16, 3, 2, "bf16", 10, none=0.0)
    offsets, order, _ = bk.group_sort(c.ids.cuda(), 3)
    X, dY, A, B = c.X.cuda(), c.dY.cuda(), c.A.cuda(), c.B.cuda()
    base = torch.randn(rows, 70, device="cuda").bfloat16()
    want = bk.adapter_matmul(X, A, B, offsets, order, base=base)
    bad = order.clone()
    lost = bad[[1, rows - 2]].long()
    bad[1], bad[rows - 2] = rows, -4
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = base.clone()
    bk.adapter_matmul(X, A, B, offsets, bad, base=out, out=out, dev_status=status)
    assert status.item() == bk.DEV_BAD_INDEX
    keep = torch.ones(rows, dtype=torch.bool, device="cuda")
    keep[lost] = False
    assert torch.equal(out[keep], want[keep]) and torch.equal(out[lost], base[lost])
    status.zero_()
    _, da, db = bk.adapter_matmul_grad(dY, X, A, B, offsets, bad, dev_status=status, want_x=False)
    assert status.item() == bk.DEV_BAD_INDEX
    Z, D = X.clone(), dY.clone()
    Z[lost], D[lost] = 0, 0
    _, wa, wb = bk.adapter_matmul_grad(D, Z, A, B, offsets, order, want_x=False)
    assert torch.equal(da, wa) and torch.equal(db, wb)


@pytest.mark.parametrize("rows", [30, 1500])
def test_offsets_that_fall(bk, rows):
    """Nothing outside the tensors is touched; the result is not defined."""
    c = Case(rows, 70, 40, 16, 4, 2, "bf16", 11)
    _, order, _ = bk.group_sort(c.ids.cuda(), 4)
    X, dY, A, B = c.X.cuda(), c.dY.cuda(), c.A.cuda(), c.B.cuda()
    for values in ([0, rows, 0, rows, 0], [0, rows, -3, rows, rows + 9], [5, rows, 2, rows, rows], [0, -1, -1, -1, -1]):
        offsets = torch.tensor(values, dtype=torch.int32, device="cuda")
        guard = torch.full((rows + 2, 70), 3.0, dtype=torch.bfloat16, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        bk.adapter_matmul(X, A, B, offsets, order, out=guard[1:-1], dev_status=status)
        bk.adapter_matmul_grad(dY, X, A, B, offsets, order, dev_status=status)
        torch.cuda.synchronize()
        assert status.item() == bk.DEV_BAD_INDEX and (guard[0] == 3.0).all() and (guard[-1] == 3.0).all()


def test_no_rows(bk):
    c = Case(4, 70, 40, 16, 3, 1, "bf16", 12)
    X, dY, A, B = c.X.cuda()[:0], c.dY.cuda()[:0], c.A.cuda(), c.B.cuda()
    offsets, order, _ = bk.group_sort(c.ids.cuda()[:0], 3)
    assert bk.adapter_matmul(X, A, B, offsets, order).shape == (0, 70)
    dx, da, db = bk.adapter_matmul_grad(dY, X, A, B, offsets, order)
    assert dx.shape == (0, 40) and (da == 0).all() and (db == 0).all() and da.shape == A.shape and db.shape == B.shape


@pytest.mark.parametrize("rows", [33, 2000])
def test_captured_and_replayed(bk, rows):
    def inputs(seed):
        c = Case(rows, 200, 136, 16, 4, 5, "bf16", seed)
        return [t.cuda() for t in (c.X, c.A, c.B, c.ids, c.scale, c.dY)]

    def run(X, A, B, ids, scale, dY):
        offsets, order, _ = bk.group_sort(ids, 4)
        return (bk.adapter_matmul(X, A, B, offsets, order, scale),
                *bk.adapter_matmul_grad(dY, X, A, B, offsets, order, scale))
    state = inputs(20)
    run(*state)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run(*state)
    for seed in (21, 22, 23):
        for t, n in zip(state, inputs(seed)):
            t.copy_(n)
        want = run(*state)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_another_stream(bk):
    c = Case(300, 200, 136, 16, 4, 5, "f16", 30)
    offsets, order, _ = bk.group_sort(c.ids.cuda(), 4)
    args = c.A.cuda(), c.B.cuda(), offsets, order, c.scale.cuda()
    X, dY = c.X.cuda(), c.dY.cuda()
    want = bk.adapter_matmul(X, *args), *bk.adapter_matmul_grad(dY, X, *args)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = bk.adapter_matmul(X, *args, stream=side), *bk.adapter_matmul_grad(dY, X, *args, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_beside_a_rounded_projection(bk):
    """The use of it: fp8 weights of a solve's codes shared by all, adapters by request, added in place."""
    rows, N, K, rank, groups = 90, 256, 384, 16, 5
    c = Case(rows, N, K, rank, groups, 4, "bf16", 31)
    g = torch.Generator().manual_seed(1)
    codes = torch.randint(-7, 8, (N, K), generator=g, dtype=torch.int8)
    sw = torch.rand(N, generator=g) * 0.01 + 0.005
    W8 = bk.fp8_from_codes(codes.cuda())
    X8, sx = bk.fp8_quantize(c.X.cuda())
    Y = bk.fp8_matmul(X8, sx, W8, sw.cuda())
    base = Y.clone().cpu()
    offsets, order, _ = bk.group_sort(c.ids.cuda(), groups)
    bk.adapter_matmul(c.X.cuda(), c.A.cuda(), c.B.cuda(), offsets, order, c.scale.cuda(), base=Y, out=Y)
    close(Y, *c.forward(base))


def test_refusals(bk):
    c = Case(8, 70, 40, 16, 3, 1, "bf16", 32)
    X, dY, A, B = c.X.cuda(), c.dY.cuda(), c.A.cuda(), c.B.cuda()
    offsets, order, _ = bk.group_sort(c.ids.cuda(), 3)
    f, m = bk.adapter_matmul, bk.adapter_matmul_grad
    base = torch.zeros(8, 70, device="cuda")
    for call in (lambda: f(X.float(), A, B, offsets, order), lambda: f(X, A.half(), B, offsets, order),
                 lambda: f(X, A, B, None, order), lambda: f(X, A, B[:2], offsets, order),
                 lambda: f(X, A[:, :8], B, offsets, order), lambda: f(X[:, :30], A, B, offsets, order),
                 lambda: f(X, A, B, offsets[:3], order), lambda: f(X, A, B, offsets, order[:7]),
                 lambda: f(X, A, B, offsets, order.long()), lambda: f(X, A, B, offsets, order, torch.ones(2, device="cuda")),
                 lambda: f(X, A, B, offsets, order, base=base.half()), lambda: f(X, A, B, offsets, order, base=base[:, :60]),
                 lambda: f(X, A, B, offsets, order, base=base, out_dtype=torch.bfloat16),
                 lambda: f(X, A, B, offsets, order, base=base, out=base.bfloat16()),
                 lambda: f(X, A, B, offsets, order, out_dtype=torch.float16),
                 lambda: f(X, A.transpose(1, 2).contiguous().transpose(1, 2), B, offsets, order),
                 lambda: f(X, torch.zeros(3, 257, 40, device="cuda").bfloat16(),
                           torch.zeros(3, 70, 257, device="cuda").bfloat16(), offsets, order),
                 lambda: f(X.cpu(), A, B, offsets, order), lambda: m(dY[:7], X, A, B, offsets, order),
                 lambda: m(dY.half(), X, A, B, offsets, order), lambda: m(dY, X, A, B, offsets, order, w_dtype=torch.float16),
                 lambda: m(dY, X, A, B, offsets, order, want_x=False, base=X),
                 lambda: m(dY, X, A, B, offsets, order, base=X.half())):
        with pytest.raises(bk.BakronError):
            call()
