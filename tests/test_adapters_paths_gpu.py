"""Adapters where each form of the kernels runs whole tiles: ranks of every number of 32-rank steps with
256 columns and more, few rows and many, long rows that workgroups share, tables of adapters far larger
than the batch, and gradients whose offsets pass 32 bits.

The cases' 64-bit results and tolerances are those of test_adapters_gpu, which derives them.
"""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_adapters_gpu import Case, close, strided  # noqa: E402


@pytest.fixture(scope="module")
def bk():
    from two_sided_gptq_amd import bakron
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    bakron.load()
    return bakron


def both_ways(bk, c, pad, shift, otype):
    ot = c.t if otype == "same" else torch.float32
    offsets, order, _ = bk.group_sort(c.ids.cuda(), c.groups)
    X, dY, A, B, scale = strided(c.X, pad, shift), strided(c.dY, pad, shift), c.A.cuda(), c.B.cuda(), c.scale.cuda()
    g = torch.Generator().manual_seed(9)
    for base in (None, torch.randn(len(c.ids), c.N, generator=g).to(ot)):
        b = None if base is None else strided(base, pad, shift)
        close(bk.adapter_matmul(X, A, B, offsets, order, scale, base=b, out_dtype=ot), *c.forward(base))
    base = torch.randn(len(c.ids), c.K, generator=g).to(ot)
    got = bk.adapter_matmul_grad(dY, X, A, B, offsets, order, scale, base=strided(base, pad, shift), w_dtype=ot)
    for t, want in zip(got, c.backward(base)):
        close(t, *want)


# rows, N, K, adapters, rows of a request, elements between rows, elements before the first
SHAPES = [(37, 300, 520, 3, 2, 0, 0), (130, 520, 264, 2, 30, 3, 1), (1100, 300, 264, 3, 77, 0, 0), (1300, 257, 300, 2, 1, 1, 3)]


@pytest.mark.parametrize("rank", [8, 24, 40, 64, 72, 104, 128, 136, 200, 256])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("otype", ["same", "f32"])
def test_ranks_with_whole_columns(bk, shape, rank, dtype, otype):
    rows, N, K, groups, run, pad, shift = shape
    both_ways(bk, Case(rows, N, K, rank, groups, run, dtype, rank + rows), pad, shift, otype)


# whole tiles without a ragged end anywhere
@pytest.mark.parametrize("rows,N,K,rank,groups", [(64, 256, 256, 64, 1), (1024, 512, 256, 64, 1), (4096, 256, 512, 128, 4)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_nothing_ragged(bk, rows, N, K, rank, groups, dtype):
    both_ways(bk, Case(rows, N, K, rank, groups, rows // groups, dtype, 3, none=0.0), 0, 0, "same")


@pytest.mark.parametrize("rows,K,rank,groups", [(1, 4100, 16, 1), (1, 8200, 16, 2), (8, 8192, 8, 3), (3, 16400, 24, 2), (8, 16400, 40, 8), (40, 8200, 16, 3)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_long_rows(bk, rows, K, rank, groups, dtype):
    both_ways(bk, Case(rows, 300, K, rank, groups, 1, dtype, K + rows), 0, 0, "same")


@pytest.mark.parametrize("rows", [1, 8, 64])
@pytest.mark.parametrize("groups", [128, 1024, 4096])
@pytest.mark.parametrize("rank", [16, 40])
def test_tables_far_larger_than_the_batch(bk, rows, groups, rank):
    """Most adapters have no row; their gradients are 0."""
    c = Case(rows, 260, 264, rank, groups, 1, "bf16", groups + rows)
    c.ids[-1] = groups - 1
    offsets, order, _ = bk.group_sort(c.ids.cuda(), groups)
    X, dY, A, B, scale = (t.cuda() for t in (c.X, c.dY, c.A, c.B, c.scale))
    out = bk.adapter_matmul(X, A, B, offsets, order, scale)
    dX, dA, dB = bk.adapter_matmul_grad(dY, X, A, B, offsets, order, scale)
    used = c.ids[c.ids >= 0].unique()
    rest = torch.ones(groups, dtype=torch.bool)
    rest[used.long()] = False
    assert not dA[rest.cuda()].any() and not dB[rest.cuda()].any()
    # the same with a table of the adapters that have rows
    few = Case(rows, 260, 264, rank, len(used), 1, "bf16", 0)
    few.X, few.dY, few.A, few.B, few.scale = c.X, c.dY, c.A[used.long()], c.B[used.long()], c.scale[used.long()]
    few.ids = torch.where(c.ids < 0, -1, torch.searchsorted(used, c.ids))
    close(out, *few.forward(None))
    dx, da, db = few.backward(None)
    close(dX, *dx), close(dA[used.long().cuda()], *da), close(dB[used.long().cuda()], *db)


@pytest.mark.parametrize("N,K,groups", [(64, 33000, 4096), (33000, 64, 4096), (64, 33000, 8)])
def test_gradients_beyond_32_bits(bk, N, K, groups):
    """131072 rows of 33000 inputs or outputs, 4.3e9 elements, and with 4096 adapters matrices of 2.2e9."""
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 60 * 2 ** 30:
        pytest.skip("needs 60 GiB of GPU memory")
    rows, rank = 131072, 16
    g = torch.Generator(device="cuda").manual_seed(1)
    ids = torch.randint(0, groups, (rows,), device="cuda", generator=g)
    offsets, order, _ = bk.group_sort(ids, groups)

    def normal(*shape):
        return torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    X, dY, A, B = normal(rows, K), normal(rows, N), normal(groups, rank, K), normal(groups, N, rank)
    dX, dA, dB = bk.adapter_matmul_grad(dY, X, A, B, offsets, order)

    def close_to(got, want, error):
        assert ((got.double() - want).abs() <= error + 2.0 ** -8 * (want.abs() + error)).all()

    def between(v, w):
        """v w^T and how far it may be off."""
        p = v @ w.t()
        return p, (v.shape[1] + 8) * 2.0 ** -23 * (v.abs() @ w.abs().t()) + (2.0 ** -16 + 2.0 ** -23) * p.abs()
    for r in (0, 1, rows // 2 - 1, rows // 2, rows - 1):
        a = A[ids[r]].double()
        u, e = between(dY[r:r + 1].double(), B[ids[r]].double().t())
        close_to(dX[r:r + 1], u @ a, e @ a.abs() + (4 * rank + 8) * 2.0 ** -23 * (u.abs() @ a.abs()))
    for i in (0, 1, groups // 2, groups - 1):
        m = (ids == i).nonzero().squeeze(1)
        x, dy = X[m].double(), dY[m].double()
        (u, eu), (p, ep), k = between(dy, B[i].double().t()), between(x, A[i].double()), (4 * len(m) + 8) * 2.0 ** -23
        close_to(dA[i], u.t() @ x, eu.t() @ x.abs() + k * (u.abs().t() @ x.abs()))
        close_to(dB[i], dy.t() @ p, dy.abs().t() @ ep + k * (dy.abs().t() @ p.abs()))
