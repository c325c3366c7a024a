"""Rows sorted by group and back, against plain 64-bit implementations.

Tolerances, fixed before the kernels first ran:
  sort, copies, fp8 codes and scales: exact.
  combine: k products and sums in fp32, each off by half a step: (k + 1) 2^-24 sum |w y|,
    and the output's rounding (half a step of its type, fp16 also 2^-25).
  gradient of Y: one product, 2^-24 |w d|, and the output's rounding.
  gradient of the weights: `cols` products and sums in fp32 in any order,
    (cols + 1) 2^-24 sum |d y|.
"""
import itertools

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TINY = {"f32": 0.0, "bf16": 0.0, "f16": 2.0 ** -25}


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
    n, k = t.shape
    full = torch.zeros(n * (k + pad) + shift, dtype=t.dtype, device="cuda")
    v = full.as_strided((n, k), (k + pad, 1), shift)
    v.copy_(t)
    return v


def sorted_plain(ids, groups):
    flat = ids.flatten().tolist()
    members = [[] for _ in range(groups + 1)]
    for i, g in enumerate(flat):
        members[g if 0 <= g < groups else groups].append(i)
    offsets = [0] + list(itertools.accumulate(len(m) for m in members[:groups]))
    order = [i for m in members for i in m]
    slots = [0] * len(flat)
    for s, i in enumerate(order):
        slots[i] = s
    i32 = torch.int32
    return (torch.tensor(offsets, dtype=i32), torch.tensor(order, dtype=i32),
            torch.tensor(slots, dtype=i32).view(ids.shape))


def random_ids(tokens, k, groups, seed, dropped=0.2, dtype=torch.int64):
    ids = torch.randint(0, groups, (tokens, k), generator=gen(seed))
    ids[torch.rand(tokens, k, generator=gen(seed + 1)) < dropped] = -1
    return ids.to(dtype)


def check_sort(bk, ids, groups, status=None):
    got = bk.group_sort(ids.cuda(), groups, dev_status=status)
    for g, w in zip(got, sorted_plain(ids, groups)):
        assert g.dtype == torch.int32 and torch.equal(g.cpu(), w)
    return got


# ---------------------------------------------------------------- sort

@pytest.mark.parametrize("tokens,k,groups", [
    (1, 1, 1), (1, 8, 64), (63, 1, 2), (64, 1, 1), (65, 3, 7), (513, 1, 1023), (512, 8, 1024), (1365, 3, 5),
    (2048, 2, 60), (4097, 1, 3), (100, 1, 1025), (5, 2, 4096), (9000, 8, 128), (40000, 2, 4096), (32768, 8, 64),
    (300007, 1, 33), (70001, 4, 2500)])
@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
def test_sort(bk, tokens, k, groups, dtype):
    check_sort(bk, random_ids(tokens, k, groups, tokens + k, dtype=dtype), groups)


@pytest.mark.parametrize("n", [1, 64, 4096, 4097, 300000])
def test_sort_of_one_group_and_of_none(bk, n):
    check_sort(bk, torch.full((n,), 2), 5)
    check_sort(bk, torch.full((n,), -1), 5)
    check_sort(bk, torch.arange(n) % 5, 5)
    check_sort(bk, 4 - torch.arange(n) % 5, 5)
    check_sort(bk, (torch.arange(n) * 5) // n, 5)


@pytest.mark.parametrize("n", [100, 5000, 300000])
def test_sort_reports_groups_that_are_too_large(bk, n):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ids = torch.arange(n) % 9
    check_sort(bk, ids - 1, 8, status)
    assert status.item() == 0
    check_sort(bk, ids, 8, status)  # 8 is none of 8 groups
    assert status.item() == bk.DEV_BAD_INDEX
    status.zero_()
    ids[n // 2] = (1 << 40) + 1
    check_sort(bk, torch.where(ids == 8, -1, ids), 8, status)
    assert status.item() == bk.DEV_BAD_INDEX


def test_nothing_to_sort(bk):
    offsets, order, slots = bk.group_sort(torch.empty((0, 4), dtype=torch.int64, device="cuda"), 3)
    assert offsets.tolist() == [0, 0, 0, 0] and order.shape == (0,) and slots.shape == (0, 4)
    X = torch.empty((0, 16), dtype=torch.bfloat16, device="cuda")
    assert bk.group_gather(X, slots, offsets).shape == (0, 16)
    q, s = bk.group_gather_fp8(X, slots, offsets)
    assert q.shape == (0, 16) and s.shape == (1, 0)
    assert bk.group_combine(X, slots, offsets).shape == (0, 16)
    w = torch.empty((0, 4), device="cuda")
    dy, dw = bk.group_combine_grad(X, X, slots, offsets, w)
    assert dy.shape == (0, 16) and dw.shape == (0, 4)


# ---------------------------------------------------------------- rows

# tokens, k, groups, cols, elements between rows, elements before the first
ROWS = [(1, 1, 1, 1, 0, 0), (1, 8, 9, 4096, 0, 0), (3, 64, 70, 7, 0, 0), (7, 2, 3, 8, 8, 8), (65, 9, 12, 513, 3, 1),
        (130, 4, 8, 1025, 0, 0), (33, 3, 5, 2050, 6, 2), (700, 2, 16, 1000, 0, 0), (530, 8, 64, 2048, 0, 0),
        (600, 5, 6, 127, 1, 3), (515, 1, 4, 2177, 0, 1), (9, 17, 20, 520, 8, 0)]


def rows_case(bk, shape, seed, dropped=0.25):
    tokens, k, groups, cols, pad, shift = shape
    ids = random_ids(tokens, k, groups, seed, dropped)
    offsets, order, slots = bk.group_sort(ids.cuda(), groups)
    return ids, offsets, order, slots


@pytest.mark.parametrize("shape", ROWS, ids=str)
@pytest.mark.parametrize("dtype", list(DT))
def test_gather(bk, shape, dtype):
    tokens, k, groups, cols, pad, shift = shape
    ids, offsets, order, slots = rows_case(bk, shape, 3)
    x = torch.randn(tokens, cols, generator=gen(1)).to(DT[dtype])
    X = strided(x, pad, shift)
    out = strided(torch.full((tokens * k, cols), 7.0).to(DT[dtype]), pad, shift)
    got = bk.group_gather(X, slots, offsets, out=out)
    assert got is out
    want = x[order.cpu().long() // k]
    want[int(offsets[-1]):] = 0
    assert torch.equal(got.cpu(), want)
    assert torch.equal(bk.group_gather(X, slots, offsets).cpu(), want)


@pytest.mark.parametrize("dtype", list(DT))
def test_gather_copies_every_bit_pattern(bk, dtype):
    words = torch.randint(-2 ** 31, 2 ** 31 - 1, (50, 300), generator=gen(5), dtype=torch.int64).to(torch.int32)
    X = words.view(DT[dtype]).cuda()
    ids = random_ids(50, 3, 4, 9, 0.0)
    offsets, order, slots = bk.group_sort(ids.cuda(), 4)
    got = bk.group_gather(X, slots, offsets).cpu()
    assert torch.equal(got.view(torch.int32), words[order.cpu().long() // 3])


@pytest.mark.parametrize("shape", ROWS, ids=str)
@pytest.mark.parametrize("dtype", list(DT))
def test_gather_fp8(bk, shape, dtype):
    """The codes and scales of fp8_quantize, row by row; a dropped row is one of zeros."""
    tokens, k, groups, cols, pad, shift = shape
    ids, offsets, order, slots = rows_case(bk, shape, 4)
    x = torch.randn(tokens, cols, generator=gen(2))
    x[:, ::7] *= 30.0
    x[tokens // 2, :cols // 2] = 0.0
    X = strided(x.to(DT[dtype]), pad, shift)
    q, s = bk.fp8_quantize(X)
    source = order.cpu().long() // k
    end = int(offsets[-1])
    wq, ws = q.cpu().view(torch.uint8)[source], s.cpu()[:, source]
    wq[end:], ws[:, end:] = 0, 1.0
    out = strided(torch.full((tokens * k, cols), 7.0).to(torch.float8_e4m3fn), pad, shift)
    got, scales = bk.group_gather_fp8(X, slots, offsets, out=out)
    assert torch.equal(got.cpu().view(torch.uint8), wq) and torch.equal(scales.cpu(), ws)


def test_gather_fp8_of_values_without_a_scale(bk):
    """A NaN or an infinity makes its block NaN and is reported, but not where the row is dropped."""
    X = torch.ones(4, 300, device="cuda")
    X[1, 200], X[2, 5] = float("nan"), float("inf")
    for ids, flag in (([0, 1, 0, 1], bk.DEV_NONFINITE), ([0, -1, -1, 1], 0)):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        offsets, order, slots = bk.group_sort(torch.tensor(ids, device="cuda"), 2)
        q, s = bk.group_gather_fp8(X, slots, offsets, dev_status=status)
        assert status.item() == flag
        if flag:
            wq, ws = bk.fp8_quantize(X[order.long()])
            assert torch.equal(q.view(torch.uint8), wq.view(torch.uint8))
            assert torch.equal(s.isnan(), ws.isnan()) and s.isnan().sum() == 2


def rounded(want, error, dtype):
    return error + HALF[dtype] * (want.abs() + error) + TINY[dtype]


@pytest.mark.parametrize("shape", ROWS, ids=str)
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("weighted", [True, False])
def test_combine(bk, shape, dtype, weighted):
    tokens, k, groups, cols, pad, shift = shape
    ids, offsets, order, slots = rows_case(bk, shape, 5)
    y = torch.randn(tokens * k, cols, generator=gen(3)).to(DT[dtype])
    y[int(offsets[-1]):] = float("nan")  # rows of no group are not read
    w = torch.randn(tokens, k, generator=gen(4))
    out = strided(torch.full((tokens, cols), 7.0).to(DT[dtype]), pad, shift)
    got = bk.group_combine(strided(y, pad, shift), slots, offsets, w.cuda() if weighted else None, out=out)
    assert got is out
    kept = (ids >= 0)[:, :, None]
    terms = torch.where(kept, y.double()[slots.cpu().long()], 0.0) * (w.double()[:, :, None] if weighted else 1.0)
    want = terms.sum(1)
    error = (k + 1) * 2.0 ** -24 * terms.abs().sum(1)
    assert ((got.cpu().double() - want).abs() <= rounded(want, error, dtype)).all()
    same = bk.group_combine(strided(y, pad, shift), slots, offsets, w.cuda() if weighted else None)
    assert torch.equal(same, got)


@pytest.mark.parametrize("shape", ROWS, ids=str)
@pytest.mark.parametrize("dtype", list(DT))
def test_combine_grad(bk, shape, dtype):
    tokens, k, groups, cols, pad, shift = shape
    ids, offsets, order, slots = rows_case(bk, shape, 6)
    y = torch.randn(tokens * k, cols, generator=gen(5)).to(DT[dtype])
    y[int(offsets[-1]):] = float("nan")
    d = torch.randn(tokens, cols, generator=gen(6)).to(DT[dtype])
    w = torch.randn(tokens, k, generator=gen(7))
    out = strided(torch.full((tokens * k, cols), 7.0).to(DT[dtype]), pad, shift)
    dy, dw = bk.group_combine_grad(strided(d, pad, shift), strided(y, pad, shift), slots, offsets, w.cuda(), out=out)
    assert dy is out and dw.dtype == torch.float32
    kept = ids >= 0
    at = slots.cpu().long()
    rows = torch.where(kept[:, :, None], w.double()[:, :, None] * d.double()[:, None, :], 0.0)
    want = torch.empty(tokens * k, cols, dtype=torch.float64)
    want[at.flatten()] = rows.flatten(0, 1)
    assert ((dy.cpu().double() - want).abs() <= rounded(want, 2.0 ** -24 * want.abs(), dtype)).all()
    terms = torch.where(kept[:, :, None], d.double()[:, None, :] * y.double()[at], 0.0)
    assert ((dw.cpu().double() - terms.sum(2)).abs() <= (cols + 1) * 2.0 ** -24 * terms.abs().sum(2)).all()


def test_gradients_against_differences(bk):
    """Of L = sum(c * combine(gather(x) * m, w)): by the calls, and by differences in 64 bits."""
    tokens, k, groups, cols = 5, 3, 4, 11
    ids = random_ids(tokens, k, groups, 1)
    offsets, order, slots = bk.group_sort(ids.cuda(), groups)
    x, w = torch.randn(tokens, cols, generator=gen(1)), torch.randn(tokens, k, generator=gen(2))
    m, c = torch.randn(tokens * k, cols, generator=gen(3)), torch.randn(tokens, cols, generator=gen(4))
    Y = bk.group_gather(x.cuda(), slots, offsets) * m.cuda()
    dY, dw = bk.group_combine_grad(c.cuda(), Y, slots, offsets, w.cuda())
    dx = bk.group_combine(dY * m.cuda(), slots, offsets)

    def loss(x, w):
        rows = x[torch.arange(tokens)[:, None].expand(-1, k)] * m.double()[slots.cpu().long()]
        return (c.double() * (torch.where(ids >= 0, w, 0.0)[:, :, None] * rows).sum(1)).sum()
    h = 1e-5
    for value, grad, which in ((x, dx, 0), (w, dw, 1)):
        value = value.double()
        for i in range(value.numel()):
            e = torch.zeros(value.numel(), dtype=torch.float64)
            e[i] = h
            e = e.view(value.shape)
            args = [x.double(), w.double()]
            args[which] = value + e
            up = loss(*args)
            args[which] = value - e
            # the loss is linear in each: the difference is exact but for 64-bit rounding
            assert abs((up - loss(*args)) / (2 * h) - grad.cpu().flatten()[i].double()) < 1e-4


def test_slots_out_of_range_are_left_out(bk):
    X = torch.randn(6, 700, device="cuda")
    offsets, order, slots = bk.group_sort(torch.arange(6, device="cuda") % 2, 2)
    bad = slots.clone()
    bad[1], bad[4] = 6, -3
    w = torch.ones(6, device="cuda")

    def flagged(call):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        result = call(status)
        assert status.item() == bk.DEV_BAD_INDEX
        return result
    out = torch.full((6, 700), 7.0, device="cuda")
    flagged(lambda st: bk.group_gather(X, bad, offsets, out=out, dev_status=st))
    want = X[order.long()].clone()
    want[slots[[1, 4]].long()] = 7.0
    assert torch.equal(out, want)
    flagged(lambda st: bk.group_gather_fp8(X, bad, offsets, dev_status=st))
    got = flagged(lambda st: bk.group_combine(X, bad, offsets, w, dev_status=st))
    want = X[slots.long()].clone()
    want[[1, 4]] = 0.0
    assert torch.equal(got, want)
    out.fill_(7.0)
    dy, dw = flagged(lambda st: bk.group_combine_grad(X, X, bad, offsets, w, out=out, dev_status=st))
    assert dw[[1, 4]].tolist() == [0.0, 0.0] and (dy[slots[[1, 4]].long()] == 7.0).all()


@pytest.mark.parametrize("last", [-5, 1000])
def test_a_last_offset_out_of_range_is_kept_inside(bk, last):
    X = torch.randn(8, 64, device="cuda")
    _, order, slots = bk.group_sort(torch.arange(8, device="cuda") % 2, 2)
    offsets = torch.tensor([0, 4, last], dtype=torch.int32, device="cuda")
    got = bk.group_gather(X, slots, offsets)
    assert torch.equal(got, X[order.long()] if last > 0 else torch.zeros_like(X))
    back = bk.group_combine(got, slots, offsets)
    assert torch.equal(back, X if last > 0 else torch.zeros_like(X))


# ---------------------------------------------------------------- graphs and streams

def layer(bk, X, W, ids, weights, groups):
    offsets, order, slots = bk.group_sort(ids, groups)
    Xs = bk.group_gather(X, slots, offsets)
    Y = bk.grouped_matmul(Xs, W, offsets)
    out = bk.group_combine(Y, slots, offsets, weights)
    dY, dw = bk.group_combine_grad(out, Y, slots, offsets, weights)
    dXs, dW = bk.grouped_matmul_grad(dY, Xs, W, offsets)
    return out, dw, dW, bk.group_combine(dXs, slots, offsets)


def layer_inputs(tokens, k, groups, width, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    X = torch.randn(tokens, width, device="cuda", generator=g).bfloat16()
    W = (torch.randn(groups, width, width, device="cuda", generator=g) * width ** -0.5).bfloat16()
    ids = torch.rand(tokens, groups, device="cuda", generator=g).topk(k, dim=1).indices
    return X, W, ids, torch.rand(tokens, k, device="cuda", generator=g)


@pytest.mark.parametrize("tokens", [40, 3000])
def test_a_layer_of_experts(bk, tokens):
    """Forward and backward of a whole layer against autograd in 64 bits.  bf16's rounding of
    Y, dY and the outputs, half a step (2^-8) each, is taken relative to the norms: three
    of them at most lie between the inputs and a result."""
    groups, k = 6, 2
    X, W, ids, weights = layer_inputs(tokens, k, groups, 128, 1)
    out, dw, dW, dX = layer(bk, X, W, ids, weights, groups)
    x, w, p = (t.double().cpu().requires_grad_() for t in (X, W, weights))
    terms = []
    for j in range(k):
        e = ids[:, j].cpu()
        y = torch.zeros(tokens, 128, dtype=torch.float64)
        for g in range(groups):
            y = y + torch.where((e == g)[:, None], x @ w[g].t(), 0.0)
        terms.append(p[:, j:j + 1] * y)
    want = sum(terms)
    want.backward(out.cpu().double())
    for got, ref in ((out, want), (dw, p.grad), (dW, w.grad), (dX, x.grad)):
        assert (got.cpu().double() - ref).norm() <= 3 * 2.0 ** -8 * ref.norm()


def test_captured_and_replayed(bk):
    groups = 7
    X, W, ids, weights = layer_inputs(5000, 2, groups, 64, 2)
    layer(bk, X, W, ids, weights, groups)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = layer(bk, X, W, ids, weights, groups)
    for seed in (3, 4, 5):
        for t, n in zip((X, W, ids, weights), layer_inputs(5000, 2, groups, 64, seed)):
            t.copy_(n)
        want = layer(bk, X, W, ids, weights, groups)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_another_stream(bk):
    groups = 7
    X, W, ids, weights = layer_inputs(5000, 2, groups, 64, 6)
    offsets, order, slots = bk.group_sort(ids, groups)
    want = bk.group_gather(X, slots, offsets)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = bk.group_sort(ids, groups, stream=side)
    rows = bk.group_gather(X, got[2], got[0], stream=side)
    q, s = bk.group_gather_fp8(X, got[2], got[0], stream=side)
    back = bk.group_combine(rows, got[2], got[0], weights, stream=side)
    dy, dw = bk.group_combine_grad(X, rows, got[2], got[0], weights, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, (offsets, order, slots)))
    assert torch.equal(rows, want)
    wq, ws = bk.group_gather_fp8(X, slots, offsets)
    assert torch.equal(q.view(torch.uint8), wq.view(torch.uint8)) and torch.equal(s, ws)
    assert torch.equal(back, bk.group_combine(want, slots, offsets, weights))
    for a, b in zip((dy, dw), bk.group_combine_grad(X, want, slots, offsets, weights)):
        assert torch.equal(a, b)


# ---------------------------------------------------------------- refusals of the binding

def test_refusals(bk):
    ids = torch.zeros(4, 2, dtype=torch.int64, device="cuda")
    offsets, order, slots = bk.group_sort(ids, 3)
    X = torch.zeros(4, 16, device="cuda")
    Y = torch.zeros(8, 16, device="cuda")
    w = torch.zeros(4, 2, device="cuda")
    E = bk.BakronError
    for call in (lambda: bk.group_sort(ids.float(), 3), lambda: bk.group_sort(ids.cpu(), 3),
                 lambda: bk.group_sort(ids, 0), lambda: bk.group_sort(ids, 4097), lambda: bk.group_sort(ids.t(), 3),
                 lambda: bk.group_gather(X, slots.long(), offsets), lambda: bk.group_gather(X[:3], slots, offsets),
                 lambda: bk.group_gather(X, slots, offsets[:1]), lambda: bk.group_gather(X.t(), slots, offsets),
                 lambda: bk.group_gather(X, slots, offsets.cpu()), lambda: bk.group_gather(X.long(), slots, offsets),
                 lambda: bk.group_gather(X, slots, offsets, out=Y.half()),
                 lambda: bk.group_gather_fp8(X, slots, offsets, out=Y),
                 lambda: bk.group_gather_fp8(X, slots, offsets, scales=w),
                 lambda: bk.group_combine(X, slots, offsets), lambda: bk.group_combine(Y, slots, offsets, w.half()),
                 lambda: bk.group_combine(Y, slots, offsets, w[:, :1]), lambda: bk.group_combine(Y, slots, offsets, out=Y),
                 lambda: bk.group_combine_grad(X, Y, slots, offsets, None),
                 lambda: bk.group_combine_grad(X.half(), Y, slots, offsets, w),
                 lambda: bk.group_combine_grad(Y, Y, slots, offsets, w)):
        with pytest.raises(E):
            call()
