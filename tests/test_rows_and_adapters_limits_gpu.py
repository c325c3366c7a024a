"""Rows by group, adapters and drafts where offsets pass 32 bits, at the largest numbers of pairs,
where a launch would have 2^32 threads, and with calls that run at the same time."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def bk():
    from two_sided_gptq_amd import bakron
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    bakron.load()
    return bakron


def room(gib):
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < gib * 2 ** 30:
        pytest.skip(f"needs {gib} GiB of GPU memory")


@pytest.mark.parametrize("n,groups", [(1 << 24, 1), (1 << 24, 200), ((1 << 24) - 3, 4096), ((1 << 20) + 1, 1000)])
def test_sorts_of_the_largest_size(bk, n, groups):
    g = torch.Generator(device="cuda").manual_seed(n + groups)
    ids = torch.randint(-1, groups, (n,), device="cuda", generator=g)
    offsets, order, slots = bk.group_sort(ids, groups)
    key = torch.where(ids < 0, groups, ids)
    want = torch.sort(key, stable=True).indices
    assert torch.equal(order.long(), want)
    assert torch.equal(slots[want].long(), torch.arange(n, device="cuda"))
    assert torch.equal(offsets[1:].long(), torch.bincount(key, minlength=groups + 1)[:groups].cumsum(0))


def test_rows_beyond_32_bits(bk):
    """9 GiB of sorted rows, 4.6e9 elements: copies, sums and gradients at both ends."""
    room(60)
    tokens, k, cols = 70000, 4, 16400
    ids = torch.arange(tokens * k, device="cuda").view(tokens, k) % 7
    offsets, order, slots = bk.group_sort(ids, 7)
    X = torch.zeros(tokens, cols, dtype=torch.bfloat16, device="cuda")
    marks = torch.tensor([0, 1, tokens // 2, tokens - 2, tokens - 1], device="cuda")
    X[marks] = torch.randn(5, cols, device="cuda").bfloat16()
    Y = bk.group_gather(X, slots, offsets)
    for t in marks.tolist():
        for j in range(k):
            assert torch.equal(Y[int(slots[t, j])], X[t])
    assert int((Y[:, 0] != 0).sum()) <= 5 * k
    w = torch.full((tokens, k), 0.25, device="cuda")
    assert torch.equal(bk.group_combine(Y, slots, offsets, w), X)
    dY, dw = bk.group_combine_grad(X, Y, slots, offsets, w)
    for t in marks.tolist():
        for j in range(k):
            assert torch.equal(dY[int(slots[t, j])], X[t] * 0.25)
        # dw = |x|^2: cols products and sums in fp32
        want = (X[t].double() ** 2).sum()
        assert ((dw[t].double() - want).abs() <= (cols + 1) * 2.0 ** -24 * want).all()
    del dY
    q, s = bk.group_gather_fp8(X, slots, offsets)
    wq, ws = bk.fp8_quantize(X[marks])
    for i, t in enumerate(marks.tolist()):
        for j in range(k):
            at = int(slots[t, j])
            assert torch.equal(q[at].view(torch.uint8), wq[i].view(torch.uint8)) and torch.equal(s[:, at], ws[:, i])


def test_more_threads_than_a_launch_has(bk):
    """2^24 rows of 2064 columns: 5 waves a token are more than 2^32 threads, so are 4 waves of a
    token in the gradient."""
    room(230)
    tokens, cols = 1 << 24, 2064
    ids = torch.zeros(tokens, dtype=torch.int32, device="cuda")
    offsets, order, slots = bk.group_sort(ids, 1)
    X = torch.zeros(tokens, cols, dtype=torch.bfloat16, device="cuda")
    X[:, 0] = (torch.arange(tokens, device="cuda") % 251).bfloat16()
    X[:, -1] = (torch.arange(tokens, device="cuda") % 241).bfloat16()
    for call in (lambda out: bk.group_gather(X, slots, offsets, out=out), lambda out: bk.group_combine(X, slots, offsets, out=out)):
        out = call(torch.full_like(X, 3.0))
        assert torch.equal(out[:, 0], X[:, 0]) and torch.equal(out[:, -1], X[:, -1]) and not out[:, 1:-1].any()
        del out
    w = torch.full((tokens,), 2.0, device="cuda")
    dY, dw = bk.group_combine_grad(X, X, slots, offsets, w)
    assert torch.equal(dY[:, 0], 2 * X[:, 0]) and torch.equal(dY[:, -1], 2 * X[:, -1])
    assert torch.equal(dw, X[:, 0].float() ** 2 + X[:, -1].float() ** 2)  # whole numbers: exact


def test_adapters_beyond_32_bits(bk):
    """131072 rows of 33000 outputs, 4.3e9 elements, and matrices of 2.2e9."""
    room(60)
    rows, N, K, rank, groups = 131072, 33000, 64, 16, 4096
    g = torch.Generator(device="cuda").manual_seed(1)
    ids = torch.randint(0, groups, (rows,), device="cuda", generator=g)
    offsets, order, _ = bk.group_sort(ids, groups)
    X = torch.randn(rows, K, device="cuda", generator=g).bfloat16()
    A = torch.randn(groups, rank, K, device="cuda", generator=g).bfloat16()
    B = torch.empty(groups, N, rank, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    out = bk.adapter_matmul(X, A, B, offsets, order)
    some = torch.tensor([0, 1, 65535, 65536, rows - 1], device="cuda")
    for r in some.tolist():
        a, b, x = A[ids[r]].double(), B[ids[r]].double(), X[r].double()
        p, size = a @ x, a.abs() @ x.abs()
        e = (K + 8) * 2.0 ** -23 * size + (2.0 ** -16 + 2.0 ** -23) * p.abs()
        want, error = b @ p, b.abs() @ e + (4 * rank + 8) * 2.0 ** -23 * (b.abs() @ p.abs())
        assert ((out[r].double() - want).abs() <= error + 2.0 ** -8 * (want.abs() + error)).all()


def test_calls_at_the_same_time(bk):
    """Two streams with work of their own, many calls in flight on each."""
    g = torch.Generator(device="cuda").manual_seed(2)
    sets = []
    for rows, groups in ((3000, 7), (90, 5)):
        ids = torch.randint(-1, groups, (rows,), device="cuda", generator=g)
        sets.append((ids, groups, torch.randn(rows, 512, device="cuda", generator=g).bfloat16(),
                     torch.randn(groups, 16, 512, device="cuda", generator=g).bfloat16(),
                     torch.randn(groups, 768, 16, device="cuda", generator=g).bfloat16(),
                     torch.randn(rows, 768, device="cuda", generator=g).bfloat16(),
                     torch.rand(rows, 3, 4000, device="cuda", generator=g).softmax(2), torch.rand(rows, 2, device="cuda", generator=g),
                     torch.rand(rows, device="cuda", generator=g)))

    def work(ids, groups, X, A, B, dY, p, u, v):
        offsets, order, slots = bk.group_sort(ids, groups)
        return [offsets, order, slots, bk.group_gather(X, slots, offsets), *bk.group_gather_fp8(X, slots, offsets),
                bk.adapter_matmul(X, A, B, offsets, order), *bk.adapter_matmul_grad(dY, X, A, B, offsets, order),
                *bk.verify_drafts(p, None, torch.zeros(u.shape, dtype=torch.int64, device="cuda"), u, v)]
    want = [work(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(8):
        for i, stream in enumerate(streams):
            with torch.cuda.stream(stream):
                got[i].append(work(*sets[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for result in got[i]:
            for a, b in zip(result, want[i]):
                if a.dtype == torch.float8_e4m3fn:
                    a, b = a.view(torch.uint8), b.view(torch.uint8)
                assert torch.equal(a, b)


def test_graphs_that_take_turns(bk):
    """Two captured graphs with memory of one pool, replayed in turn, with eager calls between."""
    g = torch.Generator(device="cuda").manual_seed(3)
    rows, groups = 2500, 6
    ids = torch.randint(-1, groups, (rows,), device="cuda", generator=g)
    X = torch.randn(rows, 256, device="cuda", generator=g).bfloat16()
    A = torch.randn(groups, 16, 256, device="cuda", generator=g).bfloat16()
    B = torch.randn(groups, 320, 16, device="cuda", generator=g).bfloat16()
    dY = torch.randn(rows, 320, device="cuda", generator=g).bfloat16()

    def forward():
        offsets, order, slots = bk.group_sort(ids, groups)
        return [order, bk.adapter_matmul(X, A, B, offsets, order)]

    def backward():
        offsets, order, slots = bk.group_sort(ids, groups)
        return [order, *bk.adapter_matmul_grad(dY, X, A, B, offsets, order)]
    forward(), backward()
    torch.cuda.synchronize()
    graphs, results = [], []
    pool = torch.cuda.graph_pool_handle()
    for work in (forward, backward):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, pool=pool):
            results.append(work())
        graphs.append(graph)
    for turn in range(3):
        ids.copy_(torch.randint(-1, groups, (rows,), device="cuda", generator=g))
        X.normal_(generator=g)
        for graph, result, work in zip(graphs, results, (forward, backward)):
            graph.replay()
            for a, b in zip(result, work()):
                assert torch.equal(a, b)
