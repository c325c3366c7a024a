"""verify_drafts against its definition in 64 bits: everything it returns is whole and equal.

Sums in another order differ by about 2^-50 of the whole, the distance of a 24-bit
random number times the sum to the nearest border is 2^-24 / vocab on average, so inputs drawn
at random do not fall between.
"""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module")
def bk():
    from two_sided_gptq_amd import bakron
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    bakron.load()
    return bakron


def verify_plain(p, q, drafts, u, v):
    batch, n = drafts.shape
    accepted, tokens = [], torch.full((batch, n + 1), -1, dtype=torch.int64)
    vocab = p.shape[2]
    for b in range(batch):
        i, w = 0, None
        while i < n and drafts[b, i] >= 0:
            d = int(drafts[b, i])
            if d < vocab and float(u[b, i]) * (float(q[b, i, d]) if q is not None else 1.0) < float(p[b, i, d]):
                tokens[b, i] = d
                i += 1
                continue
            w = p[b, i].double().clone()
            if q is not None:
                w = (w - q[b, i].double()).clamp(min=0.0)
            elif d < vocab:
                w[d] = 0.0
            break
        if w is None or float(w.sum()) == 0.0:
            w = p[b, i].double()
        sums = w.cumsum(0)
        if float(sums[-1]) > 0.0:
            tokens[b, i] = int((sums <= float(v[b]) * float(sums[-1])).sum().clamp(max=vocab - 1))
        accepted.append(i)
    return torch.tensor(accepted, dtype=torch.int32), tokens


def case(batch, n, vocab, dtype, seed, draft=True, ragged=False, far=0.5):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(batch, n + 1, vocab, generator=g) * 2.0
    p = x.softmax(2).to(DT[dtype])
    drafts = torch.empty(batch, n, dtype=torch.int64)
    q = None
    if draft:
        q = (x[:, :n] + far * torch.randn(batch, n, vocab, generator=g)).softmax(2)
        if n:
            drafts = torch.multinomial(q.reshape(-1, vocab), 1, generator=g).view(batch, n)
        q = q.to(DT[dtype])
    elif n:
        drafts = torch.multinomial(p[:, :n].float().reshape(-1, vocab), 1, generator=g).view(batch, n)
    if ragged and n:
        drafts[torch.arange(n) >= torch.randint(0, n + 1, (batch, 1), generator=g)] = -1
    return p, q, drafts, torch.rand(batch, n, generator=g), torch.rand(batch, generator=g)


def cuda(*tensors):
    return tuple(None if t is None else t.cuda() for t in tensors)


def check(bk, inputs, status=None):
    accepted, tokens = bk.verify_drafts(*cuda(*inputs), dev_status=status)
    assert accepted.dtype == torch.int32 and tokens.dtype == torch.int64
    want_a, want_t = verify_plain(*inputs)
    assert torch.equal(accepted.cpu(), want_a) and torch.equal(tokens.cpu(), want_t)
    return accepted, tokens


SIZES = [(1, 4, 50001), (1, 1, 1), (2, 3, 2), (5, 5, 7), (3, 0, 1000), (3, 0, 20000), (64, 2, 1000), (65, 3, 513),
         (7, 64, 100), (2, 8, 16383), (2, 8, 16384), (63, 2, 16385), (64, 2, 16385), (1, 2, 131072), (4, 1, 300001)]


@pytest.mark.parametrize("batch,n,vocab", SIZES)
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("draft", [True, False])
def test_verify(bk, batch, n, vocab, dtype, draft):
    check(bk, case(batch, n, vocab, dtype, batch + n, draft))
    check(bk, case(batch, n, vocab, dtype, batch + n + 1, draft, ragged=True, far=3.0))


@pytest.mark.parametrize("batch,vocab", [(3, 900), (3, 20000), (70, 20000)])
@pytest.mark.parametrize("draft", [True, False])
def test_extreme_random_numbers(bk, batch, vocab, draft):
    for far in (0.0, 4.0):
        p, q, drafts, u, v = case(batch, 4, vocab, "f32", 7, draft, far=far)
        for uu, vv in ((0.0, 0.0), (1 - 2.0 ** -24, 1 - 2.0 ** -24), (0.0, 1 - 2.0 ** -24), (1 - 2.0 ** -24, 0.0)):
            check(bk, (p, q, drafts, torch.full_like(u, uu), torch.full_like(v, vv)))


@pytest.mark.parametrize("vocab", [300, 40000])
@pytest.mark.parametrize("batch", [2, 80])
def test_single_tokens_and_exact_borders(bk, batch, vocab):
    """Probabilities that are powers of two: sums are exact, a v on a border takes the next token."""
    n = 3
    p, q = torch.zeros(batch, n + 1, vocab), torch.zeros(batch, n, vocab)
    drafts = torch.full((batch, n), vocab - 1)
    place = [0, vocab // 3, vocab // 2, vocab - 1]
    p[:, :, place] = 0.25
    q[:, :, vocab - 1] = 1.0  # u < 1/4 accepts; the rest is a third each of the other three
    u = torch.full((batch, n), 0.25)
    u[:, 0] = 0.2499
    for k in range(4):
        v = torch.full((batch,), 0.25 * k)
        accepted, tokens = check(bk, (p, q, drafts, u, v))
        assert accepted.tolist() == [1] * batch
    u.fill_(0.125)
    for k in range(4):
        v = torch.full((batch,), 0.25 * k)
        accepted, tokens = check(bk, (p, q, drafts, u, v))
        assert accepted.tolist() == [n] * batch and tokens[:, n].tolist() == [place[k]] * batch
    # the whole weight on one token
    p.zero_()
    p[:, :, vocab // 2] = 1.0
    for k in range(4):
        accepted, tokens = check(bk, (p, q, drafts, u, torch.full((batch,), 0.25 * k)))
        assert accepted.tolist() == [0] * batch and tokens[:, 0].tolist() == [vocab // 2] * batch


@pytest.mark.parametrize("vocab", [300, 40000])
@pytest.mark.parametrize("batch", [2, 80])
def test_rows_without_weight(bk, batch, vocab):
    """No weight in max(p - q, 0): drawn from p.  No weight in p either: -1."""
    p, q = torch.zeros(batch, 3, vocab), torch.zeros(batch, 2, vocab)
    p[:, :, 5::7] = 0.01
    q[:, :, :] = 0.5
    drafts = torch.full((batch, 2), 5)
    u, v = torch.full((batch, 2), 0.9), torch.linspace(0.0, 0.99, batch)
    accepted, tokens = check(bk, (p, q, drafts, u, v))
    assert (tokens[:, 0] % 7 == 5).all()
    p[:, 0] = 0.0
    p[:, 0, 5] = 0.5
    accepted, tokens = check(bk, (p, None, drafts, u, v))
    assert (tokens[:, 0] == 5).all()
    p.zero_()
    for draft in (q, None):
        accepted, tokens = check(bk, (p, draft, drafts, u, v))
        assert accepted.sum() == 0 and (tokens == -1).all()


@pytest.mark.parametrize("batch", [3, 100])
def test_strided_rows(bk, batch):
    p, q, drafts, u, v = case(batch, 3, 20001, "bf16", 11)
    P = torch.full((batch, 4, 20040), 9.0, dtype=p.dtype, device="cuda")[:, :, 3:20004]
    Q = torch.full((batch, 3, 20017), 9.0, dtype=p.dtype, device="cuda")[:, :, :20001]
    P.copy_(p), Q.copy_(q)
    accepted, tokens = bk.verify_drafts(P, Q, *cuda(drafts, u, v))
    want = verify_plain(p, q, drafts, u, v)
    assert torch.equal(accepted.cpu(), want[0]) and torch.equal(tokens.cpu(), want[1])


@pytest.mark.parametrize("vocab", [100, 20000])
def test_values_that_are_not_finite(bk, vocab):
    for where in ("p", "q"):
        for value in (float("nan"), float("inf")):
            p, q, drafts, u, v = case(4, 3, vocab, "f32", 13, far=0.0)
            drafts[:] = 2
            u.fill_(0.9)
            q[1, 1] = p[1, 1] * 2.0  # request 1 refuses its second draft
            q[1, 1, 7] = 0.0
            want = verify_plain(p, q, drafts, u, v)
            (p if where == "p" else q)[1, 1, 7] = value
            status = torch.zeros(1, dtype=torch.int32, device="cuda")
            accepted, tokens = bk.verify_drafts(*cuda(p, q, drafts, u, v), dev_status=status)
            assert torch.equal(accepted.cpu(), want[0])
            keep = [0, 2, 3]
            assert torch.equal(tokens.cpu()[keep], want[1][keep])
            if where == "p" or value != value:
                assert status.item() == bk.DEV_NONFINITE and tokens[1].tolist() == [2, -1, -1, -1]
            else:  # p - inf is no weight
                assert torch.equal(tokens.cpu(), verify_plain(p, q, drafts, u, v)[1])
            # rows after the refusal are not read
            p, q, drafts, u, v = case(4, 3, vocab, "f32", 13, far=0.0)
            drafts[:] = 2
            u.fill_(0.9)
            q[1, 1] = p[1, 1] * 2.0
            q[1, 1, 7] = 0.0
            p[1, 2:] = float("nan")
            q[1, 2:] = float("nan")
            status.zero_()
            check(bk, (p, q, drafts, u, v), status)
            assert status.item() == 0


@pytest.mark.parametrize("vocab", [100, 20000])
@pytest.mark.parametrize("draft", [True, False])
def test_drafts_out_of_range(bk, vocab, draft):
    p, q, drafts, u, v = case(5, 3, vocab, "f32", 17, draft, far=0.0)
    u.fill_(0.0)
    drafts[1, 1], drafts[2, 0], drafts[3, 2] = vocab, 1 << 40, vocab + 5
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    accepted, tokens = check(bk, (p, q, drafts, u, v), status)
    assert accepted.tolist() == [3, 1, 0, 2, 3] and status.item() == bk.DEV_BAD_INDEX
    # behind the end of a request's drafts nothing is looked at
    drafts[1:4] = -1
    drafts[1, 2] = vocab
    status.zero_()
    check(bk, (p, q, drafts, u, v), status)
    assert status.item() == 0


def test_random_numbers_out_of_range(bk):
    """A v of 1 or more takes the last token that has weight; a negative or NaN one counts as 0."""
    p, q, drafts, u, v = case(6, 2, 500, "f32", 19)
    p[:, :, 400:] = 0.0
    p[:, :, :3] = 0.0
    drafts.fill_(-1)
    v[:] = torch.tensor([1.0, 7.5, float("inf"), -0.5, float("nan"), 0.0])
    accepted, tokens = bk.verify_drafts(*cuda(p, q, drafts, u, v))
    assert tokens[:, 0].tolist() == [399, 399, 399, 3, 3, 3]


def test_no_requests(bk):
    p, q, drafts, u, v = case(2, 3, 50, "f32", 23)
    accepted, tokens = bk.verify_drafts(*cuda(p[:0], q[:0], drafts[:0], u[:0], v[:0]))
    assert accepted.shape == (0,) and tokens.shape == (0, 4)


def test_offsets_beyond_32_bits(bk):
    vocab, n = 1 << 21, 2
    p = torch.zeros(380, n + 1, vocab, dtype=torch.float16, device="cuda")  # 2.4e9 elements, 4.8 GB
    for b in (0, 170, 379):
        p[b, 0, 5], p[b, 1, vocab - 3], p[b, 2, b], p[b, 2, vocab - 1 - b] = 0.5, 0.25, 0.5, 0.5
    drafts = torch.tensor([[5, vocab - 3]]).expand(380, 2).contiguous()
    u = torch.full((380, 2), 0.125)
    for v, last in ((0.25, lambda b: b), (0.75, lambda b: vocab - 1 - b)):
        accepted, tokens = bk.verify_drafts(p, None, *cuda(drafts, u, torch.full((380,), v)))
        for b in (0, 170, 379):
            assert accepted[b] == 2 and tokens[b].tolist() == [5, vocab - 3, last(b)]
        assert tokens[1].tolist() == [-1, -1, -1]


@pytest.mark.parametrize("batch", [3, 90])
def test_captured_and_replayed(bk, batch):
    inputs = cuda(*case(batch, 4, 20000, "f32", 29))
    bk.verify_drafts(*inputs)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = bk.verify_drafts(*inputs)
    for seed in (30, 31, 32):
        fresh = case(batch, 4, 20000, "f32", seed)
        for t, n in zip(inputs, fresh):
            t.copy_(n)
        graph.replay()
        torch.cuda.synchronize()
        want = bk.verify_drafts(*inputs)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert all(torch.equal(a.cpu(), b) for a, b in zip(got, verify_plain(*fresh)))


def test_another_stream(bk):
    inputs = cuda(*case(3, 4, 20000, "bf16", 33))
    want = bk.verify_drafts(*inputs)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = bk.verify_drafts(*inputs, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_refusals(bk):
    p, q, drafts, u, v = cuda(*case(4, 3, 60, "f32", 37))
    E = bk.BakronError
    for call in (lambda: bk.verify_drafts(p[:, :3], q, drafts, u, v), lambda: bk.verify_drafts(p, q[:, :2], drafts, u, v),
                 lambda: bk.verify_drafts(p, q.half(), drafts, u, v), lambda: bk.verify_drafts(p, q, drafts.int(), u, v),
                 lambda: bk.verify_drafts(p, q, drafts, u.half(), v), lambda: bk.verify_drafts(p, q, drafts, u, v[:3]),
                 lambda: bk.verify_drafts(p.cpu(), q, drafts, u, v), lambda: bk.verify_drafts(p.long(), q, drafts, u, v),
                 lambda: bk.verify_drafts(p[..., ::2], q[..., ::2], drafts, u, v),
                 lambda: bk.verify_drafts(p, q, drafts[0], u, v), lambda: bk.verify_drafts(p[::2], q[::2], drafts[::2], u, v)):
        with pytest.raises(E):
            call()
