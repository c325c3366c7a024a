"""What the binding of the operators for rounded layers takes and refuses on a GPU."""
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


def test_vectors_of_another_gpu_are_refused(bk, monkeypatch):
    """Offsets, scales, targets and the like: with another GPU current, as matrices are."""
    v = torch.zeros(4, device="cuda")
    assert bk._vector(v, "v", torch.float32, (4,)) == v.data_ptr()
    monkeypatch.setattr(bk, "_device", lambda: 1)
    with pytest.raises(bk.BakronError, match="current GPU"):
        bk._vector(v, "v", torch.float32, (4,))
    monkeypatch.undo()
    with pytest.raises(bk.BakronError, match="current GPU"):
        bk._vector(torch.zeros(4), "v", torch.float32, (4,))


@pytest.mark.parametrize("groups", [1, 3])
def test_no_rows(bk, groups):
    """A rank without tokens: outputs of 0 rows, gradients of weights that are 0."""
    N, K, vocab = 24, 130, 1000
    x = torch.zeros(0, K, device="cuda", dtype=torch.bfloat16)
    w = torch.ones(groups, N, K, device="cuda", dtype=torch.bfloat16)
    off = torch.zeros(groups + 1, dtype=torch.int32, device="cuda")
    for br in (1, 128):
        q, s = bk.fp8_quantize(x, block_rows=br)
        assert q.shape == (0, K) and q.dtype == torch.float8_e4m3fn and s.shape == (2, 0)
    w8, sw = bk.fp8_quantize(w.view(-1, K))
    w8, q, s = w8.view(groups, N, K), *bk.fp8_quantize(x)
    y = bk.fp8_matmul(q, s, w8, torch.ones(groups, N, device="cuda"), off, out_dtype=torch.float16)
    assert y.shape == (0, N) and y.dtype == torch.float16
    assert bk.grouped_matmul(x, w, off, out_dtype=torch.float32).shape == (0, N)
    given = torch.empty(0, N, device="cuda", dtype=torch.bfloat16)
    assert bk.grouped_matmul(x, w, off, out=given) is given
    dx, dw = bk.grouped_matmul_grad(given, x, w, off, w_dtype=torch.float32)
    assert dx.shape == (0, K) and dw.shape == w.shape and dw.dtype == torch.float32 and bool((dw == 0).all())
    for dtype in (torch.float32, torch.bfloat16):
        logits, t = torch.zeros(0, vocab, device="cuda", dtype=dtype), torch.zeros(0, device="cuda", dtype=torch.int64)
        r = bk.token_logprobs(logits, t, top=5)
        assert r["logprob"].shape == r["lse"].shape == r["entropy"].shape == (0,)
        assert r["top_ids"].shape == r["top_logprob"].shape == (0, 5)
        d = bk.token_logprobs_grad(logits, t, r["lse"], r["entropy"], r["lse"], r["lse"])
        assert d.shape == (0, vocab) and d.dtype == dtype
    # on another stream, and what else does not fit is still refused
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    _, dw = bk.grouped_matmul_grad(given, x, w, off, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert bool((dw == 0).all())
    for call in (lambda: bk.grouped_matmul(x[:, :0], w[..., :0], off), lambda: bk.grouped_matmul(x, w[:, :0], off),
                 lambda: bk.fp8_quantize(x[:, :0]), lambda: bk.token_logprobs(logits, t[:0].float()),
                 lambda: bk.grouped_matmul(x, w, off, out=torch.empty(1, N, device="cuda", dtype=torch.bfloat16))):
        with pytest.raises(bk.BakronError):
            call()


def test_groups_of_one_row(bk):
    """Weights of one row a group: the stride inside a group means nothing, the groups' is
    the distance between rows."""
    g = torch.Generator().manual_seed(2)
    full = torch.randn(5, 4, 64, generator=g).bfloat16().cuda()
    x = torch.randn(40, 64, generator=g).bfloat16().cuda()
    off = torch.tensor([0, 8, 16, 16, 30, 40], dtype=torch.int32, device="cuda")
    for w in (full[:, :1], full[:, 2:3], full[:, 0].contiguous().unsqueeze(0).transpose(0, 1)):
        assert w.shape == (5, 1, 64)
        assert torch.equal(bk.grouped_matmul(x, w, off), bk.grouped_matmul(x, w.clone(memory_format=torch.contiguous_format), off))
        dy = torch.ones(40, 1, device="cuda", dtype=torch.bfloat16)
        a, b = bk.grouped_matmul_grad(dy, x, w, off), bk.grouped_matmul_grad(dy, x, w.clone(memory_format=torch.contiguous_format), off)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    with pytest.raises(bk.BakronError, match="rows apart"):
        bk.grouped_matmul(x, full[:, :2], off)
