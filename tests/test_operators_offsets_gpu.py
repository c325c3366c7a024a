"""The operators for rounded layers where element offsets pass 32 bits.

Operands of more than 2^31 elements or 2^32 bytes; the parts that lie beyond are
compared with the formula in 64 bits.  Tolerances, fixed before the first run, are
those of sums in fp32 with one rounding of the output: products (R + 8) 2^-23 of the
sum of magnitudes, fp8 products 2^-12 of it; bf16 outputs 2^-8 of the value; log
probabilities 2^-20 (1 + |lse| + max |x|); their gradient 2^-20 (1 + |x| + |lse|) p
and the output's rounding.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

BF16, F8 = torch.bfloat16, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def bk():
    from two_sided_gptq_amd import bakron
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    bakron.load()
    yield bakron
    torch.cuda.empty_cache()


def noise(shape, seed, dtype=BF16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(generator=g)


def e4m3(shape, seed):
    """Finite codes only: a magnitude below 0x7f and a sign."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    c = torch.empty(shape, dtype=torch.uint8, device="cuda").random_(0, 256, generator=g)
    for part in c.view(-1).split(1 << 30):
        part.masked_fill_((part & 0x7f) == 0x7f, 0)
    return c.view(F8)


def near(got, want, mass, share, rounding=2.0 ** -8):
    bad = (got.double() - want).abs() > share * mass + rounding * want.abs()
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} values are off"


def offsets_of(counts):
    return torch.tensor([0, *counts], dtype=torch.int64).cumsum(0).to(torch.int32).cuda()


@pytest.mark.parametrize("rows", [40, 9000], ids=["few", "many"])
def test_weights_of_many_experts(bk, rows):
    groups, n, k = 72, 8192, 4096           # 2.4e9 elements, 4.8 GB
    W = noise((groups, n, k), 1)
    counts = [0] * groups
    counts[0], counts[-1] = rows // 4, rows - rows // 4
    off, X = offsets_of(counts), noise((rows, k), 2)
    Y = bk.grouped_matmul(X, W, off)
    dX, _ = bk.grouped_matmul_grad(Y, X, W, off, want_w=False)
    x, y, w = X[rows // 4:][:64].double(), Y[rows // 4:][:64], W[-1].double()
    near(y, x @ w.T, x.abs() @ w.abs().T, (k + 8) * 2.0 ** -23)
    y = y.double()
    near(dX[rows // 4:][:64], y @ w, y.abs() @ w.abs(), (n + 8) * 2.0 ** -23)


def test_gradient_of_many_experts(bk):
    groups, n, k, rows = 72, 8192, 4096, 720
    X, dY = noise((rows, k), 3), noise((rows, n), 4)
    off = offsets_of([10] * groups)
    W = torch.empty((groups, n, k), dtype=BF16, device="cuda")
    _, dW = bk.grouped_matmul_grad(dY, X, W, off, want_x=False)
    for g in (0, 65, 71):
        a, b = dY[10 * g:10 * g + 10].double(), X[10 * g:10 * g + 10].double()
        near(dW[g], a.T @ b, a.abs().T @ b.abs(), 18 * 2.0 ** -23)


@pytest.mark.parametrize("rows", [60, 9000], ids=["few", "many"])
def test_fp8_weights_of_many_experts(bk, rows):
    groups, n, k = 136, 8192, 4096          # 4.6 GB
    W = e4m3((groups, n, k), 5)
    X, sx = bk.fp8_quantize(noise((rows, k), 6))
    sw = noise((groups, k // 128, n // 128), 7, torch.float32).abs() + 0.1
    counts = [0] * groups
    counts[3], counts[-1] = rows // 4, rows - rows // 4
    Y = bk.fp8_matmul(X, sx, W, sw, offsets_of(counts))
    at = slice(rows // 4, rows // 4 + 40)
    x = X[at].float().double() * sx[:, at].double().repeat_interleave(128, 0).T
    w = W[-1].float().double() * sw[-1].double().repeat_interleave(128, 0).repeat_interleave(128, 1).T
    near(Y[at], x @ w.T, x.abs() @ w.abs().T, 2.0 ** -12)


@pytest.mark.parametrize("ld", [1 << 20, (1 << 20) + 1, 1 << 21], ids=["whole chunks", "odd", "long rows"])
def test_rows_far_apart(bk, ld):
    rows, n, k = 4400, 520, 264             # the last row begins past 2^32 elements, or past 2^33 bytes
    full = torch.empty(rows * ld, dtype=BF16, device="cuda")
    X, Y = full.as_strided((rows, k), (ld, 1)), full.as_strided((rows, n), (ld, 1), 1024)
    X.copy_(noise((rows, k), 8))
    W = noise((1, n, k), 9)
    bk.grouped_matmul(X, W, out=Y)
    for at in (slice(0, 50), slice(rows - 300, rows)):
        x, w = X[at].double(), W[0].double()
        near(Y[at], x @ w.T, x.abs() @ w.abs().T, (k + 8) * 2.0 ** -23)
    dX, dW = bk.grouped_matmul_grad(Y, X, W)
    y, x, w = Y.double(), X.double(), W[0].double()
    near(dX, y @ w, y.abs() @ w.abs(), (n + 8) * 2.0 ** -23)
    near(dW[0], y.T @ x, y.abs().T @ x.abs(), (rows + 8) * 2.0 ** -23)


def test_log_probabilities(bk):
    rows, vocab = 33000, 131072             # 4.3e9 logits
    x = noise((rows, vocab), 10)
    t = torch.arange(rows, device="cuda") * 7919 % vocab
    r = bk.token_logprobs(x, t, top=3)
    g, h = noise((rows,), 11, torch.float32), noise((rows,), 12, torch.float32)
    at = slice(rows - 8, rows)
    e, ta = x[at].double(), t[at]
    lse = e.logsumexp(1)
    lp = e - lse[:, None]
    p = lp.exp()
    ent = -(p * lp).sum(1)
    tol = 2.0 ** -20 * (1 + lse.abs() + e.abs().amax(1))
    at_t = lp.gather(1, ta[:, None])[:, 0]
    for name, want in (("lse", lse), ("logprob", at_t), ("entropy", ent)):
        assert ((r[name][at].double() - want).abs() <= tol).all(), name
    best, ids = (e - torch.arange(vocab, device="cuda") * 1e-9).topk(3, 1)  # equal values: the lowest token
    assert torch.equal(r["top_ids"][at], ids)
    d = bk.token_logprobs_grad(x, t, r["lse"], r["entropy"], g, h)[at].double()
    hit = torch.zeros_like(p).scatter_(1, ta[:, None], 1.0)
    gd, hd = g[at].double()[:, None], h[at].double()[:, None]
    want = gd * (hit - p) - hd * p * (lp + ent[:, None])
    rel = 2.0 ** -20 * (1 + e.abs() + lse.abs()[:, None])
    slack = rel * p * (gd.abs() + hd.abs() * (2 + lp.abs() + ent[:, None])) + 2.0 ** -23 * gd.abs() * hit
    assert ((d - want).abs() <= slack + 2.0 ** -8 * want.abs()).all()


def test_quantisation(bk):
    rows, cols = 66000, 65544               # 4.3e9 elements
    x = noise((rows, cols), 13)
    q, s = bk.fp8_quantize(x)
    a = x[-3:, -136:].float().cpu().numpy()  # the last whole block and the narrow one

    def same(codes, scales, a, amax):
        """fp32 steps in numpy: its divisions round once."""
        assert np.array_equal(scales.cpu().numpy(), amax / np.float32(448))
        want = np.clip(a * (np.float32(448) / amax)[..., None], -448, 448).astype(np.float32)
        assert torch.equal(codes.cpu().view(torch.uint8), torch.from_numpy(want).to(F8).view(torch.uint8))

    same(q[-3:, -136:-8], s[-2, -3:], a[:, :128], np.abs(a[:, :128]).max(1))
    same(q[-3:, -8:], s[-1, -3:], a[:, 128:], np.abs(a[:, 128:]).max(1))
    del q, s
    q, s = bk.fp8_quantize(x, block_rows=128)
    amax = x[65920:, -136:-8].abs().amax().float().cpu().numpy()
    same(q[-3:, -136:-8], s[-2, -1], a[:, :128], amax)
