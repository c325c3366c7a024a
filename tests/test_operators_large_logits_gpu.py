"""Log probabilities where lse is so large that log s does not show in
it: rows of a type's lowest value (a mask that leaves nothing) and logits far from 0.

Tolerances, fixed before the first run.  A thread adds at most 275 terms of s here, and its
sums pass about 10 merges, so s is off by less than 2^-15 of itself; x - m is exact (the
logits are multiples of 1/64, and a power of two more) or rounds once:
  log probabilities, entropy: 2^-15 (1 + |log p|) and (1 + entropy)
"""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
E = 2.0 ** -15


@pytest.fixture(scope="module")
def bk():
    from two_sided_gptq_amd import bakron
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    bakron.load()
    return bakron


def exact(x):
    """log p, with -inf where there is no token, and the entropy, both in 64 bits."""
    x = x.double()
    d = x - x.amax(1, keepdim=True)
    e = d.exp()
    s = e.sum(1, keepdim=True)
    return d - s.log(), (s.log() - torch.where(e > 0, e * d, 0).sum(1, keepdim=True) / s)[:, 0]


def check(bk, x, k):
    rows, vocab = x.shape
    g = torch.Generator().manual_seed(rows + vocab)
    t = torch.randint(0, vocab, (rows,), generator=g)
    t[1::3] = -1
    f = bk.token_logprobs(x.cuda(), t.cuda(), top=k)
    lp, ent = exact(x)
    at = torch.where(t < 0, 0.0, lp.gather(1, t.clamp(min=0)[:, None])[:, 0])
    got = f["logprob"].double().cpu()
    assert bool(((got == at) | ((got - at).abs() <= E * (1 + at.abs()))).all())  # masked targets have -inf
    assert bool(((f["entropy"].double().cpu() - ent).abs() <= E * (1 + ent)).all())
    v, i = torch.sort(lp, dim=1, descending=True, stable=True)
    assert torch.equal(f["top_ids"].cpu(), i[:, :k])
    assert bool(((f["top_logprob"].double().cpu() - v[:, :k]).abs() <= E * (1 + v[:, :k].abs())).all())


# many rows: a workgroup each; few: split
@pytest.mark.parametrize("rows,vocab", [(5, 17), (520, 1000), (3, 70000), (515, 8193)])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_rows_of_the_lowest_value(bk, rows, vocab, dtype):
    x = torch.full((rows, vocab), torch.finfo(DT[dtype]).min, dtype=DT[dtype])
    x[2::4, vocab // 2:] = -torch.inf  # and some of them masked for good
    check(bk, x, 5)


@pytest.mark.parametrize("rows,vocab", [(5, 17), (520, 1000), (3, 70000), (515, 8193)])
@pytest.mark.parametrize("shift", [1024.0, -4096.0, 65536.0, -131072.0])
def test_logits_far_from_zero(bk, rows, vocab, shift):
    g = torch.Generator().manual_seed(vocab)
    x = torch.round(torch.randn(rows, vocab, generator=g) * 3 * 64) / 64 + shift
    x[:, 3] += 8
    check(bk, x, 5)
