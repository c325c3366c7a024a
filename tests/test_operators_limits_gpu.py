"""The operators for rounded layers at the largest sizes that they accept: more
threads in all than one launch can hold (2^32)."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def bk():
    from two_sided_gptq_amd import bakron
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    bakron.load()
    yield bakron
    torch.cuda.empty_cache()


def test_codes_beyond_one_launch(bk):
    """2^36 codes and a row more: 64 GiB in, 64 GiB out."""
    m, n = (1 << 18) + 1, 1 << 18
    codes = torch.zeros((m, n), dtype=torch.int8, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(3)
    spots = (0, 1 << 16, (1 << 17) + 1, (1 << 18) - 2, (1 << 18) - 1, 1 << 18)
    for r in spots:
        codes[r] = torch.randint(-8, 8, (n,), device="cuda", generator=g, dtype=torch.int8)
    out = torch.empty((m, n), dtype=torch.uint8, device="cuda")
    q = bk.fp8_from_codes(codes, out=out.view(torch.float8_e4m3fn))
    for r in spots:
        assert torch.equal(q[r].float(), codes[r].float()), r
    del codes, out, q
    torch.cuda.empty_cache()
