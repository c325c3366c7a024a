"""Calls on a stream that is not torch's current one: whatever a call allocates comes from
that stream's memory, where nothing of another stream can still be at work."""
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


def stream_of(address):
    """The stream whose memory holds this address, by torch's allocator."""
    for s in torch.cuda.memory_snapshot():
        if s["address"] <= address < s["address"] + s["total_size"]:
            return s["stream"]
    raise AssertionError("not allocated by torch")


def calls(bk):
    g = torch.Generator().manual_seed(1)
    x = torch.randn(300, 4096, generator=g).bfloat16().cuda()
    w = torch.randn(3, 130, 4096, generator=g).bfloat16().cuda()
    dy = torch.randn(300, 130, generator=g).bfloat16().cuda()
    off = torch.tensor([0, 100, 100, 300], dtype=torch.int32, device="cuda")
    x8, sx = bk.fp8_quantize(x)
    w8, sw = bk.fp8_quantize(w.view(390, 4096), block_rows=128)
    codes = torch.randint(-8, 8, (64, 96), generator=g, dtype=torch.int8).cuda()
    logits, t = torch.randn(4, 70000, generator=g).cuda(), torch.tensor([1, 2, 3, 4], device="cuda")
    f = bk.token_logprobs(logits, t)
    one = torch.ones(4, device="cuda")
    return {
        "fp8_quantize": lambda s: bk.fp8_quantize(x, stream=s),
        "fp8_from_codes": lambda s: bk.fp8_from_codes(codes, stream=s),
        "fp8_matmul": lambda s: bk.fp8_matmul(x8, sx, w8, sw, stream=s),
        "grouped_matmul": lambda s: bk.grouped_matmul(x, w, off, stream=s),
        "grouped_matmul_grad": lambda s: bk.grouped_matmul_grad(dy, x, w, off, stream=s),
        "token_logprobs": lambda s: bk.token_logprobs(logits, t, top=5, stream=s),
        "token_logprobs_grad": lambda s: bk.token_logprobs_grad(logits, t, f["lse"], f["entropy"], one, one, stream=s),
    }


@pytest.mark.parametrize("name", ["fp8_quantize", "fp8_from_codes", "fp8_matmul", "grouped_matmul", "grouped_matmul_grad",
                                  "token_logprobs", "token_logprobs_grad"])
def test_memory_of_another_stream(bk, name, monkeypatch):
    call = calls(bk)[name]
    want = call(None)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    spaces, space = [], bk._space
    monkeypatch.setattr(bk, "_space", lambda *a: spaces.append(space(*a)) or spaces[-1])
    got = call(side)
    assert torch.cuda.current_stream() != side
    flat = lambda r: [t for t in (r.values() if isinstance(r, dict) else r if isinstance(r, tuple) else (r,)) if t is not None]
    for t in flat(got) + [s for s in spaces if s is not None]:
        assert stream_of(t.data_ptr()) == side.cuda_stream
    if name in ("fp8_matmul", "grouped_matmul", "token_logprobs"):
        assert any(s is not None for s in spaces)  # these have a workspace here
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(flat(want), flat(got)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
