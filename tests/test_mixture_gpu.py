"""The example of a rounded mixture layer: its run, its forward pass against 64 bits, and its
gradients against autograd's in 64 bits."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mixture():
    from two_sided_gptq_amd import bakron, mixture
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    bakron.load()
    return mixture


def plain(X, experts, weights, W, adapters):
    of, A, B, scale = adapters
    out = torch.zeros(X.shape[0], W.shape[1], dtype=torch.float64)
    for j in range(experts.shape[1]):
        for e in range(W.shape[0]):
            rows = (experts[:, j] == e)[:, None]
            out = out + torch.where(rows, weights[:, j:j + 1] * (X @ W[e].t()), 0.0)
    for r in range(A.shape[0]):
        out = out + torch.where((of == r)[:, None], scale[r] * (X @ A[r].t() @ B[r].t()), 0.0)
    return out


def test_forward_and_gradients(mixture):
    """bf16 roundings of half a step (2^-8) lie between inputs and results: of the experts' products,
    the way back and the sum with the adapter's part forward, of as many and one more backward;
    each is taken relative to the norm of what it rounds."""
    X, gate, W, W8, scales, adapters = mixture.example(experts=5, tokens=300, width=128, requests=10)
    experts, weights = mixture.route(X, gate, 2)
    assert experts.shape == (300, 2) and (weights.sum(1) - 1).abs().max() < 1e-6
    out, kept = mixture.forward_original(X, experts, weights, W, adapters)
    dout = torch.randn(out.shape, device="cuda", generator=torch.Generator("cuda").manual_seed(3)).bfloat16()
    dX, dweights, dW, dA, dB = mixture.backward(dout, X, weights, W, kept, adapters)
    x, p, w, a, b = (t.detach().double().cpu().requires_grad_() for t in (X, weights, W, adapters[1], adapters[2]))
    want = plain(x, experts.cpu(), p, w, (adapters[0].cpu(), a, b, adapters[3].double().cpu()))
    want.backward(dout.double().cpu())
    assert (out.double().cpu() - want).norm() <= 3 * 2.0 ** -8 * want.norm()
    for got, ref in ((dX, x.grad), (dweights, p.grad), (dW, w.grad), (dA, a.grad), (dB, b.grad)):
        assert (got.double().cpu() - ref).norm() <= 4 * 2.0 ** -8 * ref.norm()


def test_rounded_layer(mixture):
    """The layer's product with the rounded weights' values, from activations rounded to fp8 (half a step
    is 2^-4 of a value; the errors of a sum's terms are independent, so of its norm too)."""
    X, gate, W, W8, scales, adapters = mixture.example(experts=5, tokens=300, width=128, requests=10)
    experts, weights = mixture.route(X, gate, 2)
    out = mixture.forward(X, experts, weights, W8, scales, adapters)
    values = (W8.double() * scales.double()[:, :, None]).cpu()
    want = plain(X.double().cpu(), experts.cpu(), weights.double().cpu(), values,
                 (adapters[0].cpu(), adapters[1].double().cpu(), adapters[2].double().cpu(), adapters[3].double().cpu()))
    assert (out.double().cpu() - want).norm() <= (2.0 ** -4 + 3 * 2.0 ** -8) * want.norm()


def test_drafts(mixture):
    g = torch.Generator("cuda").manual_seed(5)
    p = torch.rand(20, 4, 300, device="cuda", generator=g).softmax(2)
    drafts, accepted, tokens = mixture.verify(p, p[:, :3].contiguous(), g)
    assert (accepted == 3).all() and torch.equal(tokens[:, :3], drafts)  # u < 1: the same model keeps all
    drafts, accepted, tokens = mixture.verify(p, p.flip(2)[:, :3].contiguous(), g)
    for r in range(20):
        n = int(accepted[r])
        assert torch.equal(tokens[r, :n], drafts[r, :n]) and 0 <= int(tokens[r, n]) < 300 and (tokens[r, n + 1:] == -1).all()


def test_example_runs(mixture, monkeypatch, capsys):
    monkeypatch.setattr("sys.argv", ["mixture", "--tokens", "128", "--width", "128", "--requests", "8", "--experts", "4"])
    mixture.main()
    assert "drafts kept" in capsys.readouterr().out
