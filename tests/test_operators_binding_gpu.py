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
