"""What the example of a mixture layer refuses before it uses a GPU."""
import pytest

from two_sided_gptq_amd import mixture


@pytest.mark.parametrize("argv,word", [
    (["--tokens", "100", "--requests", "16"], "100 tokens"), (["--tokens", "16", "--requests", "16"], "16 tokens"),
    (["--requests", "0"], "requests"), (["--experts", "2", "--choices", "3"], "3 of 2 experts"), (["--choices", "0"], "experts")])
def test_arguments_that_do_not_fit(monkeypatch, capsys, argv, word):
    monkeypatch.setattr("sys.argv", ["mixture", *argv])
    monkeypatch.setattr(mixture, "example", lambda *a, **k: pytest.fail("not refused"))
    with pytest.raises(SystemExit) as end:
        mixture.main()
    assert end.value.code == 2 and word in capsys.readouterr().err
