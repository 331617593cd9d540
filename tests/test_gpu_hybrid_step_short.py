"""The hybrid example's shortest prompts."""

import pytest

from tests.test_gpu_hybrid_step import example

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cache", ["f16", "e4m3"])
@pytest.mark.parametrize("prompt", [1, 2])
def test_the_example_runs_on_short_prompts(cuda, capsys, monkeypatch, prompt, cache):
    h = example()
    monkeypatch.setattr("sys.argv", ["hybrid_step.py", "--prompt", str(prompt), "--steps", "2", "--cache", cache])
    h.main()
    assert capsys.readouterr().out.count("accepted") == 2


def test_the_example_refuses_no_prompt(cuda, monkeypatch):
    monkeypatch.setattr("sys.argv", ["hybrid_step.py", "--prompt", "0"])
    with pytest.raises(SystemExit):
        example().main()
