"""The hybrid verify step of examples/hybrid_step.py: rejected drafts leave no trace in either kind of layer."""

import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    spec = importlib.util.spec_from_file_location("hybrid_step", os.path.join(ROOT, "examples", "hybrid_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("cache", ["f16", "e4m3"])
def test_rejected_drafts_leave_no_trace(cuda, cache):
    h = example()
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    prompt = torch.randint(0, h.VOCAB, (300,), generator=g, device="cuda")
    a, b = h.HybridModel(cache=cache, max_tokens=500), h.HybridModel(cache=cache, max_tokens=500)
    for m in (a, b):
        m.prompt(prompt)
    # a verifies a block whose first 5 drafts are the model's own tokens (found one by one on a copy), then junk
    probe = h.HybridModel(cache=cache, max_tokens=500)
    probe.prompt(prompt)
    drafts = torch.randint(0, h.VOCAB, (h.T,), generator=g, device="cuda", dtype=torch.int32)
    for i in range(6):
        target, accepted = probe.verify(drafts)  # (states and cache move on by the accepted ones: start again each time)
        if i < 5:
            drafts[i] = target[i]
        else:
            drafts[5] = (target[5] + 1) % h.VOCAB
        probe = h.HybridModel(cache=cache, max_tokens=500)
        probe.prompt(prompt)
    target, accepted = a.verify(drafts)
    assert int(accepted) == 5 and int(a.kv_len) == 299 + 5
    # b verifies the same five and other junk behind them
    other = drafts.clone()
    other[5] = (target[5] + 2) % h.VOCAB
    other[6:] = (other[6:] + 7) % h.VOCAB
    _, accepted = b.verify(other)
    assert int(accepted) == 5 and int(b.kv_len) == 299 + 5
    # what follows is the same for both, bit for bit
    block = torch.randint(0, h.VOCAB, (h.T,), generator=g, device="cuda")
    assert torch.equal(a.last, b.last) and int(a.last) == int(drafts[4])
    x, y = a.forward(block, commit_all=False), b.forward(block, commit_all=False)
    assert torch.isfinite(x).all() and torch.equal(x, y)


def test_the_example_runs(cuda, capsys, monkeypatch):
    h = example()
    monkeypatch.setattr("sys.argv", ["hybrid_step.py", "--prompt", "200", "--steps", "2", "--cache", "e4m3"])
    h.main()
    assert capsys.readouterr().out.count("accepted") == 2
