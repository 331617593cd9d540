"""The hybrid verify step of examples/hybrid_step.py computes no norm that it does not read."""

import pytest
import torch

from tests.test_gpu_hybrid_step import example

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("layers", [1, 4])
def test_every_norm_is_read(cuda, monkeypatch, layers):
    """Without gates each layer reads one norm; and a norm that is changed changes the logits."""
    h = example()
    tokens = torch.randint(0, h.VOCAB, (20,), generator=torch.Generator().manual_seed(1)).cuda()
    real, calls, changed = h.dn.dn_residual_norm, [], []

    def norm(*args, **more):
        out, residual = real(*args, **more)
        calls.append(1)
        return (out * 2 if len(calls) in changed else out), residual

    monkeypatch.setattr(h.dn, "dn_residual_norm", norm)

    def logits():
        calls.clear()
        return h.HybridModel(layers=layers, max_tokens=200).forward(tokens, commit_all=True)

    want = logits()
    assert len(calls) == layers
    for i in range(layers):
        changed[:] = [i + 1]
        assert not torch.equal(logits(), want)
