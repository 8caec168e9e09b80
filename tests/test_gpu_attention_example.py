"""The attention layer's operators at work together: speculative steps of the
layer in examples/, and their rollback."""
from __future__ import annotations

import os
import sys

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import speculative_attention as ex  # noqa: E402


def test_speculative_steps_roll_back():
    """A layer that wrote and rejected drafts gives the logits of one that never saw
    them: the same values in other pages, so the same bits."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    dev = torch.device("cuda:0")
    layer, plain = ex.AttentionLayer(dev), ex.AttentionLayer(dev)
    g = torch.Generator(device=dev).manual_seed(5)
    prompt = torch.randint(0, 512, (4, 200), generator=g, device=dev)
    lengths = torch.tensor([200, 16, 33, 0], dtype=torch.int32, device=dev)
    for m in (layer, plain):
        _, granted = m.forward(prompt, lengths)
        assert granted.tolist() == [200, 16, 33, 0]
    for step in range(5):
        draft = torch.randint(0, 512, (4, 7), generator=g, device=dev)
        noise = torch.empty(4, 7, 512, device=dev).exponential_(generator=g)
        token, accepted = ex.speculative_step(layer, draft, noise, temperature=0.7)
        assert bool((accepted >= 1).all()) and bool((accepted <= 7).all())
        plain.forward(draft, accepted)
        assert torch.equal(layer.lengths, plain.lengths)
        assert ex.rollback_error(layer, plain, token[:, :1].long()) == 0.0
    # a request ends and its pages serve another one
    end = torch.tensor([-1, 1, 1, 1], dtype=torch.int32, device=dev)
    for m in (layer, plain):
        m.forward(token[:, :1].long(), end)
        assert int(m.lengths[0]) == 0 and int(m.held[0]) == 0
    assert ex.rollback_error(layer, plain, token[:, :1].long()) == 0.0
