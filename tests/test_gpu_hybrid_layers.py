"""Recurrent layers and an attention layer over the same tokens: the tokens that
page slots grant are the lengths of both, and the same counts roll both back."""
from __future__ import annotations

import os
import sys

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import speculative_attention as attention  # noqa: E402
import speculative_hybrid as recurrent  # noqa: E402


def test_layers_roll_back_together():
    """Drafts, some rejected, some refused for want of pages: states and cache are those
    of layers that never saw the rejected tokens, and a refused sequence's are untouched."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    dev = torch.device("cuda:0")
    model = recurrent.HybridModel(dev, vocab=512, d_model=256)
    layer, plain = attention.AttentionLayer(dev, pages=23), attention.AttentionLayer(dev)
    B, T = 4, 7
    g = torch.Generator(device=dev).manual_seed(3)
    prompt = torch.randint(0, 512, (B, 200), generator=g, device=dev)
    lengths = torch.tensor([200, 16, 33, 0], dtype=torch.int32, device=dev)
    state = model.new_state(B)
    _, granted = layer.forward(prompt, lengths)
    assert torch.equal(granted, lengths) and torch.equal(plain.forward(prompt, lengths)[1], lengths)
    _, state, _ = model.forward(prompt, state, lengths=granted)
    refused = 0
    for step in range(10):
        draft = torch.randint(0, 512, (B, T), generator=g, device=dev)
        _, granted = layer.forward(draft)
        _, _, keep = model.forward(draft, state, lengths=granted)
        accepted = torch.minimum(torch.randint(1, T + 1, (B,), generator=g, device=dev).int(), granted)
        layer.shorten(granted - accepted)
        rolled = model.roll_back(state, keep, accepted)
        err = recurrent.rollback_error(model, draft, accepted, state, rolled)
        # the convolutions' states are copies, the scan's the same call; the tape is
        # rounded to bf16: seven steps of 2^-9 of |delta| k, both below 2
        assert err["gdn_conv"] == 0 and err["ssm_conv"] == 0 and err["ssm"] == 0
        assert err["gdn"] < 7 * 2.0 ** -9 * 2
        out = granted == 0
        refused += int(out.sum())
        assert all(torch.equal(rolled[n][out], state[n][out]) for n in state)
        state = rolled
        assert torch.equal(plain.forward(draft, accepted)[1], accepted)
        assert torch.equal(layer.lengths, plain.lengths)
        # one more token for each: the same values in other pages, so the same bits
        nxt = draft[:, :1]
        a, granted = layer.forward(nxt)
        b, _ = plain.forward(nxt, granted)
        on = granted > 0
        refused += int((~on).sum())
        assert torch.equal(a[on], b[on]) and torch.equal(layer.lengths, plain.lengths)
        _, state, _ = model.forward(nxt, state, lengths=granted)
    assert refused > 0
