"""The operators around the recurrence at work together: one speculative step
of the small hybrid model in examples/, and its rollback."""
from __future__ import annotations

import os
import sys

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import speculative_hybrid as ex  # noqa: E402


def test_speculative_step_rolls_back():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    dev = torch.device("cuda:0")
    model = ex.HybridModel(dev, vocab=512, d_model=256)
    B, T = 5, 7
    prompt = torch.randint(0, 512, (B, 90), generator=model.gen, device=dev)
    _, state, _ = model.forward(prompt, model.new_state(B))
    draft = torch.randint(0, 512, (B, T), generator=model.gen, device=dev)
    # sequence b's draft follows the greedy continuation for b tokens
    for t in range(1, T):
        guess = model.forward(draft[:, :t], state)[0][:, -1].float().argmax(-1)
        on = torch.arange(B, device=dev) >= t
        draft[:, t] = torch.where(on, guess, (guess + 1) % 512)
    noise = torch.ones(B, T, 512, device=dev)
    before = {n: s.clone() for n, s in state.items()}
    token, accepted, rolled = ex.speculative_step(model, draft, state, noise, temperature=0.0)
    assert accepted.tolist() == [1, 2, 3, 4, 5]
    assert all(torch.equal(state[n], before[n]) for n in state)   # the snapshot is as it was
    err = ex.rollback_error(model, draft, accepted, state, rolled)
    # the convolutions' states are copies, the scan's the same call; the tape is
    # rounded to bf16: seven steps of 2^-9 of |delta| k, both below 2
    assert err["gdn_conv"] == 0 and err["ssm_conv"] == 0 and err["ssm"] == 0
    assert err["gdn"] < 7 * 2.0 ** -9 * 2


def test_prompt_in_pieces():
    """A prompt in one call and in two that hand the states on: the same states
    to rounding of the activations between the layers."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    dev = torch.device("cuda:0")
    model = ex.HybridModel(dev, vocab=512, d_model=256)
    prompt = torch.randint(0, 512, (2, 100), generator=model.gen, device=dev)
    logits, whole, _ = model.forward(prompt, model.new_state(2))
    _, state, _ = model.forward(prompt[:, :63], model.new_state(2))
    tail, state, _ = model.forward(prompt[:, 63:], state)
    assert torch.equal(state["gdn_conv"], whole["gdn_conv"])
    for n in ("gdn", "ssm"):
        assert float((state[n] - whole[n]).abs().max()) < 0.02 * float(whole[n].abs().max())
    assert float((tail - logits[:, 63:]).float().abs().max()) < 0.05 * float(logits.float().abs().max())
