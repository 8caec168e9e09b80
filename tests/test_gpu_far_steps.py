"""More steps than 32 bits count: what lies past a sequence's end is not written."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import linear_attention_recurrence_step_gb300 as gdn  # noqa: E402


def test_conv_of_more_steps_than_32_bits():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    if torch.cuda.get_device_properties(0).total_memory < 40e9:
        pytest.skip("needs a large device memory")
    gdn.load()
    T = (1 << 31) + 640
    dev = torch.device("cuda:0")
    x = torch.ones(1, T, 1, dtype=torch.bfloat16, device=dev)
    w = torch.zeros(1, 4, dtype=torch.bfloat16, device=dev)
    w[0, 3] = 2
    room = torch.full((T + 4096,), 5.0, dtype=torch.bfloat16, device=dev)
    y = room[:T].view(1, T, 1)
    for n in (7, T - 1):
        room.fill_(5.0)
        lens = torch.tensor([min(n, (1 << 31) - 1)], dtype=torch.int32, device=dev)
        out = gdn.gdn_causal_conv(x, w, lengths=lens, activation=None, y=y)
        n = int(lens)
        assert bool((room[:n] == 2).all()) and bool((room[n:] == 5).all())
        assert bool((out.state_out == 1).all())
