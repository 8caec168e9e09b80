"""The attention layer's operators where a call is unusual and still allowed."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import linear_attention_recurrence_step_gb300 as gdn  # noqa: E402
from test_gpu_attention import dev  # noqa: E402, F401


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rotary_with_one_in_place(dev, layout):  # noqa: F811
    """q or k turned in place in wider rows, the other one read from the same rows and
    written elsewhere: the bits of a call with outputs of its own."""
    g = torch.Generator(device=dev).manual_seed(6)
    wide = torch.randn(2, 9, 7, 64, generator=g, device=dev).bfloat16()
    pos = torch.randint(0, 9000, (2, 9), generator=g, device=dev, dtype=torch.int32)
    inv, scale = gdn.rotary_frequencies(32, device=dev)
    parts = lambda w: (w[:, :, :4], w[:, :, 4:6])  # noqa: E731
    q, k = parts(wide)
    plain = gdn.gdn_rotary(q, pos, inv, k=k, layout=layout, scale=scale)
    for which in (0, 1):
        w = wide.clone()
        q, k = parts(w)
        o = gdn.gdn_rotary(q, pos, inv, k=k, layout=layout, scale=scale, **{("q_out", "k_out")[which]: (q, k)[which]})
        assert torch.equal(o.q, plain.q) and torch.equal(o.k, plain.k)
        other = parts(w)[1 - which]
        assert torch.equal(other, parts(wide)[1 - which]) and torch.equal(w[:, :, 6], wide[:, :, 6])
