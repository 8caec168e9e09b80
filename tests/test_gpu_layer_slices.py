"""The operators around the recurrence on slices and other orders of wider
tensors: the bits of the same call on dense copies."""
from __future__ import annotations

import pytest

from gdn_testutil import torch_dtype

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import linear_attention_recurrence_step_gb300 as gdn  # noqa: E402


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gdn.load()
    return torch.device("cuda:0")


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("lead,D,wide,first", [((7,), 512, 576, 0), ((7,), 512, 576, 64), ((2, 5), 200, 333, 8),
                                               ((2, 5), 77, 99, 3), ((1,), 64, 80, 5), ((3,), 9001, 9009, 1),
                                               ((300,), 4096, 6144, 2048)])
def test_norm_rows_of_a_projection(dev, dtype, lead, D, wide, first):
    gen = torch.Generator(device="cuda").manual_seed(D)
    full = lambda: torch.randn(*lead, wide, generator=gen, device=dev).to(torch_dtype(dtype))  # noqa: E731
    x, gate = full()[..., first:first + D], full()[..., first:first + D]
    w, res = full().flatten()[:D].clone(), torch.randn(*lead, D, generator=gen, device=dev).to(x.dtype)
    for kw in (dict(), dict(gate=gate), dict(gate=gate.contiguous()), dict(gate=gate, gate_first=True, residual=res)):
        dense = {k: v.contiguous() if isinstance(v, torch.Tensor) else v for k, v in kw.items()}
        for a in (x, x.contiguous()):
            got = gdn.gdn_gated_norm(a, w, **kw)
            want = gdn.gdn_gated_norm(x.contiguous(), w, **dense)
            # (rows that start on other boundaries may sum their squares in another order)
            assert (got.y.float() - want.y.float()).abs().max() <= 2.0 ** -7 * want.y.float().abs().max()
            if "residual" in kw:
                assert torch.equal(got.residual_out, want.residual_out)
            if not (D * x.element_size() % 16 or wide * x.element_size() % 16 or first * x.element_size() % 16):
                assert torch.equal(got.y, want.y)
