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


@pytest.mark.parametrize("T,C,dtype", [(1, 64, "bf16"), (9, 96, "f32"), (70, 33, "f16"), (300, 256, "bf16")])
def test_steps_before_sequences(dev, T, C, dtype):
    """x, dt, B and C laid out [T,B,...]: the convolution and both forms of the
    scan."""
    gen = torch.Generator(device="cuda").manual_seed(T)
    B = 3
    mk = lambda *inner: torch.randn(T, B, *inner, generator=gen, device=dev).to(torch_dtype(dtype)).transpose(0, 1)  # noqa: E731
    lens = torch.tensor([T, T // 2, 0], dtype=torch.int32, device=dev)
    x, w = mk(C), torch.randn(C, 4, generator=gen, device=dev).to(torch_dtype(dtype))
    a, b = (gdn.gdn_causal_conv(t, w, lengths=lens) for t in (x, x.contiguous()))
    on = torch.arange(T, device=dev) < lens[:, None]
    assert torch.equal(a.y[on], b.y[on]) and torch.equal(a.state_out, b.state_out)
    H, P, N = 2, 64, 64
    ins = (mk(H, P), mk(H), -torch.rand(H, generator=gen, device=dev), mk(1, N), mk(1, N))
    a, b = (gdn.gdn_selective_scan(*(t.contiguous() if dense else t for t in ins), lengths=lens) for dense in (False, True))
    assert torch.equal(a.y[on], b.y[on]) and torch.equal(a.state_out, b.state_out)
