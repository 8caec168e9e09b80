"""The selective scan at the ends of its decays, in the tensor-core form and by
steps, for calls that end inside a chunk."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import linear_attention_recurrence_step_gb300 as gdn  # noqa: E402

INF = float("inf")


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gdn.load()
    return torch.device("cuda:0")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T", [1, 4, 32, 33, 40, 300])
def test_a_rate_of_minus_infinity(dev, T, dtype):
    """A = -inf forgets everything at each step, also where a sequence's steps
    end inside a chunk (the steps past the end have no size)."""
    x = torch.ones(2, T, 2, 64, device=dev, dtype=dtype)
    dt = torch.full((2, T, 2), 2.0, device=dev, dtype=dtype)
    Bm = torch.ones(2, T, 1, 64, device=dev, dtype=dtype)
    A = torch.tensor([-INF, -1e38], device=dev)
    st = torch.full((2, 2, 64, 64), 3.0, device=dev)
    lens = torch.tensor([T, T // 2], dtype=torch.int32, device=dev)
    out = gdn.gdn_selective_scan(x, dt, A, Bm, Bm, st, softplus=False, lengths=lens, y=torch.zeros_like(x))
    want = torch.full_like(st, 2.0)
    if T == 1:
        want[1] = 3.0
    assert torch.equal(out.state_out, want)
    assert bool((out.y[0] == 128).all()) and bool((out.y[1, :T // 2] == 128).all())
