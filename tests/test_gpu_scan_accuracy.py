"""What the tensor-core form of the selective scan loses before y is rounded,
on calls whose terms cancel so that it shows, against what the header states."""
from __future__ import annotations

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import linear_attention_recurrence_step_gb300 as gdn  # noqa: E402

N, P = 64, 16


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gdn.load()
    return torch.device("cuda:0")


def states_alone(dev, states):
    """y of 32 steps that change nothing, with C taking the difference of the
    state's first two columns: states [P,2] f64."""
    st = torch.zeros(1, 1, P, N, device=dev)
    st[0, 0, :, :2] = torch.from_numpy(states).to(dev)
    assert np.array_equal(st[0, 0, :, :2].double().cpu().numpy(), states)
    z = torch.zeros(1, 32, 1, P, device=dev, dtype=torch.bfloat16)
    C = torch.zeros(1, 32, 1, N, device=dev, dtype=torch.bfloat16)
    C[..., 0], C[..., 1] = 1, -1
    out = gdn.gdn_selective_scan(z, z[..., 0], torch.full((1,), -1.0, device=dev), torch.zeros_like(C), C, st, softplus=False)
    assert torch.equal(out.state_out, st)
    return out.y[0, :, 0].double().cpu().numpy()


def rounded(v):
    """Half a unit of a bf16 value of this size."""
    return 2.0 ** (np.floor(np.log2(np.maximum(np.abs(v), 1e-30))) - 8)


def test_the_states_part(dev):
    """State entries that lie halfway between two of what is left of them: off by
    2^-17 of each, no more."""
    rng = np.random.default_rng(1)
    states = 1 + 2.0 ** -9 + rng.integers(0, 256, (P, 2)) * 2.0 ** -17
    states[0] = 1 + 2.0 ** -9 + np.array([1, 3]) * 2.0 ** -17
    want = states[:, 0] - states[:, 1]
    y = states_alone(dev, states)
    assert (np.abs(y - want) <= 2.0 ** -17 * np.abs(states).sum(1) + rounded(want)).all()


@pytest.mark.parametrize("seed", range(3))
def test_the_steps_part(dev, seed):
    """y from the steps of one chunk alone, with inputs of both signs whose sums
    are small beside their terms: as near as float32 sums are."""
    rng = np.random.default_rng(seed)
    T = 32
    x = np.repeat(rng.standard_normal((T // 2, P)), 2, 0)
    x[1::2] *= -1                                            # each step undoes the one before
    x = torch.from_numpy(x.astype(np.float32)).bfloat16()
    Bm, Cm = (torch.from_numpy(rng.uniform(0.5, 1, (T, N)).astype(np.float32)).bfloat16() for _ in range(2))
    dt = torch.full((T,), 0.75).bfloat16()
    x64, B64, C64 = (t.double().numpy() for t in (x, Bm, Cm))
    c = np.cumsum(np.full(T, 0.75 * -2.0 ** -6))             # exact
    W = np.tril((C64 @ B64.T) * np.exp(c[:, None] - c[None]) * 0.75) + 3.0 * np.eye(T)
    want, size = W @ x64, np.abs(W) @ np.abs(x64)
    out = gdn.gdn_selective_scan(x.view(1, T, 1, P).to(dev), dt.view(1, T, 1).to(dev), torch.full((1,), -2.0 ** -6, device=dev),
                                 Bm.view(1, T, 1, N).to(dev), Cm.view(1, T, 1, N).to(dev), D=torch.full((1,), 3.0, device=dev),
                                 softplus=False)
    y = out.y[0, :, 0].double().cpu().numpy()
    # f32 sums of 64 and 32 terms, an exponential and three products
    assert (np.abs(y - want) <= 24 * 2.0 ** -24 * size + rounded(np.maximum(np.abs(want), np.abs(y)))).all()
