"""gdn_sample's cuts together: top-p narrows what top-k left and brings nothing
back, for one block per row and for clusters, in all three types."""
from __future__ import annotations

import numpy as np
import pytest

import layer_reference as ref
from gdn_testutil import torch_dtype
from sample_cases import TIED_CUTS, tied_cut

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
@pytest.mark.parametrize("name", list(TIED_CUTS))
def test_top_p_stays_inside_top_k(dev, name, dtype):
    """A token that top-k removed by its index stays out, however top-p ends:
    rows of other orders, a few (over clusters) and many (one block each)."""
    rows = [tied_cut(name, seed) for seed in range(4)]
    want = [ref.sample(l, noise, **s)[0] for l, s, noise in rows]
    for copies in (1, 50):
        pick = [i for i in range(4) for _ in range(copies)]
        l = torch.from_numpy(np.stack([rows[i][0] for i in pick])).to(torch_dtype(dtype)).to(dev)
        noise = torch.from_numpy(np.stack([rows[i][2] for i in pick])).to(dev)
        s = {k: torch.tensor([rows[i][1][k] for i in pick], device=dev,
                             dtype=torch.int32 if k == "top_k" else torch.float32) for k in rows[0][1]}
        out = gdn.gdn_sample(l, noise, **s)
        assert out.token.tolist() == [want[i] for i in pick]
