"""The attention kernel for prompts waits on its own pipeline with a bound: when a
wait runs out the call's rows are NaN, the flag is raised, and the next call runs
normally."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import linear_attention_recurrence_step_gb300 as gdn  # noqa: E402


@pytest.fixture
def restore_hooks():
    yield
    gdn.inject_wait_expiry(False)
    gdn.set_wait_bound(0)


@pytest.mark.parametrize("D,T,L", [(128, 150, 150), (128, 150, 4000), (256, 70, 900), (64, 600, 700)])
def test_wait_expiry_is_reported(restore_hooks, D, T, L):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    dev = torch.device("cuda:0")
    g = torch.Generator(device=dev).manual_seed(1)
    H, G, page = 2, 3, 64
    width = -(-L // page)
    cache = gdn.gdn_kv_cache(width, H, page, D, device=dev)
    kv = torch.randn(1, L, 2, H, D, generator=g, device=dev).half()
    gdn.gdn_kv_append(kv[:, :, 0], kv[:, :, 1], torch.arange(L, dtype=torch.int32, device=dev)[None], cache)
    q = torch.randn(1, T, H * G, D, generator=g, device=dev).half()
    table = torch.arange(width, dtype=torch.int32, device=dev)[None]
    lengths = torch.tensor([L], dtype=torch.int32, device=dev)
    call = lambda: gdn.gdn_kv_attention(q, cache, table, lengths, return_lse=True)  # noqa: E731
    clean = call()
    torch.cuda.synchronize()
    assert not gdn.wait_status()
    gdn.set_wait_bound(1)
    gdn.inject_wait_expiry(True)
    bad = call()
    torch.cuda.synchronize()
    assert gdn.wait_status() and not gdn.wait_status()
    assert bool(bad.y.isnan().all()) and bool(bad.lse.isnan().all())
    gdn.inject_wait_expiry(False)
    gdn.set_wait_bound(0)
    again = call()
    torch.cuda.synchronize()
    assert not gdn.wait_status()
    assert torch.equal(again.y, clean.y) and torch.equal(again.lse, clean.lse)
