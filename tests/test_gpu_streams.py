"""Calls on a stream given by object or by handle, while other work goes on in
the current one: the memory that a call allocates is its stream's own."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import linear_attention_recurrence_step_gb300 as gdn  # noqa: E402


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gdn.load()
    return torch.device("cuda:0")


@pytest.mark.parametrize("by_handle", [False, True])
def test_workspaces_of_another_stream(dev, by_handle):
    """Long calls wait on a side stream behind a delay of some milliseconds;
    meanwhile the current stream allocates blocks of the workspaces' sizes and
    writes over them again and again.  The results are those of calls by
    themselves."""
    gen = torch.Generator(device="cuda").manual_seed(11)
    B, T, H, P, G, N = 1, 2048, 4, 128, 2, 128
    bf = lambda *s: torch.randn(s, generator=gen, device=dev).bfloat16()  # noqa: E731
    x, dt, Bm, Cm = bf(B, T, H, P), bf(B, T, H), 0.3 * bf(B, T, G, N), 0.3 * bf(B, T, G, N)
    A = -torch.rand(H, generator=gen, device=dev) - 0.5
    k, v, g = 0.1 * bf(B, T, G, N), bf(B, T, H, P), torch.rand(B, T, H, generator=gen, device=dev).bfloat16()
    st = torch.zeros(B, H, P, N, device=dev)
    need = [gdn.gdn_selective_scan_workspace_size(B, T, H, P, N), gdn.gdn_chunk_prefill_workspace_size(B, T, H)]
    assert min(need) > 1 << 16
    torch.cuda.synchronize()
    want = [*gdn.gdn_selective_scan(x, dt, A, Bm, Cm, st), *gdn.gdn_chunk_prefill(k, k, v, g, g, st)[:2]]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    stream = side.cuda_stream if by_handle else side
    with torch.cuda.stream(side):
        torch.cuda._sleep(4_000_000)
    got = [*gdn.gdn_selective_scan(x, dt, A, Bm, Cm, st, stream=stream),
           *gdn.gdn_chunk_prefill(k, k, v, g, g, st, stream=stream)[:2]]
    assert not side.query()
    blocks = [torch.empty(n, dtype=torch.uint8, device=dev) for n in need * 2]
    for _ in range(100):
        for b in blocks:
            b.fill_(255)
    side.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    torch.cuda.synchronize()


def test_every_call_on_a_given_stream(dev):
    """Each call by stream object, by handle and by the default stream's handle:
    the bits of a call on the current stream."""
    gen = torch.Generator(device="cuda").manual_seed(12)
    x = torch.randn(2, 40, 128, generator=gen, device=dev).bfloat16()
    w = torch.randn(128, 4, generator=gen, device=dev).bfloat16()
    heads, dt = x.unflatten(-1, (2, 64)), x[..., :2].contiguous()
    bc = x[..., :64].unflatten(-1, (1, 64))
    noise = torch.empty(2, 40, 128, device=dev).exponential_(generator=gen)
    A = -torch.ones(2, device=dev)
    st = torch.zeros(2, 2, 64, 64, device=dev)

    def calls(**kw):
        rec = gdn.gdn_step_record(heads.contiguous(), heads.contiguous(), heads.contiguous(), dt.sigmoid(), dt.sigmoid(),
                                  st, capture_tape=True, **kw)
        return [*gdn.gdn_causal_conv(x, w, **kw), *gdn.gdn_selective_scan(heads, dt, A, bc, bc, **kw),
                *gdn.gdn_gated_norm(x, w[:, 0].contiguous(), residual=x, **kw),
                *gdn.gdn_sample(x, noise, top_k=5, **kw), *rec,
                gdn.gdn_state_replay(rec.delta_log, rec.k_log, rec.g_log, st, accepted=7, **kw)]

    want = calls()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream, 0, torch.cuda.default_stream()):
        side.wait_stream(torch.cuda.current_stream())
        got = calls(stream=stream)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
