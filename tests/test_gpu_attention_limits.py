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


def filled(dev, pages, H, page, D, seed, dtype=torch.bfloat16):  # noqa: F811
    """A cache of `pages` pages of normal values, and as it stands its keys and values."""
    g = torch.Generator(device=dev).manual_seed(seed)
    cache = gdn.gdn_kv_cache(pages, H, page, D, device=dev)
    kv = torch.randn(1, pages * page, 2, H, D, generator=g, device=dev).to(dtype)
    kv[:, :, 0, :, 5] = -kv[:, :, 0, :, 5].abs() - 1  # (one channel of the keys has one sign)
    gdn.gdn_kv_append(kv[:, :, 0], kv[:, :, 1], torch.arange(pages * page, device=dev, dtype=torch.int32)[None], cache)
    return cache, g


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("T,L", [(1, 1), (1, 2), (2, 2), (1, 300), (70, 70), (70, 71), (150, 150), (150, 2000)])
@pytest.mark.parametrize("scale,window", [(0.1, 0), (-0.1, 1), (0.0, 2)])
def test_infinite_queries_of_few_tokens(dev, dtype, D, T, L, scale, window):  # noqa: F811
    """A row that holds an infinity is NaN whatever the scores' sign, when it sees one
    token or many; the others are what they were, and one that sees nothing stays 0.

    Rows of a warp move their softmax reference together, so without one of them the
    others' weights may be rounded elsewhere.  Their scores keep their bits: per call a
    weight is off by 2^-12 (f16; float32 calls 2^-23), by 2^-18 from the difference to
    the reference and its power, and L/16 sums by 2^-23 each, together 2^-16: below
    2^-11.5 (float32: 2^-15) of the largest value, which is at most 6 of normal ones.
    Twice that, and a rounding of each y; log-sum-exps below 2^6 twice by 2^-17."""
    H, G, page = 2, 2, 16
    cache, g = filled(dev, -(-L // page), H, page, D, T)
    q = torch.randn(1, T, H * G, D, generator=g, device=dev).to(dtype)
    table = torch.arange(-(-L // page), device=dev, dtype=torch.int32)[None]

    def call(q, n):
        return gdn.gdn_kv_attention(q, cache, table, torch.tensor([n], device=dev, dtype=torch.int32), scale=scale,
                                    window=window, return_lse=True)

    clean = call(q, L)
    assert not bool(clean.y.isnan().any())
    bad = torch.zeros(1, T, H * G, dtype=torch.bool, device=dev)
    for i, t in enumerate({0, min(1, T - 1), T - 1}):
        for h, x in ((i, float("inf")), (3, -float("inf"))):
            q[0, t, h, 5], bad[0, t, h] = x, True
    o = call(q, L)
    assert bool(o.y[bad].isnan().all()) and bool(o.lse[bad].isnan().all())
    by = 6 * 2.0 ** (-14 if dtype == torch.float32 else -10.5) + torch.finfo(dtype).eps * clean.y.double().abs()
    assert bool(((o.y.double() - clean.y.double()).abs() <= by)[~bad].all())
    assert bool(((o.lse - clean.lse).abs() <= 2.0 ** -16)[~bad].all())
    if T > 1:  # one token less: the first row sees none
        o = call(q, T - 1)
        assert bool((o.y[0, 0] == 0).all()) and bool((o.lse[0, 0] == -float("inf")).all())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 2, 1 << 30])
@pytest.mark.parametrize("T,lengths", [(9, [4, 0, 9, 300, 5]), (70, [2, 0, 70, 69, 1000]), (300, [2, 299, 700, 1, 0])])
def test_largest_windows(dev, dtype, window, T, lengths):  # noqa: F811
    """A window past every token is none, also for sequences with fewer tokens than
    queries, whose first ones stand before the first token."""
    H, G, page, D = 2, 2, 32, 64
    width = 32
    cache, g = filled(dev, width, H, page, D, T)
    B = len(lengths)
    q = torch.randn(B, T, H * G, D, generator=g, device=dev).to(dtype)
    table = torch.arange(width, device=dev, dtype=torch.int32).expand(B, -1).contiguous()
    at = torch.tensor(lengths, device=dev, dtype=torch.int32)
    want = gdn.gdn_kv_attention(q, cache, table, at, return_lse=True)
    got = gdn.gdn_kv_attention(q, cache, table, at, window=window, return_lse=True)
    assert torch.equal(got.y, want.y) and torch.equal(got.lse, want.lse)
    for b, n in enumerate(lengths):  # rows that see a token are not empty
        seen = torch.arange(T, device=dev) >= T - n
        assert torch.equal(got.lse[b].isfinite().all(-1), seen) and torch.equal((got.y[b] != 0).flatten(1).any(-1), seen)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("B,T,G,H,L", [
    (2, 1, 4, 2, 500), (2, 3, 5, 2, 500), (120, 1, 3, 8, 60), (70, 5, 2, 8, 60),   # few rows: cut, whole
    (2, 70, 1, 2, 500), (2, 99, 2, 2, 500), (2, 67, 1, 2, 4000), (1, 150, 2, 1, 4000)])  # tiles: whole, cut
def test_rows_at_odd_addresses(dev, dtype, D, B, T, G, H, L):  # noqa: F811
    """Queries whose rows begin at odd elements, and outputs that do, give the bits of
    dense ones; nothing beside the outputs is written."""
    page = 64
    width = -(-L // page)
    cache, g = filled(dev, width, H, page, D, L)
    q = torch.randn(B, T, H * G, D, generator=g, device=dev).to(dtype)
    table = torch.arange(width, device=dev, dtype=torch.int32).expand(B, -1).contiguous()
    lengths = torch.randint(1, L + 1, (B,), generator=g, device=dev, dtype=torch.int32)
    lengths[0] = L
    new = torch.randint(0, T + 1, (B,), generator=g, device=dev, dtype=torch.int32)
    new[0] = T
    on = torch.arange(T, device=dev) < new[:, None]
    want = gdn.gdn_kv_attention(q, cache, table, lengths, new=new, y=torch.full_like(q, 7.0))
    n = q.numel()
    # a slice that begins one element into rows with odd strides; a y one element behind a boundary
    wide = torch.full((B, T + 1, H * G * D + 33), float("nan"), device=dev, dtype=dtype)
    odd = wide[:, :T, 1:H * G * D + 1].unflatten(-1, (H * G, D))
    odd.copy_(q)
    assert odd.data_ptr() % 16 != 0 and (T == 1 or odd.stride(1) % 2 == 1)
    for x in (q, odd):
        flat = torch.full((n + 18,), 7.0, device=dev, dtype=dtype)
        y = flat[1:1 + n].view(q.shape)
        assert y.data_ptr() % 16 != 0
        gdn.gdn_kv_attention(x, cache, table, lengths, new=new, y=y)
        assert torch.equal(y, want.y) and bool((y[~on] == 7.0).all())
        assert bool((flat[:1] == 7.0).all()) and bool((flat[1 + n:] == 7.0).all())
    assert torch.equal(gdn.gdn_kv_attention(odd, cache, table, lengths, new=new, y=torch.full_like(q, 7.0)).y, want.y)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("B,T,G,L", [(2, 1, 7, 4000), (2, 2, 7, 1500), (120, 1, 7, 150), (2, 11, 7, 700), (2, 20, 7, 4000),
                                     (1, 30, 7, 4000)])
def test_scores_of_any_size(dev, dtype, D, sign, B, T, G, L):  # noqa: F811
    """Rows whose scores reach from ones to 1e37 side by side, the best ones below 0 and
    above, on three tokens far apart: the softmax of the exact scores.

    A row's scores are one size times 1, 2, 4 or 8, so from 1e3 on all but the best weigh
    nothing and a score's own error moves nothing.  Weights are off by 2^-12 (f16) or 2^-23, and
    at scores of at most 8 by twice 8 40 2^-23 + 2^-20 < 2^-13; values are at most 6.
    Log-sum-exps are off by a few roundings of the score."""
    H, page, at = 8 if B > 2 else 2, 32, torch.tensor([3, L // 2, L - T - 5])
    g = torch.Generator().manual_seed(D + L)
    k, v = torch.zeros(1, L, H, D), torch.randn(1, L, H, D, generator=g)
    best, other = ((-1, (-2, -4)), (-8, (-2, -4)))[sign < 0]
    k[0, :, :, 5] = torch.tensor(other)[torch.randint(0, 2, (L, H), generator=g)].float()
    k[0, at, :, 5] = float(best)
    width = -(-L // page)
    cache = gdn.gdn_kv_cache(width, H, page, D, device=dev)
    slots = torch.arange(L, device=dev, dtype=torch.int32)
    gdn.gdn_kv_append(k.to(dev), v.to(dev), slots[None], cache)
    kr, vr = (t.double().cpu() for t in gdn.gdn_kv_read(cache, slots, dtype=torch.float32))
    sizes = torch.tensor([1.0, 1e3, 1e6, 1e9, 1e20, 1e30, 1e37])
    q = torch.zeros(B, T, H * G, D)
    q[..., 5] = sign * sizes.repeat(H)
    q = q.to(dtype)
    table = torch.arange(width, device=dev, dtype=torch.int32).expand(B, -1).contiguous()
    o = gdn.gdn_kv_attention(q.to(dev), cache, table, torch.full((B,), L, device=dev, dtype=torch.int32), scale=1.0,
                             return_lse=True)
    b = B - 1
    assert torch.equal(o.y, o.y[:1].expand_as(o.y)) or B <= 2
    x = torch.einsum("thgd,lhd->thgl", q[b].double().unflatten(1, (H, G)), kr)
    x = x.masked_fill((torch.arange(L) > L - T + torch.arange(T)[:, None])[:, None, None], -float("inf"))
    want, lse = torch.einsum("thgl,lhd->thgd", x.softmax(-1), vr).flatten(1, 2), x.logsumexp(-1).flatten(1, 2)
    by = 6 * (2.0 ** -11 if dtype != torch.float32 else 0.0) + 6 * 2.0 ** -13 + torch.finfo(dtype).eps * want.abs()
    assert bool(((o.y[b].cpu().double() - want).abs() <= by).all()), float((o.y[b].cpu().double() - want).abs().max())
    assert bool(((o.lse[b].cpu().double() - lse).abs() <= lse.abs() * 2.0 ** -20 + 2.0 ** -12).all())


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("D,B,T,G,H", [(128, 16, 17, 4, 8), (128, 29, 64, 4, 8), (256, 16, 17, 4, 8), (64, 29, 50, 4, 8),
                                       (128, 25, 64, 4, 4)])  # whole units, and parts of 43690 tokens
@pytest.mark.parametrize("drift", [0.0, 12.0])
def test_sums_over_long_contexts(dev, dtype, D, B, T, G, H, drift):  # noqa: F811
    """131072 tokens whose values have one sign: sums that only grow, where every unit cut
    off is seen.

    Beside the weights' 2^-12 and twice the scores' 40 2^-23 of sum |q k| and 2^-20 (as in
    attention_bounds), a sum is off by 2^-23 at each addition to it since it was last set
    down: 16384/16 and 16 more, below 2^-13 + 2^-19.  The outputs' rounding goes either
    way: in the mean over 8704 and more of them it leaves 2^-16 at most (five standard
    deviations of 2^-11 / sqrt(3 8704))."""
    L, page = 131072, 128
    g = torch.Generator(device=dev).manual_seed(D + B)
    cache = gdn.gdn_kv_cache(L // page, H, page, D, device=dev)
    at = torch.arange(L, device=dev, dtype=torch.int32)
    for i in range(0, L, 16384):
        k, v = (torch.randn(1, 16384, H, D, generator=g, device=dev) for _ in range(2))
        k[0, :, :, 5] += drift * at[i:i + 16384, None] / L  # (later tokens weigh more: the reference moves)
        gdn.gdn_kv_append(k, v.abs() + 1, at[None, i:i + 16384], cache)
    q = (0.05 * torch.randn(B, T, H * G, D, generator=g, device=dev))
    q[..., 5] = 1.0
    q = q.to(dtype)
    table = torch.arange(L // page, device=dev, dtype=torch.int32).expand(B, -1).contiguous()
    lengths = torch.full((B,), L, device=dev, dtype=torch.int32)
    flat = torch.full((q.numel() + 8,), 7.0, device=dev, dtype=dtype)
    o = gdn.gdn_kv_attention(q, cache, table, lengths, scale=1.0, return_lse=True)
    for b, h in ((0, 0), (B - 1, H - 1)):
        keys, vals = (t[:, h].double() for t in gdn.gdn_kv_read(cache, at, dtype=torch.float32))
        rows = q[b, :, h * G:(h + 1) * G].double().reshape(-1, D)
        x = rows @ keys.T
        pos = L - T + torch.arange(T, device=dev).repeat_interleave(G)
        x = x.masked_fill(torch.arange(L, device=dev) > pos[:, None], -float("inf"))
        want, lse = x.softmax(-1) @ vals, x.logsumexp(-1)
        size = rows.norm(dim=-1).max() * keys.norm(dim=-1).max()
        ds = float(size) * 40 * 2.0 ** -23 + 2.0 ** -20
        err = o.y[b, :, h * G:(h + 1) * G].double().reshape(-1, D) - want
        by = want * (2.0 ** -12 + 2.0 ** -13 + 2.0 ** -19 + 2 * ds + torch.finfo(dtype).eps / 2) + vals.sum(0) * 2.0 ** -31
        assert bool((err.abs() <= by).all()), float((err.abs() - by).max())
        if dtype == torch.float16:
            assert abs(float((err / want).mean())) <= 2.0 ** -13 + 2.0 ** -19 + 2.0 ** -16 + 2.0 ** -20
        assert bool(((o.lse[b, :, h * G:(h + 1) * G].double().reshape(-1) - lse).abs() <= ds + lse.abs() * 2.0 ** -22).all())
    # y at an odd address: the same bits, nothing beside it
    y = flat[1:1 + q.numel()].view(q.shape)
    gdn.gdn_kv_attention(q, cache, table, lengths, scale=1.0, y=y)
    assert torch.equal(y, o.y) and bool((flat[:1] == 7.0).all()) and bool((flat[1 + q.numel():] == 7.0).all())


@pytest.mark.parametrize("T", [17, 50])
def test_rows_of_long_contexts(dev, T):  # noqa: F811
    """Over 40000 tokens: a row with an infinity, rows that are not there, a window that
    ends before the last sums are set down, sequences of other lengths."""
    H, G, D, page, B, L = 8, 4, 128, 128, 29, 40000
    width = -(-L // page)
    cache, g = filled(dev, width, H, page, D, T)
    q = torch.randn(B, T, H * G, D, generator=g, device=dev).half()
    q[1, 2, 3, 7], q[2, T - 1, 0, 0] = float("inf"), float("nan")
    table = torch.arange(width, device=dev, dtype=torch.int32).expand(B, -1).contiguous()
    lengths = torch.randint(0, L + 1, (B,), generator=g, device=dev, dtype=torch.int32)
    new = torch.randint(0, T + 1, (B,), generator=g, device=dev, dtype=torch.int32)
    lengths[:4], new[:4] = L, T
    new[3] = T - 3
    for window in (0, 20000):
        y = torch.full_like(q, 7.0)
        o = gdn.gdn_kv_attention(q, cache, table, lengths, new=new, window=window, y=y, return_lse=True)
        bad = torch.zeros(B, T, H * G, dtype=torch.bool, device=dev)
        bad[1, 2, 3] = bad[2, T - 1, 0] = True
        assert torch.equal(y.isnan().all(-1), bad) and torch.equal(y.isnan().any(-1), bad)
        on = torch.arange(T, device=dev) < new[:, None]
        assert bool((y[~on] == 7.0).all())
        # rows in calls of 16 tokens' worth of few rows: the other kernel
        for b, t in ((0, 0), (0, T - 1), (3, T - 4), (1, 5)):
            n = lengths[b:b + 1] - new[b] + t + 1
            one = gdn.gdn_kv_attention(q[b:b + 1, t:t + 1], cache, table[b:b + 1], n.int(), window=window, return_lse=True)
            # values of at most 6, two calls each off by 2^-12 of the weights, 2^-13 of the sums
            # and 2^-13 of the scores, and rounded
            by = 6 * 2 * (2.0 ** -12 + 2.0 ** -12) + 2.0 ** -10 * one.y.float().abs()
            assert bool(((one.y.float() - y[b:b + 1, t:t + 1].float()).abs() <= by).all())
            assert bool(((one.lse - o.lse[b:b + 1, t:t + 1]).abs() <= 2.0 ** -12).all())


@pytest.mark.parametrize("dtype,L", [(torch.float16, 262144), (torch.bfloat16, 2 ** 21)])
@pytest.mark.parametrize("D,B,G,H", [(64, 120, 4, 8), (128, 95, 4, 8), (256, 60, 4, 8), (64, 77, 12, 8), (128, 58, 12, 8),
                                     (256, 39, 12, 8), (128, 90, 4, 8)])  # units that are whole, and one call that is cut
def test_sums_of_few_rows(dev, dtype, L, D, B, G, H):  # noqa: F811
    """Values of one sign over more tokens than the tensor cores' own sums are good for.

    As in test_sums_over_long_contexts, with sums that are added outside: L/64 terms to a
    warp, each time by half a unit, 2^-24, either way, so 2^-24 sqrt(L/64 / 3) in the mean
    and five times that at most, below 2^-14.  The pages repeat, so the softmax is that over
    the first ones."""
    n, page = 8192, 128
    g = torch.Generator(device=dev).manual_seed(D + B)
    cache = gdn.gdn_kv_cache(n // page, H, page, D, device=dev)
    at = torch.arange(n, device=dev, dtype=torch.int32)
    k, v = (torch.randn(1, n, H, D, generator=g, device=dev) for _ in range(2))
    gdn.gdn_kv_append(k, v.abs() + 1, at[None], cache)
    q = (0.05 * torch.randn(B, 1, H * G, D, generator=g, device=dev)).to(dtype)
    table = (torch.arange(L // page, device=dev, dtype=torch.int32) % (n // page)).expand(B, -1).contiguous()
    lengths = torch.full((B,), L, device=dev, dtype=torch.int32)
    o = gdn.gdn_kv_attention(q, cache, table, lengths, scale=1.0, return_lse=True)
    mean = []
    for b, h in ((0, 0), (B // 2, 3), (B - 1, H - 1)):
        keys, vals = (t[:, h].double() for t in gdn.gdn_kv_read(cache, at, dtype=torch.float32))
        rows = q[b, 0, h * G:(h + 1) * G].double()
        x = rows @ keys.T
        want, lse = x.softmax(-1) @ vals, x.logsumexp(-1) + torch.log(torch.tensor(L / n, dtype=torch.float64))
        ds = float(rows.norm(dim=-1).max() * keys.norm(dim=-1).max()) * 40 * 2.0 ** -23 + 2.0 ** -20
        err = o.y[b, 0, h * G:(h + 1) * G].double() - want
        by = want * (2.0 ** -12 + 2.0 ** -14 + 2 * ds + torch.finfo(dtype).eps / 2) + vals.sum(0) * (L / n) * 2.0 ** -31
        assert bool((err.abs() <= by).all()), float((err.abs() - by).max())
        assert bool(((o.lse[b, 0, h * G:(h + 1) * G].double() - lse).abs() <= ds + lse.abs() * 2.0 ** -22).all())
        mean.append((err / want).flatten())
    mean = torch.cat(mean)
    # the outputs' rounding: five standard deviations of their mean
    assert abs(float(mean.mean())) <= 2.0 ** -14 + 5 * torch.finfo(dtype).eps / 2 / (3 * mean.numel()) ** 0.5


@pytest.mark.parametrize("B,H", [(29, 8), (25, 4)])  # whole units, parts
def test_waits_of_long_contexts(dev, B, H):  # noqa: F811
    """Waits that run out where sums are set down: NaN, the flag, and the next call runs."""
    T, G, D, page, L = 50, 4, 64, 128, 65536
    cache, g = filled(dev, L // page, H, page, D, 1)
    q = torch.randn(B, T, H * G, D, generator=g, device=dev).half()
    table = torch.arange(L // page, device=dev, dtype=torch.int32).expand(B, -1).contiguous()
    lengths = torch.full((B,), L, device=dev, dtype=torch.int32)
    call = lambda: gdn.gdn_kv_attention(q, cache, table, lengths, return_lse=True)  # noqa: E731
    clean = call()
    torch.cuda.synchronize()
    assert not gdn.wait_status()
    gdn.set_wait_bound(1)
    gdn.inject_wait_expiry(True)
    try:
        bad = call()
        torch.cuda.synchronize()
    finally:
        gdn.inject_wait_expiry(False)
        gdn.set_wait_bound(0)
    assert gdn.wait_status() and not gdn.wait_status()
    assert bool(bad.y.isnan().all()) and bool(bad.lse.isnan().all())
    again = call()
    assert torch.equal(again.y, clean.y) and torch.equal(again.lse, clean.lse) and bool(again.y.isfinite().all())
