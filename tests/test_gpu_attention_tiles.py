"""Attention of many query rows: units of one tile and of two, whole and cut along
their tokens, where a mask, a page, a score or a row is unusual."""
from __future__ import annotations

import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import attention_reference as ref  # noqa: E402
import linear_attention_recurrence_step_gb300 as gdn  # noqa: E402
from test_gpu_attention import attend_case, dev, ints, make_cache  # noqa: E402, F401


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("T,Hq,window", [(13, 5, 0), (32, 4, 0), (33, 2, 50), (43, 3, 700), (64, 4, 1)])
def test_rows_of_one_and_two_tiles(dev, dtype, D, T, Hq, window):  # noqa: F811
    """65 to 256 rows over a few tokens, none of their own, and enough to be cut."""
    attend_case(dev, dtype, 3, T, Hq, 1, D, 16, [2500, 0, T + 1], [T, T, T - 5], window, seed=T)


@pytest.mark.parametrize("D", [64, 128])
def test_many_sequences_of_few_rows(dev, D):  # noqa: F811
    attend_case(dev, "bf16", 40, 7, 14, 2, D, 32, [(37 * i) % 400 for i in range(40)], [(i % 9) for i in range(40)], seed=D)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("T", [20, 50])
def test_sharp_scores_of_tiles(dev, dtype, T):  # noqa: F811
    """Scores of hundreds (one token takes all), tiny ones, scales of zero and below."""
    for sharp, scale in ((40.0, 0.5), (1e-6, 1.0), (1.0, 0.0), (3.0, -0.3)):
        attend_case(dev, dtype, 2, T, 8, 2, 128, 16, [1400, 77], seed=5, sharp=sharp, scale=scale)


@pytest.mark.parametrize("T", [20, 50])
def test_bad_pages_of_tiles(dev, T):  # noqa: F811
    """Entries that name no page take their tokens out of sight, all of them too.

    A probability is rounded to f16 (2^-11 of itself) and its score is off by at most
    64 2^-24 sum |q k| / 8, below 2^-13 where that sum is at most 256; numerator and
    denominator both see the latter: weights are off by 2^-11 + 2^-12 < 2^-10, y by as
    much of sum w |v| and a rounding of its own."""
    B, Hq, D, page, lengths = 3, 4, 64, 16, [900, 64, 77]
    g = torch.Generator().manual_seed(2)
    width = 57
    cache, ((kc, kb), (vc, vb)) = make_cache(g, B * width, 1, page, D, list(range(B * width * page)))
    table = torch.randperm(B * width, generator=g).int().view(B, width)
    q = torch.randn(B, T, Hq, D, generator=g).half()
    k, v = ref.values(kc, kb, None), ref.values(vc, vb, None)
    tab = table.clone()
    for b, i, entry in [(0, 2, -1), (0, 5, 1 << 30), (1, 0, -5)] + [(2, i, -1) for i in range(5)]:
        tab[b, i] = entry
    o = gdn.gdn_kv_attention(q.to(dev), cache.to(dev), tab.to(dev), ints(lengths, dev), return_lse=True)
    for b, L in enumerate(lengths):
        j = torch.arange(L)
        at = table[b].long()[j // page] * page + j % page
        kk, vv = k[at, 0], v[at, 0]
        prod = torch.einsum("thd,ld->thl", q[b].double(), kk) / 8
        assert float(torch.einsum("thd,ld->thl", q[b].double().abs(), kk.abs()).max()) <= 256
        unseen = (tab[b][j // page] != table[b][j // page]) | (j > L - T + torch.arange(T)[:, None])
        w = prod.masked_fill(unseen[:, None], -math.inf).softmax(-1).nan_to_num(0.0)
        want, size = w @ vv, w @ vv.abs()
        got = o.y[b].cpu().double()
        assert bool(((got - want).abs() <= 2.0 ** -10 * size + 2.0 ** -11 * want.abs() + 2.0 ** -24).all())
        none = unseen.all(-1)
        assert bool((got[none] == 0).all()) and torch.equal((o.lse[b] == -math.inf).all(-1).cpu(), none)


@pytest.mark.parametrize("T", [20, 50])
@pytest.mark.parametrize("L", [150, 1100])
def test_nonfinite_rows_of_tiles(dev, T, L):  # noqa: F811
    """A query row with an infinity or a NaN is NaN, and no other row is."""
    g = torch.Generator().manual_seed(0)
    cache, _ = make_cache(g, 80, 2, 16, 64, list(range(80 * 16)))
    q = torch.randn(1, T, 8, 64, generator=g).bfloat16()
    q[0, 1, 2, 5], q[0, T - 1, 7, 0] = math.inf, math.nan
    o = gdn.gdn_kv_attention(q.to(dev), cache.to(dev), torch.arange(80, device=dev, dtype=torch.int32)[None],
                             ints([L], dev))
    bad = torch.zeros(1, T, 8, dtype=torch.bool)
    bad[0, 1, 2] = bad[0, T - 1, 7] = True
    assert torch.equal(o.y.isnan().all(-1).cpu(), bad) and torch.equal(o.y.isnan().any(-1).cpu(), bad)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D,T,Hq,window", [(64, 1, 32, 0), (128, 3, 64, 0), (256, 2, 32, 30)])
def test_many_units(dev, dtype, D, T, Hq, window):  # noqa: F811
    """Units that fill the GPU by themselves are not cut: of 8 rows and of 16, some of
    sequences without tokens."""
    B = 62
    attend_case(dev, dtype, B, T, Hq, 16, D, 16, [(53 * i) % 170 for i in range(B)], [(i + 1) % (T + 2) for i in range(B)],
                window, seed=D)


@pytest.mark.parametrize("tokens", [4864, 4865])
def test_rotary_of_many_tokens(dev, tokens):  # noqa: F811
    """One token per block and four: the same bits."""
    g = torch.Generator(device=dev).manual_seed(3)
    q = torch.randn(1, tokens, 2, 64, generator=g, device=dev).bfloat16()
    pos = torch.randint(-1, 1 << 20, (1, tokens), generator=g, device=dev, dtype=torch.int32)
    inv, scale = gdn.rotary_frequencies(32, device=dev)
    y = torch.full_like(q, 7.0)
    gdn.gdn_rotary(q, pos, inv, q_out=y, scale=scale)
    for at in range(0, tokens, 1000):
        piece = torch.full_like(q[:, at:at + 1000], 7.0)
        gdn.gdn_rotary(q[:, at:at + 1000].contiguous(), pos[:, at:at + 1000].contiguous(), inv, q_out=piece, scale=scale)
        assert torch.equal(piece, y[:, at:at + 1000])


@pytest.mark.parametrize("B,T", [(8, 256), (3, 682), (64, 30)])
def test_slots_by_one_kernel_and_two(dev, B, T):  # noqa: F811
    """Tokens of a call of few slots (one kernel) and of a call of many (two): the same."""
    g = torch.Generator().manual_seed(B)
    page, width = 16, T // 16 + 20
    lengths = torch.randint(0, 300, (B,), generator=g).int().to(dev)
    held = (lengths + page - 1) // page
    pages = B * width
    ring = torch.randperm(pages, generator=g).int().to(dev)
    used, outs = int(held.sum()), []
    table = torch.zeros(B, width, dtype=torch.int32, device=dev)
    at = 0
    for b in range(B):
        table[b, :int(held[b])] = ring[at:at + int(held[b])]
        at += int(held[b])
    add = torch.randint(0, 20, (B,), generator=g).int().to(dev)
    for wide in (T, 4 * T):
        tab, rg = table.clone(), ring.clone()
        s = gdn.gdn_page_slots(lengths, add, held, ints([used, pages - used], dev), tab, rg, T=wide, page=page)
        assert bool((s.slots[:, T:] == -1).all()) and torch.equal(s.granted, add)
        outs.append((s.slots[:, :20].clone(), s.positions[:, :20].clone(), tab, rg, s.lengths_out, s.held_out, s.ring_state_out))
    for a, b in zip(*outs):
        assert torch.equal(a, b)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rotary_into_slices(dev, layout):  # noqa: F811
    """Both outputs in one wider buffer, whose other channels stay."""
    g = torch.Generator(device=dev).manual_seed(4)
    q, k = (torch.randn(2, 9, h, 64, generator=g, device=dev).half() for h in (4, 2))
    pos = torch.randint(0, 9000, (2, 9), generator=g, device=dev, dtype=torch.int32)
    inv, scale = gdn.rotary_frequencies(64, device=dev)
    plain = gdn.gdn_rotary(q, pos, inv, k=k, layout=layout, scale=scale)
    wide = torch.full((2, 9, 7, 64), 7.0, device=dev).half()
    gdn.gdn_rotary(q, pos, inv, k=k, layout=layout, scale=scale, q_out=wide[:, :, :4], k_out=wide[:, :, 4:6])
    assert torch.equal(wide[:, :, :4], plain.q) and torch.equal(wide[:, :, 4:6], plain.k)
    assert bool((wide[:, :, 6] == 7.0).all())
