"""The operators of an attention layer against their formulas in float64."""
from __future__ import annotations

import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import attention_reference as ref  # noqa: E402
import linear_attention_recurrence_step_gb300 as gdn  # noqa: E402
from gdn_testutil import guarded_full, torch_dtype  # noqa: E402


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gdn.load()
    return torch.device("cuda:0")


def ints(v, dev):
    return torch.tensor(v, dtype=torch.int32, device=dev)


# -------------------------------------------------------------------- slots
def slots_case(B, T, page, longest, seed, tight=False, ends=0.1, rolled=True):
    g = torch.Generator().manual_seed(seed)
    width = -(-(longest + T) // page)
    lengths = torch.randint(0, longest + 1, (B,), generator=g)
    held = (lengths + page - 1) // page
    if rolled:
        held = (held + torch.randint(0, 3, (B,), generator=g)).clamp(max=width)
    add = torch.randint(0, T + 1, (B,), generator=g)
    add[torch.rand(B, generator=g) < ends] = -1
    pages = max(int(held.sum()) + B * (T // page + 1), 1)
    perm = torch.randperm(pages, generator=g).tolist()
    table = [[-1] * width for _ in range(B)]
    for b in range(B):
        for i in range(int(held[b])):
            table[b][i] = perm.pop()
    head = int(torch.randint(0, pages, (1,), generator=g))
    ring = [-7] * pages
    for i, p in enumerate(perm):
        ring[(head + i) % pages] = p
    count = len(perm) // 3 if tight else len(perm)
    return lengths.tolist(), add.tolist(), held.tolist(), [head, count], table, ring


@pytest.mark.parametrize("B,T,page,longest,tight", [
    (1, 1, 16, 40, False), (7, 1, 64, 1000, False), (300, 1, 16, 100, True), (33, 5, 32, 500, False),
    (1500, 3, 16, 64, True), (2500, 2, 128, 300, False), (20, 700, 16, 2000, True), (3, 4096, 128, 5000, False)])
@pytest.mark.parametrize("in_place", [False, True])
def test_page_slots(dev, B, T, page, longest, tight, in_place):
    lengths, add, held, state, table, ring = slots_case(B, T, page, longest, B + T, tight)
    d = {"lengths": ints(lengths, dev), "held": ints(held, dev), "ring_state": ints(state, dev)}
    dt, dr = guarded_full((B, len(table[0])), 0, torch.int32, dev), guarded_full((len(ring),), 0, torch.int32, dev)
    dt.copy_(ints(table, dev))
    dr.copy_(ints(ring, dev))
    out = {n: guarded_full(s, 99, torch.int32, dev) for n, s in
           {"slots": (B, T), "positions": (B, T), "granted": (B,)}.items()}
    out |= ({n + "_out": t for n, t in d.items()} if in_place else
            {n + "_out": guarded_full(t.shape, 99, torch.int32, dev) for n, t in d.items()})
    o = gdn.gdn_page_slots(d["lengths"], ints(add, dev), d["held"], d["ring_state"], dt, dr, T=T, page=page, **out)
    want = ref.page_slots(lengths, add, held, state, table, ring, T, page)
    for name, got, w in zip(o._fields, o, want):
        assert got.tolist() == w, name
    assert dt.tolist() == table and dr.tolist() == ring
    if not in_place:  # a repeated call gives the same
        o2 = gdn.gdn_page_slots(d["lengths"], ints(add, dev), d["held"], d["ring_state"], dt, dr, T=T, page=page)
        assert all(torch.equal(a, b) for a, b in zip(o, o2))
        assert dt.tolist() == table and dr.tolist() == ring


def test_page_slots_without_add_and_with_wrong_counts(dev):
    """add = None is T for each; counts out of range act as the nearest possible."""
    lengths, held, table, ring = [0, -5, 30, 1000], [0, -2, 99, 0], [[5, 6], [3, 3], [1, 2], [0, 0]], list(range(10, 17))
    dt, dr = ints(table, dev), ints(ring, dev)
    o = gdn.gdn_page_slots(ints(lengths, dev), None, ints(held, dev), ints([3, 1000], dev), dt, dr, T=2, page=16)
    want = ref.page_slots(lengths, None, held, [3, 7], table, ring, 2, 16)
    # (page 13 is past the pool of 7 pages: no slot)
    assert o.positions.tolist() == want[1] and o.granted.tolist() == want[2] == [2, 2, 2, 0]
    assert o.slots.tolist() == [[-1, -1], [-1, -1], [2 * 16 + 14, 2 * 16 + 15], [-1, -1]]
    assert dt.tolist() == table and o.ring_state_out.tolist() == want[5]


def test_page_slots_over_many_steps(dev):
    """Requests come, grow, are rolled back and end: no page is ever held twice or lost."""
    B, page, width, pages = 9, 16, 12, 60
    g = torch.Generator().manual_seed(3)
    lengths, held, state = (torch.zeros(n, dtype=torch.int32, device=dev) for n in (B, B, 2))
    state[1] = pages
    table, ring = torch.full((B, width), -1, dtype=torch.int32, device=dev), torch.arange(pages, dtype=torch.int32, device=dev)
    for step in range(60):
        add = torch.randint(-1, 25, (B,), generator=g).int().to(dev)
        o = gdn.gdn_page_slots(lengths, add, held, state, table, ring, T=24, page=page, lengths_out=lengths,
                               held_out=held, ring_state_out=state)
        used = o.slots[o.slots >= 0].tolist()
        assert len(set(used)) == len(used)
        owned = [int(p) for b in range(B) for p in table[b, :int(held[b])]]
        head, count = state.tolist()
        free = [int(ring[(head + i) % pages]) for i in range(count)]
        assert sorted(owned + free) == list(range(pages)), step
        # some drafts are rejected
        lengths -= (torch.rand(B, generator=g).to(dev) * o.granted).int()


# ------------------------------------------------------------------- rotary
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("B,T,Hq,Hk,D,R,pad", [
    (1, 1, 1, 0, 2, 2, 0), (3, 5, 4, 2, 64, 64, 0), (2, 3, 3, 1, 96, 24, 8), (2, 700, 8, 2, 128, 128, 33),
    (5, 1, 16, 2, 256, 64, 64), (1, 2, 2, 1, 30, 14, 1), (1, 1300, 1, 1, 64, 32, 0)])
def test_rotary(dev, dtype, layout, B, T, Hq, Hk, D, R, pad):
    dt, g = torch_dtype(dtype), torch.Generator().manual_seed(B * T + D)
    wide = torch.randn(B, T, (Hq + Hk) * D + pad, generator=g).to(dt)
    positions = torch.randint(-1, 2 ** 31 - 1, (B, T), generator=g, dtype=torch.int64)
    positions[torch.rand(B, T, generator=g) < 0.5] %= 5000
    positions[torch.rand(B, T, generator=g) < 0.1] = -1
    inv, scale = gdn.rotary_frequencies(R, scaling="parts_scaled", factor=16.0, trained=4096)
    wd = wide.to(dev)
    q, k = wd[..., :Hq * D].unflatten(-1, (Hq, D)), wd[..., Hq * D:(Hq + Hk) * D].unflatten(-1, (Hk, D)) if Hk else None
    qo = guarded_full((B, T, Hq, D), 7.0, dt, dev)
    ko = guarded_full((B, T, Hk, D), 7.0, dt, dev) if Hk else None
    pos = positions.int()
    for inverse in (False, True):
        o = gdn.gdn_rotary(q, pos.to(dev), inv.to(dev), k=k, layout=layout, scale=scale, inverse=inverse, q_out=qo, k_out=ko)
        off = (pos < 0)
        for x, y in ((q, o.q), (k, o.k)):
            if x is None:
                continue
            want, size = ref.rotary(x.cpu(), pos, inv, layout, scale, inverse)
            # sines within 4e-7 (the fraction's float, the function, the scale), two
            # products and a sum in float32, one rounding (half of the subnormals' step
            # below the smallest normal value); angles of float64 precision on either
            # side: the reference's product, the kernel's constant and product
            angle = pos.double().clamp(min=0)[..., None, None] * float(inv.max())
            tol = size * (6e-7 + angle * 2.0 ** -51) + want.abs() * torch.finfo(dt).eps / 2
            tol = tol + torch.finfo(dt).smallest_normal * torch.finfo(dt).eps / 2
            tol[..., R:] = 0
            err = (y.cpu().double() - want).abs()
            assert bool((err <= tol)[~off].all()), float((err - tol)[~off].max())
            assert bool((y.cpu()[off] == 7.0).all())
    # in place on the slices of the wider rows, whose other channels stay
    keep = wd.clone()
    o2 = gdn.gdn_rotary(q, pos.to(dev), inv.to(dev), k=k, layout=layout, scale=scale, inverse=True, q_out=q, k_out=k)
    on = (pos >= 0).to(dev)
    assert torch.equal(o2.q[on], o.q[on]) and (k is None or torch.equal(o2.k[on], o.k[on]))
    assert torch.equal(wd[~on], keep[~on]) and torch.equal(wd[..., (Hq + Hk) * D:], keep[..., (Hq + Hk) * D:])


def test_rotary_gradient(dev):
    """`inverse` is the transposed map: <turn(x), w> = <x, turn back(w)>, and the
    gradient that float64 autograd finds."""
    g = torch.Generator().manual_seed(1)
    x, w = (torch.randn(2, 3, 4, 64, generator=g) for _ in range(2))
    pos = torch.randint(0, 100000, (2, 3), generator=g).int()
    inv, _ = gdn.rotary_frequencies(32)
    xd = x.double().requires_grad_()
    a = pos.double()[..., None, None] * inv.double()
    u, v = xd[..., :16], xd[..., 16:32]
    y = torch.cat([u * a.cos() - v * a.sin(), u * a.sin() + v * a.cos(), xd[..., 32:]], -1) * 1.0
    (y * w.double()).sum().backward()
    got = gdn.gdn_rotary(w.to(dev), pos.to(dev), inv.to(dev), inverse=True).q.cpu().double()
    assert float((got - xd.grad).abs().max()) < 6e-7 * 2 * float(w.abs().max()) + 2.0 ** -24 * float(w.abs().max())


# ------------------------------------------------------------ write and read
def head_scales(H, g, exact=True):
    return torch.exp2(torch.randint(-6, 7, (H,), generator=g).float()) if exact else torch.rand(H, generator=g) + 0.01


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("B,T,H,D,page,pad,scales", [
    (1, 1, 1, 64, 16, 0, None), (3, 5, 2, 128, 32, 0, "exact"), (2, 70, 3, 64, 128, 3, "any"),
    (4, 33, 1, 256, 64, 8, "exact"), (1, 300, 4, 128, 16, 0, None)])
def test_append_and_read(dev, dtype, B, T, H, D, page, pad, scales):
    dt, g = torch_dtype(dtype), torch.Generator().manual_seed(B + T + D)
    wide = torch.randn(B, T, 2 * H * D + pad, generator=g) * torch.exp(2 * torch.randn(B, T, 1, generator=g))
    wide[torch.rand(wide.shape, generator=g) < 0.02] = 0.0
    # values on the borders between codes and between scales
    tie = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, -0.25, -5.0, 12 * 17 / 16 * 6 / 12, 1e-6, 3e-3, 0, 448, 3000])
    wide[0, 0, :16] = tie
    wide[-1, -1, -pad - 16:wide.shape[-1] - pad] = tie[torch.randperm(16, generator=g)] * 2.0 ** -7
    special = wide.clone()
    special[0, -1, 16:20] = torch.tensor([math.nan, math.inf, -math.inf, 1.0])
    special = special.to(dt)
    wd = special.to(dev)
    k, v = wd[..., :H * D].unflatten(-1, (H, D)), wd[..., H * D:2 * H * D].unflatten(-1, (H, D))
    ks = vs = None
    if scales:
        ks, vs = head_scales(H, g, scales == "exact"), head_scales(H, g, scales == "exact")
    pages = -(-B * T // page) + 2
    slots = torch.randperm(pages * page, generator=g)[:B * T].int().view(B, T)
    slots[torch.rand(B, T, generator=g) < 0.2] = -1
    slots[0, 0] = pages * page - 1 if not (slots == pages * page - 1).any() else slots[0, 0]
    if T > 2:
        slots[0, 1] = pages * page + 3  # past the last page
    cache = guarded_full((pages, H, page, 9 * D // 8), 0x5A, torch.uint8, dev)
    want = cache.cpu()
    on = (slots >= 0) & (slots < pages * page)
    for i, (x, s) in enumerate(((k, ks), (v, vs))):
        codes, byte = ref.quantise(x.cpu(), s)
        ref.put(want, slots[on].tolist(), codes[on], byte[on], i)
    to = lambda t: None if t is None else t.to(dev)  # noqa: E731
    gdn.gdn_kv_append(k, v, slots.to(dev), cache, k_scale=to(ks), v_scale=to(vs))
    # codes of zero may carry either sign
    got = cache.cpu()
    same = got == want
    D2, per = D // 2, page * (D // 2 + D // 16)
    flat = (torch.arange(2 * per) % per < page * D2).view(page, -1).expand(pages, H, page, -1)
    zero_sign = ((got ^ want) & 0x77) == 0
    lo_ok = ((got ^ want) & 0x0F == 0) | (got & 0x07 == 0)
    hi_ok = ((got ^ want) & 0xF0 == 0) | (got & 0x70 == 0)
    assert bool((same | (flat & zero_sign & lo_ok & hi_ok)).all())
    ko, vo = guarded_full(k.shape, 7.0, dt, dev), guarded_full(k.shape, 7.0, dt, dev)
    o = gdn.gdn_kv_read(cache, slots.to(dev), dtype=dt, k_scale=to(ks), v_scale=to(vs), k=ko, v=vo)
    for x, y, s in ((k, o.k, ks), (v, o.v, vs)):
        codes, byte = ref.quantise(x.cpu(), s)
        w = ref.values(codes, byte, s)
        y = y.cpu()
        # a float32 product, then the rounding to the type (2688 head scales may pass f16's range)
        lim = torch.finfo(dt).max
        tol = w.abs() * (torch.finfo(dt).eps / 2 + 2.0 ** -24) + (torch.finfo(dt).smallest_normal * torch.finfo(dt).eps)
        ok = ((y.double() - w).abs() <= tol) | ((w.abs() > lim) & (y.double().abs() >= lim))
        assert bool(ok[on].all())
        assert bool((y[~on] == 7.0).all())


# ---------------------------------------------------------------- attention
def make_cache(g, pages, H, page, D, used):
    """A cache whose `used` slots hold normal values and every other byte 0xff (NaN
    scales), on the CPU, and the values."""
    cache = torch.full((pages, H, page, 9 * D // 8), 0xFF, dtype=torch.uint8)
    out = []
    for kv in range(2):
        x = torch.randn(len(used), H, D, generator=g) * 2
        codes, byte = ref.quantise(x, None)
        ref.put(cache, used, codes, byte, kv)
        out.append((codes, byte))
    return cache, out


def attend_case(dev, dtype, B, T, Hq, H, D, page, lengths, fresh=None, window=0, pad=0, seed=0, scale=None, sharp=1.0,
                bad=None, **kw):
    dt, g = torch_dtype(dtype), torch.Generator().manual_seed(seed)
    width = max(1, -(-max(lengths) // page))
    pages = B * width + 2
    table = torch.randperm(pages, generator=g)[:B * width].view(B, width)
    used, at = [], []
    for b in range(B):
        at.append(len(used))
        used += [int(table[b, j // page]) * page + j % page for j in range(lengths[b])]
    cache, (kq, vq) = make_cache(g, pages, H, page, D, used)
    ks, vs = head_scales(H, g), head_scales(H, g)
    ks = ks / ks.max()
    wide = (torch.randn(B, T, Hq * D + pad, generator=g) * sharp).to(dt)
    n = [T] * B if fresh is None else [min(max(f, 0), T) for f in fresh]
    for b in range(B):  # rows that are not there may hold anything
        wide[b, n[b]:] = math.nan
    q = wide.to(dev)[..., :Hq * D].unflatten(-1, (Hq, D))
    y, lse = guarded_full((B, T, Hq, D), 7.0, dt, dev), guarded_full((B, T, Hq), 7.0, torch.float32, dev)
    gone = torch.zeros(B, width, dtype=torch.bool)
    tab = table.int()
    for b, i, entry in bad or ():
        tab[b, i], gone[b, i] = entry, True
    args = dict(new=None if fresh is None else ints(fresh, dev), scale=scale, window=window, k_scale=ks.to(dev),
                v_scale=vs.to(dev))
    call = lambda: gdn.gdn_kv_attention(q, cache.to(dev), tab.to(dev), ints(lengths, dev), y=y, lse=lse, **args, **kw)  # noqa: E731
    call()
    torch.cuda.synchronize()
    sc = 1 / math.sqrt(D) if scale is None else scale
    for b in range(B):
        L, nb = lengths[b], n[b]
        sel = slice(at[b], at[b] + L)
        k = ref.values(kq[0][sel], kq[1][sel], ks)
        v = ref.values(vq[0][sel], vq[1][sel], vs)
        qb = q[b].cpu()
        if gone[b].any():  # tokens out of sight: as if their scores were -inf
            keep = ~gone[b].repeat_interleave(page)[:L]
            assert nb == 1 and not window
            k, v = k[keep], v[keep]
        wy, wl, pv, size, all_v = (r[max(0, nb - len(k)):] for r in ref.attention(qb, k, v, min(nb, max(len(k), nb)), sc, window))
        skip = nb - len(wy)
        by, bl = ref.attention_bounds(wy, wl, pv, size, all_v, dt, L)
        gy, gl = y[b, skip:nb].cpu().double(), lse[b, skip:nb].cpu().double()
        assert bool(((gy - wy).abs() <= by).all()), (b, float(((gy - wy).abs() - by).max()))
        assert bool((((gl - wl).abs() <= bl) | (gl == wl)).all()), (b, float((gl - wl).abs().max()))
        assert bool((y[b, :skip] == 0).all()) and bool((lse[b, :skip] == -math.inf).all())
        assert bool((y[b, nb:] == 7.0).all()) and bool((lse[b, nb:] == 7.0).all())
    first = y.clone(), lse.clone()
    call()
    assert torch.equal(y, first[0]) and torch.equal(lse, first[1])  # run to run
    return y


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("B,T,Hq,H,page,lengths", [
    (1, 1, 1, 1, 16, [1]), (3, 1, 8, 2, 16, [1, 17, 700]), (2, 1, 12, 4, 128, [129, 1000]), (4, 1, 16, 1, 32, [5, 64, 65, 2049]),
    (2, 3, 10, 2, 64, [3, 400])])
def test_attention_tokens(dev, dtype, D, B, T, Hq, H, page, lengths):
    attend_case(dev, dtype, B, T, Hq, H, D, page, lengths, seed=D + B)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("D,page", [(64, 64), (128, 16), (256, 32)])
@pytest.mark.parametrize("window", [0, 1, 37])
def test_attention_drafts(dev, dtype, D, page, window):
    """Ragged drafts of several rows per key head, empty sequences, rows before
    the first token, windows, slices of a wider projection."""
    attend_case(dev, dtype, 6, 9, 6, 2, D, page, [0, 4, 9, 100, 333, 64], [0, 9, 9, 5, -3, 12], window, pad=24, seed=page)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("D,T,Hq,H,lengths,window", [
    (128, 200, 4, 1, [200, 500], 0), (64, 150, 2, 2, [700, 150], 100), (256, 67, 8, 2, [67, 300], 0), (128, 130, 5, 1, [131, 600], 0)])
def test_attention_prompts(dev, dtype, D, T, Hq, H, lengths, window):
    attend_case(dev, dtype, 2, T, Hq, H, D, 32, lengths, [T, T - 3], window, seed=T)


@pytest.mark.parametrize("D,T,Hq,H,lengths", [(128, 200, 4, 1, [200]), (128, 300, 1, 1, [900]), (64, 90, 1, 1, [1100]), (256, 140, 2, 1, [1200])])
def test_attention_prompts_again(dev, D, T, Hq, H, lengths):
    """Row blocks of one tile over several steps, whole and in parts, many times: the
    same results each time."""
    y = attend_case(dev, "f16", 1, T, Hq, H, D, 16, lengths, seed=T).clone()
    for _ in range(15):
        assert torch.equal(attend_case(dev, "f16", 1, T, Hq, H, D, 16, lengths, seed=T), y)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_attention_sharp_scores(dev, dtype):
    """Scores of hundreds (one token takes all), tiny ones, scales of zero and below."""
    for sharp, scale in ((40.0, 0.5), (1e-6, 1.0), (1.0, 0.0), (3.0, -0.3)):
        attend_case(dev, dtype, 2, 2, 4, 2, 128, 16, [900, 77], seed=5, sharp=sharp, scale=scale)


@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_attention_bad_pages(dev, dtype):
    """Entries that name no page take their tokens out of sight, all of them too."""
    attend_case(dev, dtype, 3, 1, 4, 2, 64, 16, [100, 64, 16], seed=2, bad=[(0, 2, -1), (0, 5, 1 << 30), (2, 0, -5)])


def test_attention_nonfinite_rows(dev):
    """A query row with an infinity or a NaN is NaN, and no other row is."""
    g = torch.Generator().manual_seed(0)
    cache, _ = make_cache(g, 10, 2, 16, 64, list(range(160)))
    q = torch.randn(1, 3, 8, 64, generator=g)
    q[0, 1, 2, 5], q[0, 2, 7, 0] = math.inf, math.nan
    o = gdn.gdn_kv_attention(q.to(dev), cache.to(dev), torch.arange(10, device=dev, dtype=torch.int32)[None],
                             ints([150], dev))
    bad = torch.zeros(1, 3, 8, dtype=torch.bool)
    bad[0, 1, 2] = bad[0, 2, 7] = True
    assert torch.equal(o.y.isnan().all(-1).cpu(), bad) and torch.equal(o.y.isnan().any(-1).cpu(), bad)


def test_attention_far_pages(dev):
    """Blocks that start past 2^32 bytes."""
    H, page, D = 4, 128, 256
    pages = 2 ** 32 // (H * page * 9 * D // 8) + 40
    cache = torch.zeros(pages, H, page, 9 * D // 8, dtype=torch.uint8, device=dev)
    g = torch.Generator(device=dev).manual_seed(0)
    kv = torch.randn(1, 300, 2, H, D, generator=g, device=dev, dtype=torch.bfloat16)
    q = torch.randn(1, 1, 8, D, generator=g, device=dev, dtype=torch.bfloat16)
    outs = []
    for first in (0, pages - 3):
        table = torch.arange(first, first + 3, device=dev, dtype=torch.int32)[None]
        slots = (first * page + torch.arange(300, device=dev, dtype=torch.int64)).int()[None]
        gdn.gdn_kv_append(kv[:, :, 0], kv[:, :, 1], slots, cache)
        outs.append((gdn.gdn_kv_attention(q, cache, table, ints([300], dev)).y, gdn.gdn_kv_read(cache, slots).k))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
    assert float(outs[0][0].float().abs().max()) > 0


# ---------------------------------------------------------------- together
def test_layer_with_rollback(dev):
    """A prompt, drafts that are partly rejected, a request that ends and one that
    takes its pages, against the same operators over a dense cache in float64."""
    B, H, G, D, page, width, R = 4, 2, 3, 64, 16, 20, 32
    pages = 50
    g = torch.Generator(device=dev).manual_seed(11)
    cache = gdn.gdn_kv_cache(pages, H, page, D, device=dev)
    cache.fill_(0xFF)
    lengths, held, state = (torch.zeros(n, dtype=torch.int32, device=dev) for n in (B, B, 2))
    state[1] = pages
    table, ring = torch.zeros(B, width, dtype=torch.int32, device=dev), torch.randperm(pages, generator=g, device=dev).int()
    inv, scale = gdn.rotary_frequencies(R, device=dev)
    past = [[] for _ in range(B)]
    # (tokens per sequence, accepted of them)
    steps = [([100, 37, 0, 16], None), ([5, 5, 5, 0], [2, 5, 1, 0]), ([5, 5, 5, 5], [5, 1, 1, 3]), ([-1, 1, 1, 1], None),
             ([90, 1, 1, 1], None), ([1, 1, 1, 1], None)]
    for add, accepted in steps:
        T = max(add)
        q = torch.randn(B, T, H * G, D, generator=g, device=dev).bfloat16()
        kv = torch.randn(B, T, 2, H, D, generator=g, device=dev).bfloat16()
        s = gdn.gdn_page_slots(lengths, ints(add, dev), held, state, table, ring, T=T, page=page, lengths_out=lengths,
                               held_out=held, ring_state_out=state)
        assert s.granted.tolist() == [max(a, 0) for a in add]
        r = gdn.gdn_rotary(q, s.positions, inv, k=kv[:, :, 0], scale=scale)
        gdn.gdn_kv_append(r.k, kv[:, :, 1], s.slots, cache)
        o = gdn.gdn_kv_attention(r.q, cache, table, lengths, new=s.granted, return_lse=True)
        kr, vr = gdn.gdn_kv_read(cache, s.slots, dtype=torch.float32)
        for b in range(B):
            n = max(add[b], 0)
            if add[b] < 0:
                past[b] = []
                continue
            for t in range(n):
                want, size = ref.rotary(kv[b, t, 0].cpu(), s.positions[b, t].cpu(), inv.cpu())
                assert float((r.k[b, t].cpu().double() - want).abs().max()) <= float(want.abs().max()) * 2.0 ** -8 + 1e-5
                codes, byte = ref.quantise(r.k[b, t].cpu(), None)
                assert torch.equal(kr[b, t].cpu().double(), ref.values(codes, byte, None))
                past[b].append((kr[b, t].cpu().double(), vr[b, t].cpu().double()))
            if n == 0:
                continue
            k, v = (torch.stack([p[i] for p in past[b]]) for i in range(2))
            wy, wl, pv, size, all_v = ref.attention(r.q[b].cpu(), k, v, n, 1 / math.sqrt(D))
            by, bl = ref.attention_bounds(wy, wl, pv, size, all_v, torch.bfloat16, len(k))
            assert bool(((o.y[b, :n].cpu().double() - wy).abs() <= by).all())
            assert bool(((o.lse[b, :n].cpu().double() - wl).abs() <= bl).all())
            if accepted is not None:
                del past[b][len(past[b]) - (n - accepted[b]):]
        if accepted is not None:  # the rejected tokens go; their pages stay held
            lengths -= s.granted - ints(accepted, dev)
    assert lengths.tolist() == [len(p) for p in past]


def test_captured_and_on_another_stream(dev):
    """A step captured in a graph and replayed over changed inputs, and calls on a
    stream of their own, give what plain calls give."""
    B, H, G, D, page, pages = 3, 2, 4, 128, 32, 30
    g = torch.Generator(device=dev).manual_seed(4)
    inv, _ = gdn.rotary_frequencies(D, device=dev)
    q = torch.randn(B, 2, H * G, D, generator=g, device=dev).half()
    kv = torch.randn(B, 2, 2, H, D, generator=g, device=dev).half()

    def fresh_state():
        return dict(lengths=ints([40, 70, 0], dev), held=ints([2, 3, 0], dev), ring_state=ints([0, 20], dev),
                    block_table=torch.arange(30, 60, dtype=torch.int32, device=dev).view(3, 10) % 30,
                    ring=torch.arange(30, dtype=torch.int32, device=dev) % 20, cache=gdn.gdn_kv_cache(pages, H, page, D, device=dev))

    def step(st, stream=None):
        s = gdn.gdn_page_slots(st["lengths"], None, st["held"], st["ring_state"], st["block_table"], st["ring"], T=2,
                               page=page, lengths_out=st["lengths"], held_out=st["held"],
                               ring_state_out=st["ring_state"], stream=stream)
        r = gdn.gdn_rotary(q, s.positions, inv, k=kv[:, :, 0], stream=stream)
        gdn.gdn_kv_append(r.k, kv[:, :, 1], s.slots, st["cache"], stream=stream)
        return gdn.gdn_kv_attention(r.q, st["cache"], st["block_table"], st["lengths"], new=s.granted, stream=stream).y

    plain = fresh_state()
    want = [step(plain).clone() for _ in range(3)]
    other = fresh_state()
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    got = [step(other, stream=st) for _ in range(3)]
    st.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    captured = fresh_state()
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step({n: t.clone() for n, t in captured.items()})
    torch.cuda.current_stream().wait_stream(side)
    with torch.cuda.graph(graph):
        y = step(captured)
    start = fresh_state()
    for n, t in captured.items():
        t.copy_(start[n])
    for w in want:
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, w)
