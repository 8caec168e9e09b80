"""The attention layer's operators step by step in float64 (torch, CPU), and the
bounds that their kernels are held to."""
from __future__ import annotations

import math

import torch

E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
E4M3 = [(b & 7) * 2.0 ** -9 if b < 8 else (8 + (b & 7)) * 2.0 ** ((b >> 3) - 10) for b in range(127)]


def page_slots(lengths, add, held, ring_state, table, ring, T, page):
    """Plain integers; table (list of rows) and ring (list) are changed in place."""
    width, pages = len(table[0]), len(ring)
    head, count = ring_state
    slots, positions, granted, lengths_out, held_out, upto, back, taken = [], [], [], [], [], 0, [], 0
    for b in range(len(lengths)):
        n, h = max(lengths[b], 0), min(max(held[b], 0), width)
        want = T if add is None else min(add[b], T)
        got, pos = 0, []
        if want < 0:
            back += table[b][:h]
            n = h = 0
        elif n + want <= width * page:
            need = max(0, -(-(n + want) // page) - h)
            upto += need
            if need == 0 or upto <= count:
                for i in range(need):
                    table[b][h + i] = ring[(head + upto - need + i) % pages]
                taken += need
                h, got = h + need, want
                pos = list(range(n, n + want))
        slots.append([table[b][p // page] * page + p % page for p in pos] + [-1] * (T - got))
        positions.append(pos + [-1] * (T - got))
        granted.append(got)
        lengths_out.append(n + got)
        held_out.append(h)
    for i, p in enumerate(back):
        ring[(head + count + i) % pages] = p
    return slots, positions, granted, lengths_out, held_out, [(head + taken) % pages, count - taken + len(back)]


def rotary(x, positions, inv_freq, layout="half", scale=1.0, inverse=False):
    """float64 result, and what an error of one in the sines would make of it."""
    x = x.double()
    R = 2 * inv_freq.shape[0]
    angle = positions.double()[..., None, None] * inv_freq.double()
    c, s = torch.cos(angle), torch.sin(angle) * (-1 if inverse else 1)
    a, b = (x[..., :R // 2], x[..., R // 2:R]) if layout == "half" else (x[..., 0:R:2], x[..., 1:R:2])
    y, size = x.clone(), torch.zeros_like(x)
    first, second = ((slice(0, R // 2), slice(R // 2, R)) if layout == "half" else (slice(0, R, 2), slice(1, R, 2)))
    y[..., first], y[..., second] = scale * (a * c - b * s), scale * (a * s + b * c)
    size[..., first] = size[..., second] = abs(scale) * (a.abs() + b.abs())
    return y, size


def _nearest(x, values):
    """Index of the nearest of the sorted values, between two the even one."""
    hi = torch.searchsorted(values, x.contiguous()).clamp(1, len(values) - 1)
    up, down = values[hi] - x, x - values[hi - 1]
    return torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, hi - 1)


def quantise(x, head_scale):
    """Codes [..., D] and scale bytes [..., D/16] of x [..., H, D] (head_scale [H] float32 or None)."""
    u = (x.float() if head_scale is None else x.float() / head_scale[:, None]).double()
    u = torch.nan_to_num(u, nan=0.0, posinf=3e38, neginf=-3e38).unflatten(-1, (-1, 16))
    grid = torch.tensor(E4M3, dtype=torch.float64)
    byte = _nearest((u.abs().amax(-1, keepdim=True) / 6).clamp(max=448), grid)
    s = grid[byte]
    q = torch.where(s > 0, u.abs() / s.clamp(min=1e-300), torch.zeros_like(u)).clamp(max=6)
    code = _nearest(q, torch.tensor(E2M1, dtype=torch.float64))
    return (code + 8 * (u < 0)).flatten(-2), byte[..., 0]


def values(code, byte, head_scale):
    """float64 elements of codes [..., H, D] and scale bytes [..., H, D/16]."""
    v = torch.tensor(E2M1 + [-e for e in E2M1], dtype=torch.float64)[code]
    v = v * torch.tensor(E4M3, dtype=torch.float64)[byte].repeat_interleave(16, -1)
    return v if head_scale is None else v * head_scale.double()[:, None]


def put(cache, slots, codes, bytes_, kv):
    """Codes and scale bytes [N,H,...] into the cache (CPU, uint8) at N slots, keys (0) or values (1)."""
    pages, H, page, row = cache.shape
    D = row // 9 * 8
    flat = cache.view(pages, H, -1)
    base = kv * page * (D // 2 + D // 16)
    packed = (codes[..., 0::2] | (codes[..., 1::2] << 4)).to(torch.uint8)
    for i, s in enumerate(slots):
        p, r = s // page, s % page
        flat[p, :, base + r * D // 2:base + (r + 1) * D // 2] = packed[i]
        at = base + page * D // 2 + r * D // 16
        flat[p, :, at:at + D // 16] = bytes_[i].to(torch.uint8)


def attention(q, k, v, n, scale, window=0):
    """One sequence: q [T,Hq,D], k and v [L,H,D] float64, its n last tokens the queries q[:n].

    Returns y, lse, and the sizes that the bounds go by: sum_j p_j |v_j|, the
    largest scale sum_i |q_i k_ji| over the tokens that a query sees, and their
    sum_j |v_j|."""
    L, H, D = k.shape
    Hq = q.shape[1]
    G = Hq // H
    y, lse = torch.zeros(n, Hq, D, dtype=torch.float64), torch.full((n, Hq), -math.inf, dtype=torch.float64)
    pv, size = torch.zeros_like(y), torch.zeros(n, Hq, dtype=torch.float64)
    all_v = torch.zeros_like(y)
    j = torch.arange(L)
    for t in range(n):
        pos = L - n + t
        seen = (j <= pos) & ((j > pos - window) if window else True)
        if not seen.any():
            continue
        ks, vs = k[seen].repeat_interleave(G, 1), v[seen].repeat_interleave(G, 1)
        x = torch.einsum("hd,lhd->hl", q[t].double(), ks) * scale
        p = torch.softmax(x, -1)
        y[t], lse[t] = torch.einsum("hl,lhd->hd", p, vs), torch.logsumexp(x, -1)
        pv[t] = torch.einsum("hl,lhd->hd", p, vs.abs())
        all_v[t] = vs.abs().sum(0)
        size[t] = torch.einsum("hd,lhd->hl", q[t].double().abs(), ks.abs()).amax(-1) * abs(scale)
    return y, lse, pv, size, all_v


def attention_bounds(y, lse, pv, size, all_v, dtype, L):
    """What y and lse may be off by.

    A score takes D/16 <= 16 accumulations of a unit 2^-23 of at most `size`
    each (twice as many by two terms), the queries' 2^-23 and the softmax's own
    roundings 2^-20; twice that moves y's weights.  A weight is rounded to f16
    (2^-12; two terms: 2^-23) and by 2^-25 where that is more, beside a sum of the
    weights that is 2^6 at least (float32: 2^14); a sum over L tokens in steps of 16 adds L/16
    units, and y is rounded once (by half of the subnormals' step below the
    smallest normal value)."""
    ds = size * 40 * 2.0 ** -23 + 2.0 ** -20
    weight = 2.0 ** -23 if dtype == torch.float32 else 2.0 ** -12
    least = 2.0 ** -39 if dtype == torch.float32 else 2.0 ** -31
    by = pv * (2 * ds[..., None] + 2 * weight + (L / 16 + 16) * 2.0 ** -23) + all_v * least + torch.finfo(dtype).eps / 2 * (y.abs() + torch.finfo(dtype).smallest_normal)
    return by, ds + lse.abs() * 2.0 ** -22
