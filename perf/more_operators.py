"""Cases for the operators of an attention layer between recurrent ones.

A hybrid model's attention layer keeps its keys and values in pages of 4-bit
values.  In a serving step the pages and places of the new tokens are found
from the requests' lengths, queries and keys are rotated, keys and values are
written to their places, and the queries attend over the cache.  Each case is
one call (``store``: a write and the read of what it wrote):

  slots   need = ceil((len + add) / page) - held pages for every sequence, taken
          from the ring of free pages; slot and position of every new token
  rotary  (a, b) -> (a cos - b sin, a sin + b cos) * scale, angle = position * inv_freq
  store   per 16 elements a scale s = e4m3(max|u| / 6) and codes e2m1(u / s),
          u = x / head scale; read back: head scale * s * code
  attend  y = softmax(scale q k^T) v over the visible tokens, and its log-sum-exp

``own`` picks the side that ``run`` takes: elementary torch operations in 32
bits (False; angles and values next to a rounding border in 64) or the
library's kernels (True).
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
ESIZE = {"f32": 4, "bf16": 2, "f16": 2}
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # one new token for each of 64 requests: latency counts
        {"name": "slots_decode_b64", "op": "slots", "B": 64, "T": 1, "page": 16, "longest": 8192, "tight": False},
        # 64 prompts of ragged lengths arrive at once, some requests end, and the pool is short of pages
        {"name": "slots_prompts_b64", "op": "slots", "B": 64, "T": 4096, "page": 64, "longest": 2000, "tight": True},
        # one token of 32 sequences, a quarter of wide heads is rotated
        {"name": "rotary_decode_b32", "op": "rotary", "B": 32, "T": 1, "Hq": 16, "Hk": 2, "D": 256, "R": 64,
         "layout": "half", "scaled": False, "dtype": "bf16", "ragged": False, "far": 8192, "pad": 0},
        # a piece of a long document, frequencies scaled for it, slices of one projection, whole heads
        {"name": "rotary_prompt_t4096", "op": "rotary", "B": 1, "T": 4096, "Hq": 32, "Hk": 8, "D": 128, "R": 128,
         "layout": "interleaved", "scaled": True, "dtype": "f16", "ragged": False, "far": 1000000, "pad": 1024},
        # keys and values of one token of 32 sequences
        {"name": "store_decode_b32", "op": "store", "B": 32, "T": 1, "H": 8, "D": 128, "page": 16, "dtype": "f32",
         "ragged": False},
        # keys and values of 4 prompts of ragged lengths
        {"name": "store_prompt_t4096", "op": "store", "B": 4, "T": 4096, "H": 8, "D": 128, "page": 64,
         "dtype": "bf16", "ragged": True},
        # one token of one sequence with a short context: latency counts
        {"name": "attend_decode_b1", "op": "attend", "B": 1, "T": 1, "Hq": 16, "H": 2, "D": 256, "L": 1000,
         "page": 16, "window": 0, "dtype": "bf16", "ragged": False},
        # one token of 32 sequences of ragged lengths
        {"name": "attend_decode_b32", "op": "attend", "B": 32, "T": 1, "Hq": 32, "H": 8, "D": 128, "L": 8192,
         "page": 16, "window": 0, "dtype": "bf16", "ragged": True},
        # one token of 8 sequences with long documents
        {"name": "attend_decode_l131072", "op": "attend", "B": 8, "T": 1, "Hq": 32, "H": 8, "D": 128, "L": 131072,
         "page": 64, "window": 0, "dtype": "bf16", "ragged": False},
        # five draft tokens, a sliding window, heads of 64 in threes, float32
        {"name": "attend_window_f32", "op": "attend", "B": 7, "T": 5, "Hq": 9, "H": 3, "D": 64, "L": 5001,
         "page": 32, "window": 1000, "dtype": "f32", "ragged": True},
        # verification of eight draft tokens of 16 sequences
        {"name": "attend_verify_b16_t8", "op": "attend", "B": 16, "T": 8, "Hq": 32, "H": 8, "D": 128, "L": 8192,
         "page": 32, "window": 0, "dtype": "f16", "ragged": True},
        # a piece of a long prompt behind what is cached already
        {"name": "attend_prompt_t2048", "op": "attend", "B": 1, "T": 2048, "Hq": 32, "H": 8, "D": 128, "L": 8192,
         "page": 64, "window": 0, "dtype": "bf16", "ragged": False},
    ]


def _log_int(rng, lo, hi):
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return min(max(n, lo), hi)


def draw(rng):
    op = rng.choice(["slots", "rotary", "store", "attend", "attend", "attend"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    page = rng.choice([16, 32, 64, 128])
    if op == "slots":
        T = rng.choice([1, rng.randint(2, 16), _log_int(rng, 17, 4096)])
        return {"op": op, "B": _log_int(rng, 1, min(512, 64 * 4096 // T)), "T": T, "page": page,
                "longest": _log_int(rng, 100, 8192), "tight": rng.random() < 0.4}
    T = rng.choice([1, 1, rng.randint(2, 12), _log_int(rng, 13, 2048)])
    if op == "rotary":
        D = rng.choice([64, 96, 128, 256])
        Hk = rng.choice([1, 2, 4, 8])
        Hq = Hk * rng.randint(1, 8)
        most = 4096 * 40 * 128 * 2 // ((Hq + Hk) * D * ESIZE[dtype])
        T = min(T, most)
        return {"op": op, "B": _log_int(rng, 1, max(1, min(64, most // T))), "T": T, "Hq": Hq, "Hk": Hk, "D": D,
                "R": rng.choice([D, D, D // 2, D // 4]), "layout": rng.choice(["half", "interleaved"]),
                "scaled": rng.random() < 0.5, "dtype": dtype, "ragged": rng.random() < 0.5,
                "far": _log_int(rng, 5000, 1000000), "pad": rng.choice([0, 0, 64, 33])}
    D, H = rng.choice([64, 128, 128, 256]), rng.choice([1, 2, 3, 4, 8])
    if op == "store":
        most = 4 * 4096 * 8 * 128 * 2 // (H * D * ESIZE[dtype])
        T = min(T, most)
        return {"op": op, "B": _log_int(rng, 1, max(1, min(64, most // T))), "T": T, "H": H, "D": D, "page": page,
                "dtype": dtype, "ragged": rng.random() < 0.5}
    G = rng.choice([1, 2, 3, 4, 5, 8])
    L = _log_int(rng, max(T, 20), 131072)
    pairs = 2048 * 7168 * 32 * 128 // (T * L * H * G * D * (4 if dtype == "f32" else 1))
    B = min(8 * 131072 * 8 * 128 // (L * H * D), pairs)
    if B < 1:
        L = max(T, 20, min(L, 8192 // (4 if dtype == "f32" else 1)))
    return {"op": op, "B": _log_int(rng, 1, max(1, min(64, B))), "T": T, "Hq": H * G, "H": H, "D": D, "L": L,
            "page": page, "window": rng.choice([0, 0, 0, _log_int(rng, 16, 4096)]), "dtype": dtype,
            "ragged": rng.random() < 0.5}


# --------------------------------------------------------------- the inputs
def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return {"slots": _prepare_slots, "rotary": _prepare_rotary, "store": _prepare_store,
            "attend": _prepare_attend}[case["op"]](case, gen)


def _randn(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda")


def _randint(gen, lo, hi, *shape):
    return torch.randint(lo, hi + 1, shape, generator=gen, device="cuda", dtype=torch.int32)


def _prepare_slots(c, gen):
    B, T, page = c["B"], c["T"], c["page"]
    width = -(-(c["longest"] + T) // page)
    pool = B * width
    lengths = _randint(gen, 0, c["longest"], B)
    add = torch.full((B,), T, device="cuda", dtype=torch.int32) if T == 1 else _randint(gen, 0, T, B)
    add[torch.rand(B, generator=gen, device="cuda") < 0.06] = -1          # requests that end
    # up to two pages more are held than the length needs: drafts that were rolled back
    held = ((lengths + page - 1) // page + _randint(gen, 0, 2, B) * (lengths > 0)).clamp(max=width).int()
    perm = torch.randperm(pool, generator=gen, device="cuda").int()
    first = held.cumsum(0) - held
    col = torch.arange(width, device="cuda")
    at = (first[:, None] + col).clamp(max=pool - 1)
    table = torch.where(col < held[:, None], perm[at], -1).int()
    # the pages that nobody holds stand in the ring from a place in its middle on, in a shuffled order
    used = held.sum()
    free = pool - used
    head = pool // 3
    ring = perm[(used + (torch.arange(pool, device="cuda") - head) % pool).clamp(max=pool - 1)]
    need = ((lengths + add.clamp(min=0) + page - 1) // page - held).clamp(min=0).sum()
    count = torch.minimum(free, need // 2) if c["tight"] else free
    e = lambda *s: torch.empty(s, device="cuda", dtype=torch.int32)  # noqa: E731
    return {"op": "slots", "T": T, "page": page, "lengths": lengths, "add": add, "held": held, "table": table,
            "ring": ring.contiguous(), "ring_state": torch.stack([torch.full_like(count, head), count]).int(),
            "slots": e(B, T), "positions": e(B, T), "granted": e(B), "lengths_out": e(B), "held_out": e(B),
            "ring_state_out": e(2)}


def _prepare_rotary(c, gen):
    B, T, Hq, Hk, D, R, dt = c["B"], c["T"], c["Hq"], c["Hk"], c["D"], c["R"], DTYPES[c["dtype"]]
    wide = _randn(gen, B, T, (Hq + Hk) * D + c["pad"]).to(dt)
    f = 10000.0 ** -(torch.arange(0, R, 2, dtype=torch.float64) / R)
    scale = 1.0
    if c["scaled"]:  # low frequencies stretched 32 times, a ramp between wavelengths of 1/32 and 1 of 8192 tokens
        turns = 8192 * f / (2 * math.pi)
        keep = ((turns - 1) / 31).clamp(0, 1)
        f, scale = f * (keep + (1 - keep) / 32), 1 + 0.1 * math.log(32)
    start = _randint(gen, 0, c["far"], B)
    t = torch.arange(T, device="cuda", dtype=torch.int32)
    positions = start[:, None] + t
    if c["ragged"]:
        positions = torch.where(t < _randint(gen, 0, T, B)[:, None], positions, -1)
    return {"op": "rotary", "q": wide[..., :Hq * D].unflatten(-1, (Hq, D)),
            "k": wide[..., Hq * D:(Hq + Hk) * D].unflatten(-1, (Hk, D)), "positions": positions.contiguous(),
            "inv_freq": f.float().cuda(), "layout": c["layout"], "scale": scale,
            "q_out": torch.zeros(B, T, Hq, D, dtype=dt, device="cuda"),
            "k_out": torch.zeros(B, T, Hk, D, dtype=dt, device="cuda")}


def _head_scale(gen, H):
    """Scales as calibration leaves them, powers of two."""
    return torch.exp2(_randint(gen, -3, 3, H).float())


def _prepare_store(c, gen):
    B, T, H, D, page, dt = c["B"], c["T"], c["H"], c["D"], c["page"], DTYPES[c["dtype"]]
    # some channels of the keys are much larger than the others
    k = _randn(gen, B, T, H, D) * torch.exp(0.7 * _randn(gen, H, D))
    v = _randn(gen, B, T, H, D)
    pages = -(-B * T * 5 // (4 * page)) + 1
    slots = torch.randperm(pages * page, generator=gen, device="cuda")[:B * T].int().view(B, T)
    if T > 1:  # a prompt fills its pages in order
        per = -(-T // page)
        order = torch.randperm(max(pages, B * per), generator=gen, device="cuda")[:B * per].int().view(B, per)
        pages = max(pages, B * per)
        t = torch.arange(T, device="cuda")
        slots = order[:, t // page] * page + (t % page).int()
    if c["ragged"]:
        slots = torch.where(torch.arange(T, device="cuda") < _randint(gen, 0, T, B)[:, None], slots, -1).int()
    return {"op": "store", "k": k.to(dt), "v": v.to(dt), "slots": slots.contiguous(), "page": page,
            "k_scale": _head_scale(gen, H), "v_scale": _head_scale(gen, H),
            "cache": torch.zeros(pages, H, page, 9 * D // 8, dtype=torch.uint8, device="cuda"),
            "k_out": torch.zeros(B, T, H, D, dtype=dt, device="cuda"),
            "v_out": torch.zeros(B, T, H, D, dtype=dt, device="cuda")}


def _prepare_attend(c, gen):
    B, T, Hq, H, D, L, page = c["B"], c["T"], c["Hq"], c["H"], c["D"], c["L"], c["page"]
    width = -(-L // page)
    pages = B * width + 3
    # a cache of normal values; a page is one block per head: the keys' codes and scales, then the values'
    cache = torch.empty(pages, H, page * 9 * D // 8, dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 27) // (H * page * D))
    for i in range(0, pages, step):
        part = cache[i:i + step]
        at = 0
        for _ in range(2):
            codes, scales = _quantise(_randn(gen, part.shape[0], H, page, D // 16, 16))
            codes = codes.flatten(-2).to(torch.uint8)
            codes = codes[..., 0::2] | (codes[..., 1::2] << 4)
            for piece in (codes, scales.float().to(torch.float8_e4m3fn).view(torch.uint8)):
                flat = piece.flatten(2)
                part[..., at:at + flat.shape[-1]] = flat
                at += flat.shape[-1]
    lengths = torch.full((B,), L, device="cuda", dtype=torch.int32)
    new = None
    if c["ragged"]:
        lengths = torch.maximum(_randint(gen, L // 4, L, B), torch.tensor(T, device="cuda")).int()
        if T > 1:
            new = _randint(gen, 1, T, B)
    table = torch.randperm(pages, generator=gen, device="cuda")[:B * width].int().view(B, width).contiguous()
    dt = DTYPES[c["dtype"]]
    return {"op": "attend", "q": (2 * _randn(gen, B, T, Hq, D)).to(dt),
            "cache": cache.view(pages, H, page, 9 * D // 8), "table": table, "lengths": lengths, "new": new,
            "window": c["window"], "scale": 1 / math.sqrt(D), "k_scale": _head_scale(gen, H) / 2,
            "v_scale": _head_scale(gen, H), "y": torch.zeros(B, T, Hq, D, dtype=dt, device="cuda"),
            "lse": torch.zeros(B, T, Hq, device="cuda")}


# ----------------------------------------------------------------- one pass
def run(state):
    return (_own if own else _plain)[state["op"]](state)


def _plain_slots(s):
    T, page, table, ring = s["T"], s["page"], s["table"], s["ring"]
    B, width = table.shape
    pool = ring.shape[0]
    head, count = s["ring_state"][0], s["ring_state"][1]
    ended = s["add"] < 0
    add = s["add"].clamp(0, T)
    total = s["lengths"] + add
    need = ((total + page - 1) // page - s["held"]).clamp(min=0)
    need = torch.where(ended | (total > width * page), 0, need)
    upto = need.cumsum(0)
    served = ~ended & (total <= width * page) & ((need == 0) | (upto <= count))
    need = torch.where(served, need, 0)
    granted = torch.where(served, add, 0)
    held = torch.where(ended, 0, s["held"] + need)
    lengths = torch.where(ended, 0, s["lengths"] + granted)
    col = torch.arange(width, device="cuda")
    from_ring = (head + (upto - need)[:, None] + col - s["held"][:, None]) % pool
    grown = (col >= s["held"][:, None]) & (col < held[:, None]) & ~ended[:, None]
    new_table = torch.where(grown, ring[from_ring.long()], table)
    # the pages of ended sequences, in order, behind the last free one
    back = torch.where(ended, s["held"], 0)
    to = (head + count + (back.cumsum(0) - back)[:, None] + col) % pool
    to = torch.where(col < back[:, None], to, pool)
    new_ring = torch.cat([ring, ring.new_zeros(1)]).scatter(0, to.flatten().long(), table.flatten())[:pool]
    t = torch.arange(T, device="cuda", dtype=torch.int32)
    there = t < granted[:, None]
    pos = s["lengths"][:, None] + t
    slot = new_table.gather(1, (pos // page).clamp(max=width - 1).long()) * page + pos % page
    taken = need.sum()
    return {"slots": torch.where(there, slot, -1).int(), "positions": torch.where(there, pos, -1).int(),
            "granted": granted.int(), "lengths": lengths.int(), "held": held.int(), "table": new_table,
            "ring": new_ring, "ring_state": torch.stack([(head + taken) % pool, count - taken + back.sum()]).int()}


def _plain_rotary(s):
    angle = s["positions"].double()[..., None, None] * s["inv_freq"].double()
    cos, sin = (torch.cos(angle) * s["scale"]).float(), (torch.sin(angle) * s["scale"]).float()
    there = (s["positions"] >= 0)[..., None, None]
    R = 2 * s["inv_freq"].shape[0]
    out = []
    for x in (s["q"], s["k"]):
        f = x.float()
        turned = f[..., :R]
        if s["layout"] == "half":
            a, b = turned[..., :R // 2], turned[..., R // 2:]
            turned = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
        else:
            a, b = turned[..., 0::2], turned[..., 1::2]
            turned = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
        out.append(torch.where(there, torch.cat([turned, f[..., R:]], -1), 0.0).to(x.dtype))
    return {"q": out[0], "k": out[1]}


def _quantise(u):
    """Codes and scales of [..., 16] values; a scale of rounding's borders is decided in 64 bits."""
    a = u.abs()
    q = (a.amax(-1).double() / 6).clamp(max=448)
    # e4m3: three bits behind the leading one, from 2^-6 on; steps of 2^-9 below
    step = torch.exp2(torch.frexp(q).exponent.clamp(min=-5).double() - 4)
    s = torch.round(q / step) * step
    d = s[..., None].float()
    code = torch.zeros_like(u, dtype=torch.int32)
    for i in range(7):  # a border between two codes goes to the even one
        border = (E2M1[i] + E2M1[i + 1]) / 2 * d
        code += (a > border) if i % 2 == 0 else (a >= border)
    code = torch.where(d > 0, code, 0)
    return code + 8 * (u < 0), s


def _values(code, s):
    mag = torch.tensor(E2M1, device=code.device)[code & 7]
    return torch.where(code >= 8, -mag, mag) * s[..., None].float()


def _plain_store(s):
    out = []
    for x, scale in ((s["k"], s["k_scale"]), (s["v"], s["v_scale"])):
        u = (x.float() / scale[:, None]).unflatten(-1, (-1, 16))
        val = _values(*_quantise(u)).flatten(-2) * scale[:, None]
        out.append(torch.where((s["slots"] >= 0)[..., None, None], val, 0.0).to(x.dtype))
    return {"k": out[0], "v": out[1]}


def _pages(s, b):
    """Keys and values [H, tokens, D] of one sequence's pages, without the heads' scales."""
    blocks = s["cache"][s["table"][b]].flatten(2)          # [width, H, bytes]
    width, H = blocks.shape[:2]
    page, D = s["cache"].shape[2], s["cache"].shape[3] * 8 // 9
    n, out = page * D // 2, []
    lut = torch.tensor(E2M1 + [-v for v in E2M1], device="cuda")
    for at in (0, n + page * D // 16):
        codes = blocks[..., at:at + n].unflatten(-1, (page, D // 2))
        scales = blocks[..., at + n:at + n + page * D // 16].contiguous().view(torch.float8_e4m3fn).float()
        both = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
        val = lut[both.int()].unflatten(-1, (-1, 16)) * scales.view(width, H, page, D // 16, 1)
        out.append(val.flatten(-2).transpose(0, 1).flatten(1, 2))
    return out


def _plain_attend(s):
    q = s["q"].float()
    B, T, Hq, D = q.shape
    H = s["cache"].shape[1]
    G = Hq // H
    y, lse = torch.zeros_like(q), torch.zeros(B, T, Hq, device="cuda")
    t = torch.arange(T, device="cuda")
    for b in range(B):
        k, v = _pages(s, b)
        j = torch.arange(k.shape[1], device="cuda")
        n = T if s["new"] is None else s["new"][b]
        pos = (s["lengths"][b] - n + t)[:, None]
        seen = (j <= pos) & (j < s["lengths"][b])
        if s["window"]:
            seen &= j > pos - s["window"]
        on = (t < n)[:, None, None]
        for h in range(H):
            qh = q[b, :, h * G:(h + 1) * G].transpose(0, 1)                     # [G,T,D]
            x = (qh @ k[h].T) * (s["scale"] * s["k_scale"][h])
            x = torch.where(seen, x, -math.inf)
            m = x.amax(-1, keepdim=True)
            e = torch.exp(x - m)
            total = e.sum(-1, keepdim=True)
            o = (e @ v[h]) / total * s["v_scale"][h]
            y[b, :, h * G:(h + 1) * G] = torch.where(on, o.transpose(0, 1), 0.0)
            lse[b, :, h * G:(h + 1) * G] = torch.where(on, (m + torch.log(total)).transpose(0, 1), 0.0)[..., 0]
    return {"y": y.to(s["q"].dtype), "lse": lse}


def _own_slots(s):
    import linear_attention_recurrence_step_gb300 as gdn
    o = gdn.gdn_page_slots(s["lengths"], s["add"], s["held"], s["ring_state"], s["table"], s["ring"], T=s["T"],
                           page=s["page"], slots=s["slots"], positions=s["positions"], granted=s["granted"],
                           lengths_out=s["lengths_out"], held_out=s["held_out"], ring_state_out=s["ring_state_out"])
    return {"slots": o.slots, "positions": o.positions, "granted": o.granted, "lengths": o.lengths_out,
            "held": o.held_out, "table": s["table"], "ring": s["ring"], "ring_state": o.ring_state_out}


def _own_rotary(s):
    import linear_attention_recurrence_step_gb300 as gdn
    o = gdn.gdn_rotary(s["q"], s["positions"], s["inv_freq"], k=s["k"], layout=s["layout"], scale=s["scale"],
                       q_out=s["q_out"], k_out=s["k_out"])
    return {"q": o.q, "k": o.k}


def _own_store(s):
    import linear_attention_recurrence_step_gb300 as gdn
    gdn.gdn_kv_append(s["k"], s["v"], s["slots"], s["cache"], k_scale=s["k_scale"], v_scale=s["v_scale"])
    o = gdn.gdn_kv_read(s["cache"], s["slots"], dtype=s["k"].dtype, k_scale=s["k_scale"], v_scale=s["v_scale"],
                        k=s["k_out"], v=s["v_out"])
    return {"k": o.k, "v": o.v}


def _own_attend(s):
    import linear_attention_recurrence_step_gb300 as gdn
    o = gdn.gdn_kv_attention(s["q"], s["cache"], s["table"], s["lengths"], new=s["new"], scale=s["scale"],
                             window=s["window"], k_scale=s["k_scale"], v_scale=s["v_scale"], y=s["y"], lse=s["lse"])
    return {"y": o.y, "lse": o.lse}


_plain = {"slots": _plain_slots, "rotary": _plain_rotary, "store": _plain_store, "attend": _plain_attend}
_own = {"slots": _own_slots, "rotary": _own_rotary, "store": _own_store, "attend": _own_attend}


# ------------------------------------------------- what a pass has to move
def work(case):
    c = case
    if c["op"] == "slots":
        # every length, count and place; a table entry read or written per page that changes hands
        pages = c["B"] * (c["T"] // c["page"] // 2 + 1)
        return {"bytes": 4 * (c["B"] * (2 * c["T"] + 6) + 2 * pages + 4), "flops": c["B"] * (2 * c["T"] + 10)}
    e = ESIZE[c["dtype"]]
    share = 0.5 if c["ragged"] else 1.0  # ragged lengths are uniform: half of the tokens are there
    if c["op"] == "rotary":
        heads = c["Hq"] + c["Hk"]
        n = c["B"] * c["T"]
        return {"bytes": share * n * heads * c["D"] * 2 * e + n * 4 + c["R"] * 2,
                "flops": share * n * (3 * heads + 10) * c["R"]}
    if c["op"] == "store":
        n = 2 * c["B"] * c["T"] * c["H"] * c["D"]  # written once and read once: codes and a scale per 16
        return {"bytes": share * n * (2 * e + 2 * 9 / 16) + c["B"] * c["T"] * 4, "flops": share * n * 6}
    # lengths are uniform from a quarter of the longest on, new tokens from 1 on
    L = c["L"] * (5 / 8 if c["ragged"] else 1.0)
    n = (c["T"] + 1) / 2 if c["ragged"] else c["T"]
    first = max(L - n - c["window"], 0.0) if c["window"] else 0.0
    seen = min(L - n / 2, c["window"]) if c["window"] else L - n / 2
    return {"bytes": c["B"] * (c["H"] * (L - first) * c["D"] * 9 / 8 + n * c["Hq"] * (2 * c["D"] * e + 4)),
            "flops": 4 * c["D"] * c["B"] * n * c["Hq"] * max(seen, 1.0)}


# ------------------------------------- the definitions, step by step in f64
def exact(case, seed):
    if case["op"] == "slots":
        return None  # whole numbers only
    s = prepare(case, seed)
    return {"rotary": _exact_rotary, "store": _exact_store, "attend": _exact_attend}[s["op"]](s)


def _exact_rotary(s):
    f, pos = s["inv_freq"].double(), s["positions"].double()
    out = {}
    for name in ("q", "k"):
        x = s[name].double()
        y = x.clone()
        n = f.shape[0]
        for i in range(n):
            a, b = (i, i + n) if s["layout"] == "half" else (2 * i, 2 * i + 1)
            c, d = torch.cos(pos * f[i])[..., None], torch.sin(pos * f[i])[..., None]
            y[..., a] = s["scale"] * (x[..., a] * c - x[..., b] * d)
            y[..., b] = s["scale"] * (x[..., a] * d + x[..., b] * c)
        y[s["positions"] < 0] = 0
        out[name] = y
    return out


def _exact_store(s):
    # every finite e4m3 value from its byte, in order; the nearest, between two the one with the even byte
    grid = torch.tensor([(b & 7) * 2.0 ** -9 if b < 8 else (8 + (b & 7)) * 2.0 ** ((b >> 3) - 10)
                         for b in range(127)], dtype=torch.float64, device="cuda")
    codes = torch.tensor(E2M1, dtype=torch.float64, device="cuda")

    def nearest(x, values):
        hi = torch.searchsorted(values, x.contiguous()).clamp(1, len(values) - 1)
        lo = hi - 1
        up, down = values[hi] - x, x - values[lo]
        return torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)

    out = {}
    for name in ("k", "v"):
        g = s[name + "_scale"].double()[:, None]
        u = s[name].double() / g
        B, T, H, D = u.shape
        u = u.reshape(B, T, H, D // 16, 16)
        size = u.abs().max(-1, keepdim=True).values
        sc = grid[nearest((size / 6).clamp(max=448), grid)]
        ratio = torch.where(sc > 0, u.abs() / torch.where(sc > 0, sc, torch.ones_like(sc)), torch.zeros_like(u))
        val = codes[nearest(ratio.clamp(max=6), codes)] * sc * torch.sign(u)
        val = val.reshape(B, T, H, D) * g
        val[s["slots"] < 0] = 0
        out[name] = val
    return out


def _exact_attend(s):
    q, cache, table = s["q"].double(), s["cache"], s["table"]
    B, T, Hq, D = q.shape
    H, page = cache.shape[1], cache.shape[2]
    G, n = Hq // H, page * D // 2
    y, lse = torch.zeros_like(q), torch.zeros(B, T, Hq, device="cuda", dtype=torch.float64)
    mags = torch.tensor(E2M1, dtype=torch.float64, device="cuda")
    for b in range(B):
        L = int(s["lengths"][b])
        new = T if s["new"] is None else int(s["new"][b])
        lo = max(0, L - new - s["window"] + 1) // page if s["window"] else 0
        ids = table[b, lo:-(-L // page)].long()
        for h in range(H):
            block = cache[ids, h].reshape(len(ids), -1)
            kv = []
            for at, g in ((0, s["k_scale"][h]), (n + page * D // 16, s["v_scale"][h])):
                byte = block[:, at:at + n].reshape(-1, D // 2)
                nib = torch.empty(byte.shape[0], D, dtype=torch.long, device="cuda")
                nib[:, 0::2], nib[:, 1::2] = byte % 16, byte // 16
                sb = block[:, at + n:at + n + page * D // 16].reshape(-1, D // 16).long()
                e, m = (sb >> 3) & 15, (sb & 7).double()
                sv = torch.where(e > 0, (1 + m / 8) * torch.exp2(e.double() - 7), m * 2.0 ** -9)
                val = mags[nib % 8] * (1 - 2 * (nib // 8)) * sv.repeat_interleave(16, 1)
                kv.append(val[:L - lo * page] * g.double())
            j = lo * page + torch.arange(kv[0].shape[0], device="cuda")
            pos = L - new + torch.arange(new, device="cuda")[:, None]
            hide = j > pos
            if s["window"]:
                hide |= j <= pos - s["window"]
            for i in range(h * G, (h + 1) * G):
                x = (q[b, :new, i] @ kv[0].T * s["scale"]).masked_fill(hide, -math.inf)
                z = torch.logsumexp(x, 1)
                y[b, :new, i] = torch.exp(x - z[:, None]) @ kv[1]
                lse[b, :new, i] = z
    return {"y": y, "lse": lse}
