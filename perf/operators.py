"""Cases for the operators that stand around the recurrence in a serving step.

A recurrent layer takes its projections through a short causal convolution,
runs a recurrence over the tokens (the gated delta rule, or the selective
state space scan timed here), normalises what comes out under its gate, and
the model's logits are sampled; the count of sampled tokens that match a
draft is what the rollback calls take.  Each case is one call of one of the
four operators:

  conv    y[t,c] = silu(bias[c] + sum_j weight[c,j] x[t-W+1+j,c]), with the last
          W-1 inputs of a sequence kept as its state
  scan    s <- exp(dt_t A) s + dt_t x_t B_t^T;  y_t = s C_t + D x_t
  norm    u = residual + scale x;  y = u / rms(u) * weight * silu(gate)
  sample  temperature, top-k, top-p and min-p, then the largest
          exp((l - max)/T) / noise among the tokens that are left

``own`` picks the side that ``run`` takes: elementary torch operations in 32
bits (False) or the library's kernels (True).
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
ESIZE = {"f32": 4, "bf16": 2, "f16": 2}


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # one new token for each of 32 sequences: q, k and v channels of 16 key heads and 32 value
        # heads of 128 together; a few microseconds, so the call itself counts
        {"name": "conv_decode_b32", "op": "conv", "B": 32, "T": 1, "C": 8192, "W": 4, "dtype": "bf16",
         "bias": False, "ragged": False, "pad": 0},
        # the rollback after eight draft tokens: every sequence keeps its own accepted prefix
        {"name": "conv_verify_b16_t8", "op": "conv", "B": 16, "T": 8, "C": 8192, "W": 4, "dtype": "f16",
         "bias": True, "ragged": True, "pad": 0},
        # a long prompt; x is a slice of a wider fused projection (its rows lie 8192 + 4096 apart)
        {"name": "conv_prompt_t4096", "op": "conv", "B": 1, "T": 4096, "C": 8192, "W": 4, "dtype": "bf16",
         "bias": True, "ragged": False, "pad": 4096},
        # one token per sequence: the whole f32 state is read and written
        {"name": "scan_decode_b32", "op": "scan", "B": 32, "T": 1, "H": 32, "P": 128, "G": 16, "N": 128,
         "dtype": "bf16", "ragged": False},
        # eight draft tokens, ragged draft lengths, heads of 64
        {"name": "scan_verify_b16_t8", "op": "scan", "B": 16, "T": 8, "H": 64, "P": 64, "G": 8, "N": 128,
         "dtype": "f32", "ragged": True},
        # a long prompt of one sequence
        {"name": "scan_prompt_t4096", "op": "scan", "B": 1, "T": 4096, "H": 32, "P": 128, "G": 16, "N": 128,
         "dtype": "bf16", "ragged": False},
        # the norm after the recurrence for one new token of 16 sequences: per head, under the gate
        {"name": "norm_gate_decode", "op": "norm", "M": 16, "K": 32, "D": 128, "dtype": "bf16",
         "gate": "after", "residual": False},
        # the norm before a block: residual added with its scale, a width that is no power of two
        {"name": "norm_residual_odd", "op": "norm", "M": 1000, "K": 1, "D": 5001, "dtype": "f32",
         "gate": "none", "residual": True},
        # the norm after the recurrence over a long prompt
        {"name": "norm_gate_t4096", "op": "norm", "M": 4096, "K": 32, "D": 128, "dtype": "bf16",
         "gate": "after", "residual": False},
        # one token of one sequence, top-k 50 (the smallest sampling call)
        {"name": "sample_topk_b1", "op": "sample", "R": 1, "V": 32000, "dtype": "f32", "mode": "topk",
         "sigma": 2.5},
        # verification of eight draft positions of 16 sequences, every row with its own settings
        {"name": "sample_verify_b16_t8", "op": "sample", "R": 128, "V": 131072, "dtype": "bf16",
         "mode": "mixed", "sigma": 2.0},
        # a large batch, plain temperature sampling over the whole vocabulary
        {"name": "sample_full_b256", "op": "sample", "R": 256, "V": 100003, "dtype": "bf16", "mode": "full",
         "sigma": 1.5},
    ]


def _log_int(rng, lo, hi):
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return min(max(n, lo), hi)


def _odd(rng, n, step):
    """n as drawn, or (half of the time) the nearest multiple of step below it."""
    n = n if rng.random() < 0.5 else max(step, n // step * step)
    return n + 1 if n % 1024 == 0 and n // 1024 == 3 else n


def draw(rng):
    op = rng.choice(["conv", "scan", "norm", "sample"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op == "conv":
        C = _odd(rng, _log_int(rng, 96, 10000), 64)
        most = 4096 * 8192 * 2 // (C * ESIZE[dtype])
        T = rng.choice([1, 1, rng.randint(2, 16), _log_int(rng, 17, min(4096, most))])
        B = _log_int(rng, 1, max(1, min(128, most // T)))
        return {"op": op, "B": B, "T": T, "C": C, "W": rng.choice([2, 3, 4, 4, 4]), "dtype": dtype,
                "bias": rng.random() < 0.5, "ragged": rng.random() < 0.5, "pad": rng.choice([0, 0, 64, 33])}
    if op == "scan":
        N, P = rng.choice([16, 64, 128, 128]), rng.choice([32, 64, 64, 80, 128])
        G = rng.choice([1, 2, 4, 8])
        H = G * rng.randint(1, max(1, 64 // G))
        T = rng.choice([1, rng.randint(2, 16), _log_int(rng, 17, 4096)])
        top = min(25 * 32 * 128 * 128 // (H * P * N), 4096 * 32 * 128 // (T * H * P))
        return {"op": op, "B": _log_int(rng, 1, max(1, min(64, top))), "T": T, "H": H, "P": P, "G": G, "N": N,
                "dtype": dtype, "ragged": rng.random() < 0.5}
    if op == "norm":
        K = rng.choice([1, 1, 8, 32])
        D = _odd(rng, _log_int(rng, 64, 16384 // K), 8)
        gate, residual = rng.choice(["none", "after", "first"]), rng.random() < 0.5
        parts = 2 + (gate != "none") + 2 * residual
        M = _log_int(rng, 1, min(20000, 100000000 // (K * D * parts * ESIZE[dtype])))
        return {"op": op, "M": M, "K": K, "D": D, "dtype": dtype, "gate": gate, "residual": residual}
    V = _odd(rng, _log_int(rng, 1000, 200000), 64)
    R = _log_int(rng, 1, min(256, 256 * 100003 * 6 // (V * (ESIZE[dtype] + 4))))
    return {"op": op, "R": R, "V": V, "dtype": dtype, "mode": rng.choice(["topk", "topp", "minp", "mixed", "full"]),
            "sigma": rng.choice([1.0, 2.0, 3.0])}


# --------------------------------------------------------------- the inputs
def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return {"conv": _prepare_conv, "scan": _prepare_scan, "norm": _prepare_norm,
            "sample": _prepare_sample}[case["op"]](case, gen)


def _randn(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda")


def _rand(gen, *shape):
    return torch.rand(shape, generator=gen, device="cuda")


def _lengths(case, gen):
    if not case["ragged"]:
        return None
    return torch.randint(0, case["T"] + 1, (case["B"],), generator=gen, device="cuda", dtype=torch.int32)


def _prepare_conv(c, gen):
    B, T, C, W, dt = c["B"], c["T"], c["C"], c["W"], DTYPES[c["dtype"]]
    wide = _randn(gen, B, T, C + c["pad"]).to(dt)
    return {"op": "conv", "x": wide[..., :C], "weight": (_randn(gen, C, W) / math.sqrt(W)).to(dt),
            "state": _randn(gen, B, W - 1, C).to(dt), "bias": (0.1 * _randn(gen, C)).to(dt) if c["bias"] else None,
            "lengths": _lengths(c, gen), "y": torch.zeros(B, T, C, dtype=dt, device="cuda"),
            "state_out": torch.empty(B, W - 1, C, dtype=dt, device="cuda")}


def _prepare_scan(c, gen):
    B, T, H, P, G, N, dt = c["B"], c["T"], c["H"], c["P"], c["G"], c["N"], DTYPES[c["dtype"]]
    # x, B and C are slices of one convolution's output, as a layer has them
    xbc = _randn(gen, B, T, H * P + 2 * G * N)
    xbc[..., H * P:] /= math.sqrt(math.sqrt(N))
    xbc = xbc.to(dt)
    # steps log-uniform on [1e-3, 1e-1] through the inverse of softplus, decay rates on [1, 16]
    step = torch.exp(_rand(gen, H) * (math.log(0.1) - math.log(1e-3)) + math.log(1e-3))
    return {"op": "scan", "x": xbc[..., :H * P].unflatten(-1, (H, P)),
            "B": xbc[..., H * P:H * P + G * N].unflatten(-1, (G, N)),
            "C": xbc[..., H * P + G * N:].unflatten(-1, (G, N)),
            "dt": (0.5 * _randn(gen, B, T, H)).to(dt), "A": -(1 + 15 * _rand(gen, H)),
            "dt_bias": step + torch.log(-torch.expm1(-step)), "D": _randn(gen, H),
            "state": 0.1 * _randn(gen, B, H, P, N), "lengths": _lengths(c, gen),
            "y": torch.zeros(B, T, H, P, dtype=dt, device="cuda"),
            "state_out": torch.empty(B, H, P, N, device="cuda")}


def _prepare_norm(c, gen):
    M, K, D, dt = c["M"], c["K"], c["D"], DTYPES[c["dtype"]]
    return {"op": "norm", "x": _randn(gen, M, K, D).to(dt), "weight": (1 + 0.1 * _randn(gen, D)).to(dt),
            "gate": _randn(gen, M, K, D).to(dt) if c["gate"] != "none" else None, "first": c["gate"] == "first",
            "residual": _randn(gen, M, K, D).to(dt) if c["residual"] else None, "scale": 0.5, "eps": 1e-6,
            "y": torch.empty(M, K, D, dtype=dt, device="cuda"),
            "residual_out": torch.empty(M, K, D, dtype=dt, device="cuda") if c["residual"] else None}


def _prepare_sample(c, gen):
    R, V, mode = c["R"], c["V"], c["mode"]
    logits = c["sigma"] * _randn(gen, R, V)
    # a few tokens stand out, as after a trained model's last layer; some places are masked
    at = torch.randint(0, V, (R, 24), generator=gen, device="cuda")
    logits.scatter_add_(1, at, 4 * c["sigma"] * _rand(gen, R, 24))
    banned = torch.randint(0, V, (R, max(1, V // 100)), generator=gen, device="cuda")
    if mode != "full":
        logits.scatter_(1, banned, -math.inf)
    noise = torch.empty(R, V, device="cuda").exponential_(generator=gen).clamp_(min=1e-30)
    on = torch.ones(R, device="cuda")
    s = {"op": "sample", "logits": logits.to(DTYPES[c["dtype"]]), "noise": noise, "temperature": 0.8 * on,
         "top_k": torch.zeros(R, dtype=torch.int32, device="cuda"), "top_p": on.clone(), "min_p": 0 * on}
    if mode == "topk":
        s["top_k"] += 50
    if mode == "topp":
        s["top_p"] *= 0.95
    if mode == "minp":
        s["min_p"] += 0.05
    if mode == "mixed":  # every request brings its own settings; an eighth of them are greedy
        s["temperature"] = 0.5 + _rand(gen, R)
        s["temperature"][torch.rand(R, generator=gen, device="cuda") < 0.125] = 0
        s["top_k"] = torch.randint(0, 200, (R,), generator=gen, device="cuda", dtype=torch.int32)
        s["top_k"][s["top_k"] > 150] = 0
        s["top_p"] = 0.7 + 0.3 * _rand(gen, R)
        s["min_p"] = 0.05 * _rand(gen, R) * (_rand(gen, R) < 0.5)
    s["token"] = torch.empty(R, dtype=torch.int32, device="cuda")
    s["logprob"] = torch.empty(R, device="cuda")
    return s


# ----------------------------------------------------------------- one pass
def run(state):
    return (_own if own else _plain)[state["op"]](state)


def _valid(s, T):
    """[B,T] truth values of the steps that a sequence has, or None for all."""
    if s["lengths"] is None:
        return None
    return torch.arange(T, device="cuda") < s["lengths"][:, None]


def _plain_conv(s):
    x, state, W = s["x"].float(), s["state"].float(), s["weight"].shape[1]
    B, T, C = x.shape
    line = torch.cat([state, x], 1)
    y = (line.unfold(1, W, 1) * s["weight"].float()).sum(-1)
    if s["bias"] is not None:
        y = y + s["bias"].float()
    y = y * torch.sigmoid(y)
    n = s["lengths"]
    if n is None:
        return {"y": y.to(s["x"].dtype), "state": line[:, T:].to(s["x"].dtype)}
    y = torch.where(_valid(s, T)[..., None], y, 0.0)
    at = (n[:, None] + torch.arange(W - 1, device="cuda"))[..., None].expand(B, W - 1, C)
    return {"y": y.to(s["x"].dtype), "state": line.gather(1, at.long()).to(s["x"].dtype)}


def _segments(a):
    """exp(a[j+1] + ... + a[i]) for j <= i, else 0, over the last axis."""
    c = a.cumsum(-1)
    d = c[..., :, None] - c[..., None, :]
    n = a.shape[-1]
    return torch.exp(d.masked_fill(~torch.ones(n, n, dtype=torch.bool, device=a.device).tril(), -math.inf))


def _plain_scan(s):
    x, Bm, Cm = s["x"].float(), s["B"].float(), s["C"].float()
    B, T, H, P = x.shape
    L = min(64, T)
    n = -(-T // L)
    dt = torch.nn.functional.softplus(s["dt"].float() + s["dt_bias"], threshold=60.0)
    valid = _valid(s, T)
    if valid is not None:
        dt = torch.where(valid[..., None], dt, 0.0)
    fill = n * L - T

    def chunks(v):  # [B,T,...] -> [B,n,L,...]; a step of length zero changes nothing
        if fill:
            v = torch.cat([v, v.new_zeros(B, fill, *v.shape[2:])], 1)
        return v.unflatten(1, (n, L))

    per = H // Bm.shape[2]
    xd = chunks(x * dt[..., None])
    Bc, Cc = (chunks(v) for v in (Bm, Cm))
    a = chunks(dt * s["A"]).permute(0, 1, 3, 2)                                    # [B,n,H,L]
    gram = torch.einsum("bnlgi,bnsgi->bngls", Cc, Bc).repeat_interleave(per, 2)
    y = torch.einsum("bnhls,bnshp->bnlhp", gram * _segments(a), xd)
    # the state that each chunk adds, and the state that each chunk starts from
    w = torch.exp(a.sum(-1, keepdim=True) - a.cumsum(-1)).permute(0, 1, 3, 2)      # [B,n,L,H]
    Bh, Ch = Bc.repeat_interleave(per, 3), Cc.repeat_interleave(per, 3)
    add = torch.einsum("bnlhp,bnlhi->bnhpi", xd * w[..., None], Bh)
    first = torch.cat([s["state"][:, None], add], 1)
    carry = _segments(torch.cat([a.new_zeros(B, 1, H), a.sum(-1)], 1).permute(0, 2, 1))
    at = torch.einsum("bhij,bjhpk->bihpk", carry, first)
    y = y + torch.einsum("bnhpi,bnlhi->bnlhp", at[:, :n], Ch) * torch.exp(a.cumsum(-1)).permute(0, 1, 3, 2)[..., None]
    y = y.flatten(1, 2)[:, :T] + s["D"][:, None] * x
    if valid is not None:
        y = torch.where(valid[..., None, None], y, 0.0)
    return {"y": y.to(s["x"].dtype), "state": at[:, n]}


def _plain_norm(s):
    u, g = s["x"].float(), None
    if s["gate"] is not None:
        g = s["gate"].float()
        g = g * torch.sigmoid(g)
    if g is not None and s["first"]:
        u = u * g
    out = {}
    if s["residual"] is not None:
        u = s["residual"].float() + s["scale"] * u
        out["residual"] = u.to(s["x"].dtype)
    y = u * torch.rsqrt(u.square().mean(-1, keepdim=True) + s["eps"]) * s["weight"].float()
    if g is not None and not s["first"]:
        y = y * g
    out["y"] = y.to(s["x"].dtype)
    return out


def _plain_sample(s):
    l, noise, k = s["logits"].float(), s["noise"], s["top_k"][:, None]
    V = l.shape[1]
    top = l.max(1, keepdim=True).values
    greedy = s["temperature"][:, None] <= 0
    d = (l - top) / torch.where(greedy, 1.0, s["temperature"][:, None])
    e = torch.exp(d)
    order = torch.sort(l, dim=1, descending=True, stable=True).indices
    es = e.gather(1, order)
    rank = torch.arange(V, device="cuda")
    keep = (k <= 0) | (rank < k)
    es_k = torch.where(keep, es, 0.0)
    before = es_k.cumsum(1) - es_k
    p = s["top_p"][:, None]
    keep &= (p >= 1) | (before < p * es_k.sum(1, keepdim=True))
    keep &= es >= s["min_p"][:, None]
    keep[:, 0] = True
    kept = torch.zeros_like(keep).scatter_(1, order, keep)
    key = torch.where(kept, e / noise, -1.0)
    token = torch.where(greedy[:, 0], l.argmax(1), key.argmax(1))
    logprob = d.gather(1, token[:, None])[:, 0] - torch.log(e.sum(1))
    return {"token": token.to(torch.int32), "logprob": logprob}


def _own_conv(s):
    import linear_attention_recurrence_step_gb300 as gdn
    o = gdn.gdn_causal_conv(s["x"], s["weight"], s["state"], bias=s["bias"], lengths=s["lengths"], y=s["y"],
                            state_out=s["state_out"])
    return {"y": o.y, "state": o.state_out}


def _own_scan(s):
    import linear_attention_recurrence_step_gb300 as gdn
    o = gdn.gdn_selective_scan(s["x"], s["dt"], s["A"], s["B"], s["C"], s["state"], D=s["D"], dt_bias=s["dt_bias"],
                               softplus=True, lengths=s["lengths"], y=s["y"], state_out=s["state_out"])
    return {"y": o.y, "state": o.state_out}


def _own_norm(s):
    import linear_attention_recurrence_step_gb300 as gdn
    o = gdn.gdn_gated_norm(s["x"], s["weight"], gate=s["gate"], gate_first=s["first"], residual=s["residual"],
                           residual_scale=s["scale"], eps=s["eps"], y=s["y"], residual_out=s["residual_out"])
    if s["residual"] is None:
        return {"y": o.y}
    return {"y": o.y, "residual": o.residual_out}


def _own_sample(s):
    import linear_attention_recurrence_step_gb300 as gdn
    o = gdn.gdn_sample(s["logits"], s["noise"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"],
                       min_p=s["min_p"], token=s["token"], logprob=s["logprob"])
    return {"token": o.token, "logprob": o.logprob}


_plain = {"conv": _plain_conv, "scan": _plain_scan, "norm": _plain_norm, "sample": _plain_sample}
_own = {"conv": _own_conv, "scan": _own_scan, "norm": _own_norm, "sample": _own_sample}


# ------------------------------------------------- what a pass has to move
def work(case):
    c, e = case, ESIZE[case["dtype"]]
    if c["op"] == "conv":
        n, st = c["B"] * c["T"] * c["C"], c["B"] * (c["W"] - 1) * c["C"]
        share = 0.5 if c["ragged"] else 1.0  # ragged lengths are uniform: half of the steps are there
        return {"bytes": 2 * n * e * share + 2 * st * e + c["C"] * (c["W"] + c["bias"]) * e,
                "flops": share * n * (2 * c["W"] + 4)}
    if c["op"] == "scan":
        tok, share = c["B"] * c["T"], 0.5 if c["ragged"] else 1.0
        st = c["B"] * c["H"] * c["P"] * c["N"]
        ins = tok * (2 * c["H"] * c["P"] + 2 * c["G"] * c["N"] + c["H"]) * e
        return {"bytes": ins * share + 2 * st * 4, "flops": share * tok * c["H"] * c["P"] * (5 * c["N"] + 3)}
    if c["op"] == "norm":
        n = c["M"] * c["K"] * c["D"]
        parts = 2 + (c["gate"] != "none") + 2 * c["residual"]
        return {"bytes": n * e * parts + c["D"] * e, "flops": n * (4 + 5 * (c["gate"] != "none") + 2 * c["residual"])}
    # the noise of a token counts where the token can be left: of all, or of the first top-k
    n, left = c["R"] * c["V"], {"full": c["R"] * c["V"], "topk": 50 * c["R"]}.get(c["mode"], c["R"])
    return {"bytes": n * e + left * 4 + c["R"] * 24, "flops": 4 * n}


# ------------------------------------- the definitions, step by step in f64
def exact(case, seed):
    s = prepare(case, seed)
    return {"conv": _exact_conv, "scan": _exact_scan, "norm": _exact_norm, "sample": _exact_sample}[s["op"]](s)


def _exact_conv(s):
    x, w = s["x"].double(), s["weight"].double()
    B, T, C = x.shape
    W = w.shape[1]
    acc = torch.zeros_like(x) if s["bias"] is None else s["bias"].double().expand(B, T, C).clone()
    old = s["state"].double()
    for j in range(W):
        back = W - 1 - j  # tap j reads the input that many steps ago
        if back < T:
            acc[:, back:] += w[:, j] * x[:, :T - back]
        for t in range(min(back, T)):
            acc[:, t] += w[:, j] * old[:, W - 1 + t - back]
    y = acc / (1 + torch.exp(-acc))
    state = torch.empty_like(old)
    for b in range(B):
        n = T if s["lengths"] is None else int(s["lengths"][b])
        y[b, n:] = 0
        for i in range(W - 1):
            t = n - (W - 1) + i
            state[b, i] = x[b, t] if t >= 0 else old[b, W - 1 + t]
    return {"y": y, "state": state}


def _exact_scan(s):
    x, Bm, Cm, st = s["x"].double(), s["B"].double(), s["C"].double(), s["state"].double()
    B, T, H, P = x.shape
    per = H // Bm.shape[2]
    raw = s["dt"].double() + s["dt_bias"].double()
    dt = torch.log1p(torch.exp(-raw.abs())) + raw.clamp(min=0)
    g = torch.exp(dt * s["A"].double())
    y = torch.zeros_like(x)
    n = torch.full((B,), T, device=x.device) if s["lengths"] is None else s["lengths"]
    for t in range(T):
        Bt, Ct = (v[:, t].repeat_interleave(per, 1) for v in (Bm, Cm))             # [B,H,N]
        new = g[:, t, :, None, None] * st + (dt[:, t, :, None] * x[:, t])[..., None] * Bt[:, :, None]
        on = (t < n)[:, None, None]
        y[:, t] = torch.where(on, (new @ Ct[..., None])[..., 0] + s["D"].double()[:, None] * x[:, t], y[:, t])
        st = torch.where(on[..., None], new, st)
    return {"y": y, "state": st}


def _exact_norm(s):
    u = s["x"].double()
    gate = None if s["gate"] is None else s["gate"].double()
    if gate is not None and s["first"]:
        u = u * gate / (1 + torch.exp(-gate))
    out = {}
    if s["residual"] is not None:
        u = s["residual"].double() + s["scale"] * u
        out["residual"] = u
    y = u / torch.sqrt((u * u).sum(-1, keepdim=True) / u.shape[-1] + s["eps"]) * s["weight"].double()
    out["y"] = y if gate is None or s["first"] else y * gate / (1 + torch.exp(-gate))
    return out


def _exact_sample(s):
    token = _plain_sample(s)["token"].long()  # which token: a whole number, compared as such
    l = s["logits"].double()
    t = s["temperature"].double()
    z = l / torch.where(t > 0, t, torch.ones_like(t))[:, None]
    return {"token": None, "logprob": z.gather(1, token[:, None])[:, 0] - torch.logsumexp(z, 1)}
