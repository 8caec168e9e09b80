"""Plain float64 forms of the operators around the recurrence, step by step,
with a bound on the rounding error of a float32 evaluation beside each value.

The bounds are worst-case sums in units of u = 2^-24: every product, sum and
function value of the float32 evaluation is off by at most a few u of its
magnitude, and magnitudes are carried through the same sums with absolute
values.  Stores to bf16 / f16 add half a unit of the stored type (the tests
add it).
"""
from __future__ import annotations

import numpy as np

U = 2.0 ** -24


def silu(x):
    with np.errstate(over="ignore", invalid="ignore"):
        return x / (1.0 + np.exp(-x))


def conv(x, w, bias, state, lengths, act=True):
    """x [B,T,C], w [C,W], state [B,W-1,C] (or None), lengths [B] (or None).
    Returns y, bound on |error of y|, state_out, valid [B,T]."""
    B, T, C = x.shape
    W = w.shape[1]
    old = np.zeros((B, W - 1, C)) if state is None else state
    n = np.full(B, T) if lengths is None else np.clip(lengths, 0, T)
    line = np.concatenate([old, x], 1)
    y = np.zeros((B, T, C))
    mag = np.zeros((B, T, C))
    for t in range(T):
        s = np.zeros((B, C)) if bias is None else np.broadcast_to(bias, (B, C)).copy()
        m = np.abs(s)
        for j in range(W):
            term = w[:, j] * line[:, t + j]
            s = s + term
            m = m + np.abs(term)
        y[:, t], mag[:, t] = s, m
    # W fused products: at most W roundings of partial sums of magnitude <= mag
    err = (W + 1) * U * mag
    if act:
        # |d silu| <= 1.1; exp, sum and quotient: the exponential of s is off by
        # 2 + |s| units or so, the quotient and the product by 4 more
        err = 1.1 * err + (8 + 2 * np.abs(y)) * U * np.abs(silu(y)) + 1e-37
        y = silu(y)
    out = np.stack([np.concatenate([old[b], x[b, :n[b]]])[n[b]:n[b] + W - 1] for b in range(B)])
    return y, err, out, np.arange(T)[None] < n[:, None]


def scan(x, dt, A, Bm, Cm, D, dt_bias, state, lengths, softplus=True):
    """x [B,T,H,P], dt [B,T,H], Bm, Cm [B,T,G,N].  Returns y, its bound,
    state_out, its bound, valid [B,T]."""
    B, T, H, P = x.shape
    G, N = Bm.shape[2:]
    s = np.zeros((B, H, P, N)) if state is None else state.copy()
    E = np.zeros_like(s)
    n = np.full(B, T) if lengths is None else np.clip(lengths, 0, T)
    y, ye = np.zeros(x.shape), np.zeros(x.shape)
    for t in range(T):
        raw = dt[:, t] + (0 if dt_bias is None else dt_bias)
        dl = np.log1p(np.exp(-np.abs(raw))) + np.maximum(raw, 0) if softplus else raw
        # units of dl: the sum, then (softplus) log1p and exp
        dl_u = np.abs(raw) + np.abs(dt[:, t]) + (0 if dt_bias is None else np.abs(dt_bias)) + 8 * np.abs(dl)
        g = np.exp(dl * A)
        g_u = (np.abs(A) * (dl_u + 2 * np.abs(dl)) + 4) * g               # units of the decay
        Bt, Ct = (np.repeat(v[:, t], H // G, 1) for v in (Bm, Cm))
        dx = dl[..., None] * x[:, t]
        dx_u = (dl_u + 2 * np.abs(dl))[..., None] * np.abs(x[:, t])
        add = dx[..., None] * Bt[:, :, None]
        new = g[..., None, None] * s + add
        Enew = g[..., None, None] * E + U * (g_u[..., None, None] * np.abs(s) + dx_u[..., None] * np.abs(Bt)[:, :, None]
                                             + 3 * (np.abs(g[..., None, None] * s) + np.abs(add)))
        on = (t < n)[:, None, None, None]
        s, E = np.where(on, new, s), np.where(on, Enew, E)
        skip = 0 if D is None else D[None, :, None] * x[:, t]
        y[:, t] = (s * Ct[:, :, None]).sum(-1) + skip
        ye[:, t] = (E * np.abs(Ct)[:, :, None]).sum(-1) + U * (8 * (np.abs(s) * np.abs(Ct)[:, :, None]).sum(-1)
                                                               + N ** 0.5 * np.abs(y[:, t]) + 2 * np.abs(skip))
    return y, ye, s, E, np.arange(T)[None] < n[:, None]


def norm(x, w, gate, first, residual, scale, eps):
    """x, gate, residual [..., K, D]; w [D] or [K,D].  Returns y, bound, new
    residual (or None), its bound."""
    D = x.shape[-1]
    gs = None if gate is None else silu(gate)
    g_u = 0 if gate is None else 8 + 2 * np.abs(gate)
    u, e = x, np.zeros_like(x)
    if gs is not None and first:
        u = x * gs
        e = (g_u + 1) * U * np.abs(u)
    r = rb = None
    if residual is not None:
        # scale is rounded to float32, one fused product and sum
        e = np.abs(scale) * e + 2 * U * np.abs(scale * u)
        u = residual + scale * u
        e = e + U * np.abs(u)
        r, rb = u, e
    ms = (u * u).mean(-1, keepdims=True)
    # the sum of squares by a tree of few levels over runs of at most 40 terms,
    # and the error of its terms
    ms_e = (2 * np.abs(u) * e).mean(-1, keepdims=True) + 64 * U * ms
    rel = 0.5 * ms_e / (ms + eps) + 6 * U
    inv = 1 / np.sqrt(ms + eps)
    y = u * inv * w
    ye = np.abs(inv * w) * e + (rel + 3 * U) * np.abs(y)
    if gs is not None and not first:
        y, ye = y * gs, ye * np.abs(gs) + (g_u + 1) * U * np.abs(y * gs)
    return y, ye + 1e-37, r, rb


def kept_order(l, temperature, top_k, top_p, min_p):
    """Indexes of the tokens of one row that are left, best first, and e."""
    l = np.where(np.isnan(l), -np.inf, np.minimum(l, np.finfo(np.float32).max)).astype(np.float64)
    if not np.isfinite(l).any():
        return np.zeros(0, int), np.zeros_like(l), l
    t = temperature if temperature > 0 else 1.0
    with np.errstate(over="ignore"):
        e = np.exp((l - l.max()) / t)
    order = np.argsort(-l, kind="stable")
    m = len(l)
    if not temperature > 0:
        m = 1
    if 0 < top_k < len(l):
        m = min(m, top_k)
    es = e[order]
    if top_p < 1 and m > 1:
        kept = es[:m]
        before = np.concatenate([[0.0], np.cumsum(kept)[:-1]])
        m = min(m, max(1, int((before < top_p * kept.sum()).sum())))
    if min_p > 0:
        m = min(m, max(1, int((es >= min_p).sum()) if min_p <= 1 else 1))
    return order[:m], e, l


def sample(l, noise, temperature, top_k, top_p, min_p):
    """Token and log probability of one row (-1, -inf where nothing is left)."""
    order, e, lv = kept_order(l, temperature, top_k, top_p, min_p)
    if not len(order):
        return -1, -np.inf
    key = e[order] / np.maximum(noise.astype(np.float64)[order], np.finfo(np.float32).tiny)
    token = int(order[0]) if not temperature > 0 else int(min(order[key == key.max()]))
    t = temperature if temperature > 0 else 1.0
    return token, (lv[token] - lv.max()) / t - np.log(e.sum())
