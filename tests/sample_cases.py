"""Rows of logits on which a nucleus (top-p) ends at the last of the top-k
tokens while tokens outside share that token's logit, with noise that lets
any token that should not be left win over all others."""
from __future__ import annotations

import numpy as np

import layer_reference as ref

# name -> (V, top_k, top_p, how the logits lie)
TIED_CUTS = {
    "one of a group inside": (6007, 300, 0.999, ("group", 299, 1)),
    "several of a group inside": (6007, 300, 0.999, ("group", 290, 10)),
    "a whole group inside": (6007, 300, 0.999, ("group", 250, 50)),
    "just above the short form": (6007, 257, 0.999, ("group", 240, 17)),
    "small k, its list overflows": (6007, 50, 0.99, ("group", 49, 1)),
    "small k, lists that fit": (6007, 50, 0.99, ("few", 49, 1)),
    "k of 230 over long rows": (33001, 230, 0.999, ("group", 229, 1)),
    "rounded normal, one inside": (32000, 300, 0.9999, ("rounded", 0.25, 1)),
    "rounded normal, three inside": (32000, 313, 0.9999, ("rounded", 0.25, 3)),
    "rounded normal, k of a thousand": (8003, 1000, 0.9999, ("rounded", 0.03125, 1)),
    "a third of the row": (9001, 3000, 0.9999, ("rounded", 0.03125, 1)),
    "a third of a flat row": (3001, 1000, 0.9999, ("group", 0, 1000)),
}


def tied_cut(name, seed=0):
    """(logits [V] f64, exact in every type; settings; noise [V] f32)."""
    V, k, p, how = TIED_CUTS[name]
    rng = np.random.default_rng(seed * 1000 + V + k)
    if how[0] == "rounded":
        # k goes to the next group from `k` on, of which so many are inside
        l = np.round(rng.standard_normal(V) / how[1]) * how[1]
        ordered = np.sort(l)[::-1]
        k = int(np.flatnonzero(ordered < ordered[k])[0]) + how[2]
    else:
        above, inside = how[1:]
        assert above + inside == k
        l = np.full(V, 0.5)
        if how[0] == "few":  # forty share the k-th logit, the others lie below
            l[40 + above:] = -3.0
        l[:above] = 1.0
        l = l[rng.permutation(V)]
    s = dict(temperature=0.9, top_k=k, top_p=p, min_p=0.0)
    order, e, _ = ref.kept_order(l, 0.9, k, p, 0.0)
    full = np.argsort(-l, kind="stable")
    # the row is what it says: the nucleus ends at the k-th token by a margin
    # well above float32's, and the next token has the same logit
    es = e[full[:k]]
    share = (es.sum() - es[-1]) / es.sum()
    assert len(order) == k and share < p * (1 - 2e-6) and (l[full[k]] == l[full[k - 1]] or "whole" in name)
    noise = np.ones(V, np.float32)
    noise[order[-1]] = 1e-10
    noise[full[k:]] = 1e-25
    return l, s, noise


def bracket_edge(seed):
    """(logits [V] f64 of float32 values, top_p near which a nucleus ends where
    the kernel's bracket for it begins).  The kernel counts tokens in 4096 bins
    over the range that can matter and bounds the mass above each bin by the
    bins' upper edges; it looks for the nucleus' end from the bin on in which
    that bound passes top_p times the mass (less a ten-thousandth).  Here 1500
    tokens lie just below such edges, so that the bound is tight, then one
    alone in its bin, in which the nucleus ends, then 1500 more; the bound
    passes exactly between the first 1500 and the one."""
    V, rng = 50000, np.random.default_rng(seed)
    bins = np.sort(rng.integers(770, 900, 1500))
    late = np.concatenate([[1000], rng.integers(1002, 1015, 1500)])
    p = 0.7
    for _ in range(100):
        z = 25.0
        for _ in range(300):
            width = -np.log(0.5 * (1 - p) * z / V) / 4096
            d, d_late = (bins - 0.47) * width, (late - 0.45) * width
            z = 1 + np.exp(-d).sum() + np.exp(-d_late).sum()
        p = (np.exp(0.5 * width) + np.exp(-(bins - 0.5) * width).sum()) / (0.9999 * z)
    l = np.full(V, -np.inf)
    l[:3002] = np.concatenate([[0.0], -d, -d_late])
    return np.random.default_rng(seed).permutation(l.astype(np.float32)).astype(np.float64), np.float32(p)
