"""The operators around the recurrence against plain float64 forms.

Outputs lie between guard bands and are filled with NaN first, so that a
value left out or written past an end shows.  Bounds come with the reference
values (tests/layer_reference.py).
"""
from __future__ import annotations

import numpy as np
import pytest

import layer_reference as ref
from gdn_testutil import guarded_full, half_ulp, to_host_f64, torch_dtype

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import linear_attention_recurrence_step_gb300 as gdn  # noqa: E402

NAN = float("nan")


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gdn.load()
    return torch.device("cuda:0")


def put(a, dtype, dev):
    """numpy f64 -> device tensor of the type, and the f64 values it holds."""
    t = torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(torch_dtype(dtype))
    return t.to(dev), t.double().numpy()


def hold(got, want, bound, dtype, what, where=None):
    """got is within bound (plus half a unit of a 16-bit store) of want; where
    it is not to be written it is still NaN."""
    got = to_host_f64(got)
    bound = bound + (half_ulp(np.maximum(np.abs(want), np.abs(np.nan_to_num(got))), dtype) if dtype != "f32" else 0)
    ok = np.abs(got - want) <= bound
    if where is not None:
        shape = where.shape + (1,) * (got.ndim - where.ndim)
        ok = np.where(where.reshape(shape), ok, np.isnan(got))
    if not ok.all():
        i = tuple(np.argwhere(~ok)[0])
        raise AssertionError(f"{what}: {int((~ok).sum())} of {ok.size} off; first at {i}: got {got[i]!r}, "
                             f"want {want[i]!r}, bound {np.broadcast_to(bound, got.shape)[i]!r}")


# ------------------------------------------------------------- convolution
CONV = [  # B, T, C, W, dtype, bias, state, lengths, pad, offset, act
    (1, 1, 64, 4, "bf16", False, True, None, 0, 0, "silu"),
    (3, 1, 1, 2, "f32", True, True, None, 0, 0, "silu"),
    (2, 5, 130, 4, "bf16", True, True, "ragged", 0, 0, "silu"),
    (2, 2, 24, 8, "f16", True, True, "ragged", 0, 0, "silu"),
    (4, 16, 136, 3, "f32", False, False, "ragged", 0, 0, None),
    (1, 700, 256, 4, "bf16", True, False, None, 64, 0, "silu"),
    (2, 333, 99, 5, "f16", False, True, "ragged", 3, 1, "silu"),
    (2, 40, 128, 4, "f32", True, True, "ragged", 5, 0, "silu"),
    (1, 129, 64, 6, "bf16", True, True, None, 8, 8, None),
    (5, 33, 72, 7, "bf16", False, True, "ragged", 0, 4, "silu"),
    (130, 1, 520, 4, "f16", True, True, "ragged", 0, 0, "silu"),
]


@pytest.mark.parametrize("B,T,C,W,dtype,bias,state,lengths,pad,off,act", CONV)
def test_conv(dev, B, T, C, W, dtype, bias, state, lengths, pad, off, act):
    rng = np.random.default_rng(B * 1000 + T)
    wide, wide64 = put(rng.standard_normal((B, T, C + pad + off)), dtype, dev)
    x, x64 = wide[..., off:off + C], wide64[..., off:off + C]
    w, w64 = put(rng.standard_normal((C, W)), dtype, dev)
    bt, b64 = put(rng.standard_normal(C), dtype, dev) if bias else (None, None)
    st, s64 = put(rng.standard_normal((B, W - 1, C)), dtype, dev) if state else (None, None)
    n = None
    if lengths:
        n = rng.integers(0, T + 1, B)
        n[0], n[-1] = T + 3, -2          # clamped
        n = n.astype(np.int32)
    nt = None if n is None else torch.from_numpy(n).to(dev)
    want, bound, s_want, on = ref.conv(x64, w64, b64, s64, n, act is not None)
    y = guarded_full((B, T, C), NAN, x.dtype, dev)
    so = guarded_full((B, W - 1, C), NAN, x.dtype, dev)
    out = gdn.gdn_causal_conv(x, w, st, bias=bt, lengths=nt, activation=act, y=y, state_out=so)
    hold(out.y, want, bound, dtype, "y", on)
    assert np.array_equal(to_host_f64(out.state_out), s_want), "state"
    # the state alone, in place
    if st is not None:
        alone = gdn.gdn_causal_conv(x, w, st, bias=bt, lengths=nt, activation=act, state_out=st, write_y=False)
        assert alone.y is None and torch.equal(alone.state_out, so)


def test_conv_pieces_join(dev):
    """A prompt in one call, in pieces that hand the state on (in place), and
    token by token: the same bits."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(2, 77, 192, generator=gen, device=dev).bfloat16()
    w = torch.randn(192, 4, generator=gen, device=dev).bfloat16()
    whole = gdn.gdn_causal_conv(x, w)
    for cuts in ([0, 40, 41, 77], list(range(78))):
        state = torch.zeros(2, 3, 192, device=dev, dtype=torch.bfloat16)
        ys = [gdn.gdn_causal_conv(x[:, a:b], w, state, state_out=state).y for a, b in zip(cuts, cuts[1:])]
        assert torch.equal(torch.cat(ys, 1), whole.y) and torch.equal(state, whole.state_out)


# -------------------------------------------------------------------- scan
SCAN = [  # B, T, H, P, G, N, dtype, state, lengths, pad, D, bias, softplus
    (1, 1, 1, 1, 1, 16, "f32", True, None, 0, True, True, True),
    (3, 1, 4, 64, 2, 128, "bf16", True, None, 0, True, True, True),
    (2, 1, 2, 128, 1, 128, "f16", False, None, 5, False, False, False),
    (4, 8, 6, 48, 3, 64, "f32", True, "ragged", 0, True, True, True),
    (2, 17, 4, 80, 4, 256, "bf16", True, "ragged", 3, True, True, True),
    (2, 16, 3, 7, 1, 32, "f16", True, "ragged", 0, False, True, True),
    (1, 200, 2, 64, 1, 128, "bf16", True, None, 0, True, True, True),
    (2, 300, 2, 33, 2, 16, "f32", False, "ragged", 0, True, True, True),
    (1, 515, 4, 64, 2, 64, "f16", True, None, 8, True, False, True),
    (2, 129, 4, 128, 2, 128, "bf16", True, "ragged", 0, True, True, True),
    (1, 64, 2, 32, 1, 128, "bf16", False, None, 0, False, True, True),
    (1, 190, 3, 96, 3, 64, "bf16", True, None, 7, True, True, True),
]


def scan_inputs(rng, B, T, H, P, G, N, dtype, dev, state, pad, D, bias):
    wide, wide64 = put(rng.standard_normal((B, T, H * P + 2 * G * N + pad)), dtype, dev)
    cut = [0, H * P, H * P + G * N, H * P + 2 * G * N]
    parts, parts64 = zip(*((wide[..., a:b], wide64[..., a:b]) for a, b in zip(cut, cut[1:])))
    shape = [(H, P), (G, N), (G, N)]
    x, Bm, Cm = (p.unflatten(-1, s) for p, s in zip(parts, shape))
    x64, B64, C64 = (p.reshape(B, T, *s) for p, s in zip(parts64, shape))
    dt, dt64 = put(rng.standard_normal((B, T, H)) * 0.5 + (0 if bias else 0.5), dtype, dev)
    A, A64 = put(-np.exp(rng.uniform(0, 2.5, H)), "f32", dev)
    Dt, D64 = put(rng.standard_normal(H), "f32", dev) if D else (None, None)
    bt, b64 = put(rng.uniform(-5, -1, H), "f32", dev) if bias else (None, None)
    st, s64 = put(rng.standard_normal((B, H, P, N)), "f32", dev) if state else (None, None)
    return (x, dt, A, Bm, Cm, st, Dt, bt), (x64, dt64, A64, B64, C64, D64, b64, s64)


@pytest.mark.parametrize("B,T,H,P,G,N,dtype,state,lengths,pad,D,bias,softplus", SCAN)
def test_scan(dev, B, T, H, P, G, N, dtype, state, lengths, pad, D, bias, softplus):
    rng = np.random.default_rng(T * 100 + H)
    (x, dt, A, Bm, Cm, st, Dt, bt), (x64, dt64, A64, B64, C64, D64, b64, s64) = scan_inputs(
        rng, B, T, H, P, G, N, dtype, dev, state, pad, D, bias)
    if not softplus:
        dt, dt64 = put(np.abs(dt64), dtype, dev)
    n = None
    if lengths:
        n = rng.integers(0, T + 1, B)
        n[0], n[-1] = T + 9, (-1 if B > 2 else T // 2)
        n = n.astype(np.int32)
    nt = None if n is None else torch.from_numpy(n).to(dev)
    want, bound, s_want, s_bound, on = ref.scan(x64, dt64, A64, B64, C64, D64, b64, s64, n, softplus)
    y = guarded_full((B, T, H, P), NAN, x.dtype, dev)
    so = guarded_full((B, H, P, N), NAN, torch.float32, dev)
    kw = dict(D=Dt, dt_bias=bt, softplus=softplus, lengths=nt)
    out = gdn.gdn_selective_scan(x, dt, A, Bm, Cm, st, y=y, state_out=so, **kw)
    hold(out.state_out, s_want, s_bound, "f32", "state")
    hold(out.y, want, bound, dtype, "y", on)
    again = gdn.gdn_selective_scan(x, dt, A, Bm, Cm, st, **kw)
    assert torch.equal(again.state_out, so), "run to run"
    if st is not None:  # the state alone, in place; then with y, in place
        keep = st.clone()
        alone = gdn.gdn_selective_scan(x, dt, A, Bm, Cm, st, state_out=st, write_y=False, **kw)
        hold(alone.state_out, s_want, s_bound, "f32", "state alone, in place")
        st.copy_(keep)
        y2 = guarded_full((B, T, H, P), NAN, x.dtype, dev)
        gdn.gdn_selective_scan(x, dt, A, Bm, Cm, st, y=y2, state_out=st, **kw)
        assert torch.equal(st, so) and torch.equal(y2.nan_to_num(7), y.nan_to_num(7)), "in place"


# the tensor-core form (bf16, N of 64 or 128, whole 16-byte rows): chunks of 32,
# one segment and several, rows of every warp count, two blocks of rows
CHUNKED = [  # B, T, H, P, G, N, lengths, D, bias
    (1, 32, 1, 8, 1, 64, None, True, True),
    (2, 33, 2, 16, 1, 128, "ragged", False, True),
    (1, 1000, 2, 64, 1, 64, None, True, True),
    (3, 700, 2, 72, 2, 128, "ragged", True, True),
    (1, 2080, 1, 128, 1, 128, None, True, False),
    (2, 130, 3, 200, 1, 64, "ragged", True, True),
    (40, 40, 8, 64, 4, 128, "ragged", True, True),
]


@pytest.mark.parametrize("B,T,H,P,G,N,lengths,D,bias", CHUNKED)
def test_scan_chunked(dev, B, T, H, P, G, N, lengths, D, bias):
    test_scan(dev, B, T, H, P, G, N, "bf16", True, lengths, 0, D, bias, True)


def test_scan_forms_agree(dev):
    """The same call on rows that are whole 16-byte pieces (the tensor-core
    form) and on rows that are not (the step form)."""
    rng = np.random.default_rng(12)
    (x, dt, A, Bm, Cm, st, Dt, bt), _ = scan_inputs(rng, 2, 300, 4, 64, 2, 128, "bf16", dev, True, 0, True, True)
    (xs, _, _, Bs, Cs, _, _, _), _ = scan_inputs(rng, 2, 300, 4, 64, 2, 128, "bf16", dev, True, 1, True, True)
    for a, b in ((xs, x), (Bs, Bm), (Cs, Cm)):
        a.copy_(b)
    lens = torch.tensor([300, 171], dtype=torch.int32, device=dev)
    a = gdn.gdn_selective_scan(x, dt, A, Bm, Cm, st, D=Dt, dt_bias=bt, lengths=lens)
    b = gdn.gdn_selective_scan(xs, dt, A, Bs, Cs, st, D=Dt, dt_bias=bt, lengths=lens)
    assert float((a.state_out - b.state_out).abs().max()) < 1e-5 * float(b.state_out.abs().max())
    on = torch.arange(300, device=dev) < lens[:, None]
    assert float((a.y.float() - b.y.float())[on].abs().max()) < 2.0 ** -7 * float(b.y.float()[on].abs().max())


def test_scan_rolls_back(dev):
    """Draft steps, then the accepted prefix again from the snapshot: the state
    that a call over just those steps gives."""
    rng = np.random.default_rng(5)
    (x, dt, A, Bm, Cm, st, Dt, bt), _ = scan_inputs(rng, 3, 8, 4, 64, 2, 128, "bf16", dev, True, 0, True, True)
    acc = torch.tensor([0, 3, 8], dtype=torch.int32, device=dev)
    back = gdn.gdn_selective_scan(x, dt, A, Bm, Cm, st, D=Dt, dt_bias=bt, lengths=acc, write_y=False).state_out
    assert torch.equal(back[0], st[0])
    for b, n in ((1, 3), (2, 8)):
        one = gdn.gdn_selective_scan(x[b:b + 1, :n], dt[b:b + 1, :n], A, Bm[b:b + 1, :n], Cm[b:b + 1, :n],
                                     st[b:b + 1], D=Dt, dt_bias=bt)
        assert torch.equal(back[b], one.state_out[0])


def test_scan_extreme_decay(dev):
    """Steps that wipe the state (the decay underflows to zero) and steps of
    length zero (it stays) leave no NaN, on short and long calls."""
    for T in (4, 300):
        x = torch.ones(1, T, 2, 64, device=dev, dtype=torch.bfloat16)
        dt = torch.zeros(1, T, 2, device=dev, dtype=torch.bfloat16)
        dt[0, T // 2, 0] = 200
        Bm = torch.ones(1, T, 1, 64, device=dev, dtype=torch.bfloat16)
        A = torch.tensor([-1.0, -1.0], device=dev)
        st = torch.full((1, 2, 64, 64), 3.0, device=dev)
        out = gdn.gdn_selective_scan(x, dt, A, Bm, Bm, st, softplus=False)
        assert torch.equal(out.state_out[0, 0], torch.full((64, 64), 200.0, device=dev))
        assert torch.equal(out.state_out[0, 1], st[0, 1])
        assert torch.isfinite(out.y).all()


# -------------------------------------------------------------------- norm
NORM = [  # lead shape, D, dtype, gate, residual, weight per head, pad
    ((1, 1), 1, "f32", "none", False, False, 0),
    ((3, 32), 128, "bf16", "after", False, False, 0),
    ((7, 4), 128, "bf16", "after", True, True, 64),
    ((2, 3, 2), 96, "f16", "first", True, True, 3),
    ((5, 1), 5001, "f32", "none", True, False, 0),
    ((4, 1), 4096, "bf16", "first", False, False, 0),
    ((3, 2), 999, "bf16", "after", True, False, 1),
    ((2, 1), 16384, "f16", "after", True, False, 0),
    ((2, 1), 20001, "bf16", "first", True, False, 0),
    ((1, 1), 40000, "f32", "after", True, False, 0),
    ((300, 8), 64, "f32", "after", False, True, 0),
    ((2, 2), 2056, "bf16", "none", True, False, 0),
    ((11, 1), 24, "bf16", "after", False, False, 0),
    # enough rows for several per thread
    ((5000, 8), 128, "bf16", "after", False, False, 0),
    ((5001, 8), 120, "f16", "first", True, True, 8),
    ((1250, 32), 256, "bf16", "after", True, False, 0),
    ((40000, 1), 64, "f32", "after", False, False, 0),
    ((9750, 4), 512, "bf16", "none", False, True, 0),
    # wide rows, whole and cut across 16-byte boundaries
    ((3, 1), 5120, "f32", "none", True, False, 0),
    ((5, 1), 10237, "f16", "after", True, False, 0),
    ((4, 1), 1031, "f32", "first", True, False, 0),
    ((6, 1), 77, "bf16", "after", True, False, 0),
    ((2, 3), 16001, "bf16", "after", True, True, 0),
]


@pytest.mark.parametrize("lead,D,dtype,gate,residual,per_head,pad", NORM)
def test_norm(dev, lead, D, dtype, gate, residual, per_head, pad):
    rng = np.random.default_rng(D)
    K = lead[-1]
    wide, wide64 = put(rng.standard_normal((*lead[:-1], K * D + pad)) * 2, dtype, dev)
    x, x64 = wide[..., :K * D].unflatten(-1, (K, D)), wide64[..., :K * D].reshape(*lead, D)
    w, w64 = put(1 + 0.3 * rng.standard_normal((K, D) if per_head else D), dtype, dev)
    g, g64 = put(3 * rng.standard_normal((*lead, D)), dtype, dev) if gate != "none" else (None, None)
    r, r64 = put(rng.standard_normal((*lead, D)), dtype, dev) if residual else (None, None)
    scale = float(np.float32(0.37))
    want, bound, r_want, r_bound = ref.norm(x64, w64, g64, gate == "first", r64, scale, 1e-6)
    y = guarded_full((*lead, D), NAN, x.dtype, dev)
    ro = guarded_full((*lead, D), NAN, x.dtype, dev) if residual else None
    kw = dict(gate=g, gate_first=gate == "first", residual_scale=scale, eps=1e-6)
    out = gdn.gdn_gated_norm(x, w, residual=r, y=y, residual_out=ro, **kw)
    hold(out.y, want, bound, dtype, "y")
    if residual:
        hold(out.residual_out, r_want, r_bound, dtype, "residual")
        # in place: the residual into its own buffer, y into a dense x
        xd = x.contiguous()
        gdn.gdn_gated_norm(xd, w, residual=r, y=xd, residual_out=r, **kw)
        assert torch.equal(r, ro) and torch.equal(xd, y)


def test_norm_extremes(dev):
    """A row of zeros, large values that overflow no sum of squares in f32, and
    gates at both ends."""
    x = torch.zeros(4, 128, device=dev)
    x[1] = 1e18
    x[2] = 1e-18
    x[3] = 2.0
    g = torch.zeros(4, 128, device=dev)
    g[3, 0], g[3, 1] = 1e4, -1e4
    y = gdn.gdn_gated_norm(x, torch.ones(128, device=dev), gate=g, eps=1e-6).y
    assert torch.equal(y[:3], torch.zeros(3, 128, device=dev))
    assert abs(float(y[3, 0]) - 1e4) < 1 and float(y[3, 1]) == 0
    y = gdn.gdn_gated_norm(x, torch.ones(128, device=dev)).y
    assert float(y[0].abs().max()) == 0 and abs(float(y[1, 5]) - 1) < 1e-5


# ------------------------------------------------------------------ sample
SAMPLE = [  # R, V, dtype, pad, settings
    (1, 1, "f32", 0, dict()),
    (3, 7, "bf16", 0, dict(top_k=3)),
    (5, 1000, "f32", 3, dict(temperature=0.7, top_k=50)),
    (4, 1003, "bf16", 1, dict(temperature=1.3, top_p=0.9)),
    (4, 50000, "f16", 0, dict(min_p=0.02, temperature=0.9)),
    (2, 131072, "bf16", 0, dict(top_k=40, top_p=0.8, min_p=0.01)),
    (2, 100003, "f32", 0, dict(top_p=0.99, temperature=1.5)),
    (3, 32000, "bf16", 0, dict(top_k=20000, top_p=0.5)),
    (2, 32000, "f32", 8, dict()),
    (200, 4100, "bf16", 0, dict(top_k=10, top_p=0.95, temperature=2.0)),
    (170, 32001, "f16", 0, dict(top_p=0.7)),
    (4, 5000, "f32", 0, dict(temperature=0.0)),
    (1, 1000000, "f32", 0, dict(top_k=100, top_p=0.9)),
    (1, 2000001, "bf16", 0, dict(top_p=0.9)),
    (2, 800000, "f32", 0, dict(temperature=0.8)),
]


def sample_rows(l64, noise, settings, R):
    one = dict(temperature=1.0, top_k=0, top_p=1.0, min_p=0.0) | settings
    rows = [ref.sample(l64[r], noise[r], **{k: (v[r] if np.ndim(v) else v) for k, v in one.items()}) for r in range(R)]
    return np.array([t for t, _ in rows]), np.array([p for _, p in rows])


def hold_sample(out, l64, noise, settings, R):
    token, logprob = sample_rows(l64, noise, settings, R)
    assert np.array_equal(out.token.cpu().numpy().reshape(-1), token)
    got = out.logprob.double().cpu().numpy().reshape(-1)
    fine = np.isfinite(logprob)
    assert np.array_equal(np.isfinite(got), fine)
    # (l - max)/T to two units; the mass to the units of its largest exponents
    # (|d| below 100 or the term is nothing) in sums of a few hundred terms
    assert (np.abs(got - logprob)[fine] <= 2e-5 + 4 * ref.U * np.abs(logprob[fine])).all()


@pytest.mark.parametrize("R,V,dtype,pad,settings", SAMPLE)
def test_sample(dev, R, V, dtype, pad, settings):
    rng = np.random.default_rng(V + R)
    wide, wide64 = put(2.5 * rng.standard_normal((R, V + pad)), dtype, dev)
    l, l64 = wide[:, :V], wide64[:, :V]
    noise = rng.standard_exponential((R, V)).astype(np.float32)
    out = gdn.gdn_sample(l, torch.from_numpy(noise).to(dev), token=guarded_full((R,), -7, torch.int32, dev),
                         logprob=guarded_full((R,), NAN, torch.float32, dev), **settings)
    hold_sample(out, l64, noise, settings, R)


def test_sample_row_settings(dev):
    """Every row with settings of its own, [B,T,V] logits, odd row strides."""
    rng = np.random.default_rng(8)
    B, T, V = 6, 5, 9001
    R = B * T
    wide, wide64 = put(2 * rng.standard_normal((B, T, V + 2)), "bf16", dev)
    noise = rng.standard_exponential((B, T, V)).astype(np.float32)
    s = dict(temperature=rng.uniform(0.3, 2, R).astype(np.float32), top_k=rng.integers(0, 60, R).astype(np.int32),
             top_p=rng.uniform(0.3, 1.2, R).astype(np.float32), min_p=rng.uniform(-0.1, 0.2, R).astype(np.float32))
    s["temperature"][::7] = 0
    s["top_k"][1::7] = V + 5
    s["top_p"][2::7] = 0
    s["min_p"][3::7] = 1.5
    out = gdn.gdn_sample(wide[..., :V], torch.from_numpy(noise).to(dev),
                         **{k: torch.from_numpy(v).to(dev).reshape(B, T) for k, v in s.items()})
    assert out.token.shape == (B, T)
    hold_sample(out, wide64[..., :V].reshape(R, V), noise.reshape(R, V), s, R)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("V,levels", [(37, 3), (3000, 5), (40000, 40), (140000, 2), (140001, 1)])
def test_sample_cut_is_exact(dev, dtype, V, levels):
    """Logits of few values, so that every cut goes through a group of equal
    ones.  The noise lets the last token that stays win, unless one that the
    cut removes were left: that one would beat it."""
    rng = np.random.default_rng(levels)
    vals = rng.choice(np.linspace(-1.5, 2, levels + 1)[:levels], V)
    l, l64 = put(np.stack([vals] * 6), dtype, dev)
    settings = dict(temperature=np.full(6, 0.9, np.float32),
                    top_k=np.array([1, 5, V // 2, 0, 30, V - 1], np.int32),
                    top_p=np.array([1, 1, 0.75, 0.6, 0.5, 1], np.float32),
                    min_p=np.array([0, 0, 0, 0, 0, 0.3], np.float32))
    noise = np.ones((6, V), np.float32)
    for r in range(6):
        order, _, _ = ref.kept_order(l64[r], *(settings[k][r] for k in ("temperature", "top_k", "top_p", "min_p")))
        full = np.argsort(-l64[r], kind="stable")
        noise[r, order[-1]] = 1e-10
        noise[r, full[len(order):]] = 1e-25
    out = gdn.gdn_sample(l, torch.from_numpy(noise).to(dev),
                         **{k: torch.from_numpy(v).to(dev) for k, v in settings.items()})
    hold_sample(out, l64, noise, settings, 6)


@pytest.mark.parametrize("seed", range(12))
def test_sample_sweep(dev, seed):
    """Rows of every shape of distribution, each with settings of its own: large
    top-k with top-p, nuclei of a handful and of most tokens, lists that do not
    fit, one CTA and clusters."""
    rng = np.random.default_rng(700 + seed)
    V = int(rng.choice([257, 4096, 9001, 33000, 70001, 131072]))
    R = int(rng.integers(2, 9))
    dtype = ["bf16", "f32", "f16"][seed % 3]
    sigma = rng.choice([0.05, 0.7, 1.5, 4.0, 12.0], R)
    logits = sigma[:, None] * rng.standard_normal((R, V)) + rng.choice([0.0, 30.0, -200.0], R)[:, None]
    logits[:, rng.integers(0, V, 5)] += sigma[:, None] * rng.uniform(0, 6, 5)
    logits[rng.random((R, V)) < 0.05] = -np.inf
    l, l64 = put(logits, dtype, dev)
    noise = rng.standard_exponential((R, V)).astype(np.float32)
    s = dict(temperature=rng.uniform(0.3, 2, R).astype(np.float32),
             top_k=rng.choice([0, 0, 5, 256, 257, V // 3, V], R).astype(np.int32),
             top_p=rng.choice([0.1, 0.5, 0.9, 0.999, 1.0], R).astype(np.float32),
             min_p=rng.choice([0.0, 0.0, 0.001, 0.2], R).astype(np.float32))
    out = gdn.gdn_sample(l, torch.from_numpy(noise).to(dev), **{k: torch.from_numpy(v).to(dev) for k, v in s.items()})
    hold_sample(out, l64, noise, s, R)
    again = gdn.gdn_sample(l, torch.from_numpy(noise).to(dev),
                           **{k: torch.from_numpy(v).to(dev) for k, v in s.items()})
    assert torch.equal(again.token, out.token) and torch.equal(again.logprob, out.logprob)


def test_sample_masks(dev):
    """Rows that a mask empties, rows of the lowest value, infinities, NaN and
    a single token that is left."""
    V = 6007
    rng = np.random.default_rng(2)
    l = rng.standard_normal((9, V)).astype(np.float32)
    l[0] = -np.inf
    l[1] = np.nan
    l[2] = np.finfo(np.float32).min
    l[3] = -np.inf
    l[3, 4321] = -5
    l[4, [7, 900]] = np.inf
    l[5, ::2] = np.nan
    l[6] = np.finfo(np.float32).min
    l[6, 17:40] = 1.0
    l[7, 1:] = -np.inf
    l[8] = 0.0
    l[8, ::2] = -0.0                       # equal to 0: ties go by index
    noise = rng.standard_exponential((9, V)).astype(np.float32)
    noise[4] = 1
    noise[8] = 1
    for settings in (dict(), dict(top_k=5), dict(top_p=0.5), dict(min_p=0.1), dict(top_k=30, top_p=0.9, min_p=0.01),
                     dict(temperature=0.0), dict(temperature=1e-30), dict(temperature=1e30, top_k=2)):
        out = gdn.gdn_sample(torch.from_numpy(l).to(dev), torch.from_numpy(noise).to(dev), **settings)
        hold_sample(out, l.astype(np.float64), noise, settings, 9)


def test_sample_distribution(dev):
    """With exponential noise the tokens come out with the probabilities of the
    tokens that are left: 40000 draws of a row of six, top-p leaves four."""
    p = np.array([0.4, 0.3, 0.15, 0.1, 0.04, 0.01])
    R = 40000
    l = torch.tensor(np.log(p), dtype=torch.float32, device=dev).expand(R, 6).contiguous()
    noise = torch.empty(R, 6, device=dev).exponential_(generator=torch.Generator(device="cuda").manual_seed(4))
    t = gdn.gdn_sample(l, noise, top_p=0.94).token
    share = torch.bincount(t.long(), minlength=6).double().cpu().numpy() / R
    want = np.array([0.4, 0.3, 0.15, 0.1, 0, 0]) / 0.95
    assert np.abs(share - want).max() < 5 * 0.5 / R ** 0.5 and share[4:].sum() == 0


# -------------------------------------------------- streams, far offsets
def test_other_stream_and_graph(dev):
    """The four calls in a row on a stream of their own, and captured in a
    graph that is replayed on new inputs: the same bits as on the default
    stream."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    B, T, H, P, G, N, V = 2, 100, 4, 64, 2, 64, 3001

    def inputs():
        return [torch.randn(B, T, H * P + 2 * G * N, generator=gen, device=dev).bfloat16(),
                torch.randn(B, T, H, generator=gen, device=dev).bfloat16(),
                torch.randn(B, T, H, P, generator=gen, device=dev).bfloat16(),
                torch.randn(B, V, generator=gen, device=dev),
                torch.empty(B, V, device=dev).exponential_(generator=gen)]

    w = torch.randn(H * P + 2 * G * N, 4, generator=gen, device=dev).bfloat16()
    A = -torch.rand(H, device=dev, generator=gen) - 0.5
    nw = torch.ones(P, device=dev, dtype=torch.bfloat16)

    def chain(xbc, dt, z, logits, noise):
        c = gdn.gdn_causal_conv(xbc, w)
        x, Bm, Cm = c.y.split([H * P, G * N, G * N], -1)
        s = gdn.gdn_selective_scan(x.unflatten(-1, (H, P)), dt, A, Bm.unflatten(-1, (G, N)), Cm.unflatten(-1, (G, N)))
        n = gdn.gdn_gated_norm(s.y, nw, gate=z)
        t = gdn.gdn_sample(logits, noise, top_k=20, top_p=0.9)
        return c.y, c.state_out, s.y, s.state_out, n.y, t.token, t.logprob

    sets = [inputs() for _ in range(3)]
    want = [chain(*s) for s in sets]
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        got = [chain(*s) for s in sets]
    st.synchronize()
    for g, w_ in zip(got, want):
        assert all(torch.equal(a, b) for a, b in zip(g, w_))
    live = [t.clone() for t in sets[0]]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = chain(*live)
    for s, w_ in zip(sets, want):
        for a, b in zip(live, s):
            a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, w_))


def test_far_offsets(dev):
    """Rows more than 2^31 elements apart give what the same rows give close
    together."""
    if torch.cuda.get_device_properties(0).total_memory < 40e9:
        pytest.skip("needs a large device memory")
    far = 2 ** 31 + 64
    big = torch.empty(far + 200000, dtype=torch.bfloat16, device=dev)
    gen = torch.Generator(device="cuda").manual_seed(9)

    def apart(t, stride0):
        """t [2,...] (dense rows) laid out with its two halves far apart."""
        v = big.as_strided(t.shape, (stride0,) + t[0].stride())
        v.copy_(t)
        return v

    x = torch.randn(2, 5, 256, generator=gen, device=dev).bfloat16()
    w = torch.randn(256, 4, generator=gen, device=dev).bfloat16()
    a, b = gdn.gdn_causal_conv(x, w), gdn.gdn_causal_conv(apart(x, far), w)
    assert torch.equal(a.y, b.y) and torch.equal(a.state_out, b.state_out)
    sx = torch.randn(2, 70, 2, 64, generator=gen, device=dev).bfloat16()
    bc = torch.randn(2, 70, 1, 64, generator=gen, device=dev).bfloat16()
    dt = torch.rand(2, 70, 2, generator=gen, device=dev).bfloat16()
    A = -torch.ones(2, device=dev)
    a = gdn.gdn_selective_scan(sx, dt, A, bc, bc)
    b = gdn.gdn_selective_scan(apart(sx, far), dt, A, bc, bc)
    assert torch.equal(a.y, b.y) and torch.equal(a.state_out, b.state_out)
    nx = torch.randn(2, 4, 128, generator=gen, device=dev).bfloat16()
    nw = torch.ones(128, device=dev, dtype=torch.bfloat16)
    assert torch.equal(gdn.gdn_gated_norm(nx, nw).y, gdn.gdn_gated_norm(apart(nx, far), nw).y)
    l = torch.randn(2, 100000, generator=gen, device=dev).bfloat16()
    noise = torch.empty(2, 100000, device=dev).exponential_(generator=gen)
    a = gdn.gdn_sample(l, noise, top_p=0.9)
    b = gdn.gdn_sample(apart(l, far), noise, top_p=0.9)
    assert torch.equal(a.token, b.token) and torch.equal(a.logprob, b.logprob)
