"""Refusals of the operators around the recurrence: every argument check of
the four C entry points and of their bindings returns before anything reaches
a device (the addresses below are fake)."""
from __future__ import annotations

import ctypes

import pytest

import linear_attention_recurrence_step_gb300 as gdn

torch = pytest.importorskip("torch")

OK, INVALID, UNSUPPORTED, MISALIGNED, CUDA = 0, 1, 2, 3, 4
F32, BF16, F16 = 0, 1, 2


def P(i: int) -> int:
    return 0x1000000 * (i + 1)


@pytest.fixture(scope="module")
def lib():
    gdn.build()
    return gdn.load()


def conv(lib, **kw):
    a = dict(x=P(0), weight=P(1), bias=P(2), state_in=P(3), lengths=P(4), y=P(5), state_out=P(6), B=2, T=3, C=64, W=4,
             sb=192, st=64, act=1, dtype=BF16) | kw
    return lib.gdn_causal_conv(*(a[k] for k in ("x", "weight", "bias", "state_in", "lengths", "y", "state_out", "B",
                                                "T", "C", "W", "sb", "st", "act", "dtype")), None)


def scan(lib, **kw):
    a = dict(x=P(0), dt=P(1), A=P(2), Bm=P(3), Cm=P(4), D=P(5), bias=P(6), state_in=P(7), lengths=P(8), y=P(9),
             state_out=P(10), B=2, T=3, H=4, P=64, G=2, N=128, strides=None, softplus=1, ws=None, ws_bytes=0,
             dtype=BF16) | kw
    st = a["strides"]
    if st is not None:
        st = ctypes.byref((ctypes.c_int64 * 8)(*st))
    return lib.gdn_selective_scan(*(a[k] for k in ("x", "dt", "A", "Bm", "Cm", "D", "bias", "state_in", "lengths", "y",
                                                   "state_out", "B", "T", "H", "P", "G", "N")), st, a["softplus"],
                                  a["ws"], a["ws_bytes"], a["dtype"], None)


def norm(lib, **kw):
    a = dict(x=P(0), weight=P(1), gate=P(2), residual=P(3), y=P(4), residual_out=P(5), M=3, K=4, D=128, xs=512, gs=512,
             wr=4, first=0, scale=0.5, eps=1e-6, dtype=BF16) | kw
    return lib.gdn_gated_norm(*(a[k] for k in ("x", "weight", "gate", "residual", "y", "residual_out", "M", "K", "D",
                                               "xs", "gs", "wr", "first", "scale", "eps", "dtype")), None)


def sample(lib, **kw):
    a = dict(logits=P(0), noise=P(1), temperature=P(2), top_k=P(3), top_p=P(4), min_p=P(5), tv=1.0, kv=0, pv=1.0,
             mv=0.0, token=P(6), logprob=P(7), R=4, V=1000, ls=1000, ns=1000, dtype=BF16) | kw
    return lib.gdn_sample(*(a[k] for k in ("logits", "noise", "temperature", "top_k", "top_p", "min_p", "tv", "kv",
                                           "pv", "mv", "token", "logprob", "R", "V", "ls", "ns", "dtype")), None)


CASES = {
    conv: {
        "B=0": (dict(B=0), INVALID), "T=-1": (dict(T=-1), INVALID), "C=0": (dict(C=0), INVALID),
        "W=0": (dict(W=0), INVALID), "W=1": (dict(W=1), UNSUPPORTED), "W=9": (dict(W=9), UNSUPPORTED),
        "dtype": (dict(dtype=5), UNSUPPORTED), "activation": (dict(act=2), INVALID),
        "null x": (dict(x=None), INVALID), "null weight": (dict(weight=None), INVALID),
        "no output": (dict(y=None, state_out=None), INVALID), "step stride": (dict(st=63), INVALID),
        "batch stride": (dict(sb=191), INVALID), "negative stride": (dict(sb=-192), INVALID),
        "overflow": (dict(B=1 << 40, T=1 << 30), INVALID), "stride overflow": (dict(sb=1 << 62, B=8), INVALID),
        "odd x": (dict(x=P(0) + 1), MISALIGNED), "odd lengths": (dict(lengths=P(4) + 2), MISALIGNED),
        "state overlap": (dict(state_out=P(3) + 16), INVALID), "y on x": (dict(y=P(0)), INVALID),
        "y on state": (dict(y=P(6)), INVALID), "state_out on x": (dict(state_out=P(0) + 64), INVALID),
    },
    scan: {
        "B=0": (dict(B=0), INVALID), "P=0": (dict(P=0), INVALID), "H%G": (dict(G=3), INVALID),
        "N=48": (dict(N=48), UNSUPPORTED), "N=512": (dict(N=512), UNSUPPORTED), "dtype": (dict(dtype=-1), UNSUPPORTED),
        "null A": (dict(A=None), INVALID), "null C": (dict(Cm=None), INVALID),
        "no output": (dict(y=None, state_out=None), INVALID),
        "x step stride": (dict(strides=(768, 255, 12, 4, 768, 256, 768, 256)), INVALID),
        "C batch stride": (dict(strides=(768, 256, 12, 4, 768, 256, 700, 256)), INVALID),
        "overflow": (dict(B=1 << 40, T=1 << 30), INVALID),
        "state misaligned": (dict(state_in=P(7) + 8), MISALIGNED), "odd x": (dict(x=P(0) + 1), MISALIGNED),
        "A misaligned": (dict(A=P(2) + 2), MISALIGNED), "state overlap": (dict(state_out=P(7) + 32), INVALID),
        "y on x": (dict(y=P(0)), INVALID), "state_out on y": (dict(state_out=P(9)), INVALID),
        "no workspace": (dict(T=4096, B=1), INVALID),
        "small workspace": (dict(T=4096, B=1, ws=P(20), ws_bytes=64), INVALID),
        "workspace misaligned": (dict(T=4096, B=1, ws=P(20) + 4, ws_bytes=1 << 30), MISALIGNED),
    },
    norm: {
        "M=0": (dict(M=0), INVALID), "D=0": (dict(D=0), INVALID), "weight rows": (dict(wr=2), INVALID),
        "eps<0": (dict(eps=-1e-6), INVALID), "eps nan": (dict(eps=float("nan")), INVALID),
        "dtype": (dict(dtype=3), UNSUPPORTED), "null y": (dict(y=None), INVALID), "null x": (dict(x=None), INVALID),
        "residual alone": (dict(residual_out=None), INVALID), "residual_out alone": (dict(residual=None), INVALID),
        "x stride": (dict(xs=511), INVALID), "gate stride": (dict(gs=100), INVALID),
        "overflow": (dict(M=1 << 50, D=1 << 20, xs=1 << 22, gs=1 << 22), INVALID),
        "odd y": (dict(y=P(4) + 1), MISALIGNED), "y partly on x": (dict(y=P(0) + 256), INVALID),
        "y on a strided x": (dict(y=P(0), xs=600), INVALID), "y on residual_out": (dict(y=P(5)), INVALID),
        "y on weight": (dict(y=P(1)), INVALID),
    },
    sample: {
        "R=0": (dict(R=0), INVALID), "V=0": (dict(V=0), INVALID), "V too large": (dict(V=(1 << 22) + 1), UNSUPPORTED),
        "dtype": (dict(dtype=7), UNSUPPORTED), "null noise": (dict(noise=None), INVALID),
        "null token": (dict(token=None), INVALID), "row stride": (dict(ls=999), INVALID),
        "noise stride": (dict(ns=10), INVALID), "stride overflow": (dict(ls=1 << 62), INVALID),
        "odd logits": (dict(logits=P(0) + 1), MISALIGNED), "odd noise": (dict(noise=P(1) + 2), MISALIGNED),
        "token on noise": (dict(token=P(1)), INVALID), "token on logprob": (dict(token=P(7)), INVALID),
        "token on top_k": (dict(token=P(3)), INVALID),
    },
}


@pytest.mark.parametrize("call,name", [(c, n) for c in CASES for n in sorted(CASES[c])],
                         ids=lambda v: v if isinstance(v, str) else v.__name__)
def test_rejects(lib, call, name):
    kw, want = CASES[call][name]
    assert call(lib, **kw) == want
    fn = {conv: "gdn_causal_conv", scan: "gdn_selective_scan", norm: "gdn_gated_norm", sample: "gdn_sample"}[call]
    assert lib.gdn_last_error().decode().startswith(fn)


@pytest.mark.parametrize("call", list(CASES), ids=lambda v: v.__name__)
def test_forced_failure_stops_before_the_device(lib, call):
    try:
        assert lib.gdn_force_launch_failures(1) == OK
        assert call(lib) == CUDA
        assert "forced by gdn_force_launch_failures" in lib.gdn_last_error().decode()
    finally:
        assert lib.gdn_force_launch_failures(0) == OK


def test_norm_takes_its_inputs_buffers(lib):
    """y and residual_out may be the dense buffers of x, gate or residual."""
    ways = [dict(y=P(0)), dict(y=P(2)), dict(residual_out=P(3)), dict(y=P(0), residual_out=P(3)),
            dict(y=P(3), residual_out=P(0))]
    try:
        assert lib.gdn_force_launch_failures(len(ways)) == OK
        for kw in ways:
            assert norm(lib, **kw) == CUDA          # accepted: it got as far as the launch
    finally:
        assert lib.gdn_force_launch_failures(0) == OK


def test_scan_workspace_size(lib):
    assert gdn.gdn_selective_scan_workspace_size(1, 1, 32, 128, 128) == 16          # no segments
    assert gdn.gdn_selective_scan_workspace_size(1, 4096, 32, 128, 128) > 32 * 128 * 128 * 4
    assert gdn.gdn_selective_scan_workspace_size(1, 4096, 32, 128, 100) == 0
    assert gdn.gdn_selective_scan_workspace_size(0, 4096, 32, 128, 128) == 0


def test_bindings_refuse(lib):
    cpu = torch.zeros(1, 2, 64)
    with pytest.raises(ValueError, match="CUDA"):
        gdn.gdn_causal_conv(cpu, torch.zeros(64, 4))
    with pytest.raises(TypeError):
        gdn.gdn_causal_conv([1.0], torch.zeros(64, 4))
    with pytest.raises(ValueError, match="dtype"):
        gdn.gdn_sample(torch.zeros(2, 8, dtype=torch.float64), torch.zeros(2, 8))
    with pytest.raises(ValueError, match="CUDA"):
        gdn.gdn_gated_norm(cpu, torch.zeros(64))
    with pytest.raises(ValueError, match="CUDA"):
        gdn.gdn_selective_scan(torch.zeros(1, 2, 4, 8), cpu, cpu, cpu, cpu)
