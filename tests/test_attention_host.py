"""Refusals of the attention layer's operators: every argument check of the C
entry points and of their bindings returns before anything reaches a device
(the addresses below are fake), and the frequencies' helper."""
from __future__ import annotations

import ctypes
import math

import pytest

import linear_attention_recurrence_step_gb300 as gdn

torch = pytest.importorskip("torch")

OK, INVALID, UNSUPPORTED, MISALIGNED, CUDA = 0, 1, 2, 3, 4
F32, BF16, F16 = 0, 1, 2


def P(i: int) -> int:
    return 0x10000000 * (i + 1)


@pytest.fixture(scope="module")
def lib():
    gdn.build()
    return gdn.load()


def slots(lib, **kw):
    names = ("lengths", "add", "held", "ring_state", "table", "ring", "slots", "positions", "granted", "lengths_out",
             "held_out", "ring_state_out")
    a = {n: P(i) for i, n in enumerate(names)} | dict(B=4, T=3, width=8, pages=100, page=16) | kw
    return lib.gdn_page_slots(*(a[n] for n in names), a["B"], a["T"], a["width"], a["pages"], a["page"], None)


def rotary(lib, **kw):
    a = dict(q=P(0), k=P(1), positions=P(2), inv_freq=P(3), q_out=P(4), k_out=P(5), B=2, T=3, Hq=4, Hk=2, D=64, R=32,
             strides=None, layout=0, scale=1.0, inverse=0, dtype=BF16) | kw
    st = a["strides"]
    if st is not None:
        st = ctypes.byref((ctypes.c_int64 * 8)(*st))
    return lib.gdn_rotary(*(a[n] for n in ("q", "k", "positions", "inv_freq", "q_out", "k_out", "B", "T", "Hq", "Hk", "D",
                                           "R")), st, a["layout"], a["scale"], a["inverse"], a["dtype"], None)


def append(lib, **kw):
    a = dict(k=P(0), v=P(1), slots=P(2), cache=P(3), ks=P(4), vs=P(5), B=2, T=3, H=4, D=64, page=16, pages=10, ksb=768,
             kst=256, vsb=768, vst=256, dtype=BF16) | kw
    return lib.gdn_kv_append(*(a[n] for n in ("k", "v", "slots", "cache", "ks", "vs", "B", "T", "H", "D", "page", "pages",
                                              "ksb", "kst", "vsb", "vst", "dtype")), None)


def read(lib, **kw):
    a = dict(cache=P(3), slots=P(2), ks=P(4), vs=P(5), k=P(0), v=P(1), N=6, H=4, D=64, page=16, pages=10, dtype=BF16) | kw
    return lib.gdn_kv_read(*(a[n] for n in ("cache", "slots", "ks", "vs", "k", "v", "N", "H", "D", "page", "pages",
                                            "dtype")), None)


def attend(lib, **kw):
    a = dict(q=P(0), cache=P(1), table=P(2), lengths=P(3), fresh=P(4), ks=P(5), vs=P(6), y=P(7), lse=P(8), B=2, T=3, Hq=8,
             H=4, D=64, width=5, page=16, pages=10, sb=1536, st=512, scale=0.125, window=0, ws=P(9), ws_bytes=1 << 28,
             dtype=BF16) | kw
    return lib.gdn_kv_attention(*(a[n] for n in ("q", "cache", "table", "lengths", "fresh", "ks", "vs", "y", "lse", "B",
                                                 "T", "Hq", "H", "D", "width", "page", "pages", "sb", "st", "scale",
                                                 "window", "ws", "ws_bytes", "dtype")), None)


CASES = {
    slots: {
        "B=0": (dict(B=0), INVALID), "T=-1": (dict(T=-1), INVALID), "pages=0": (dict(pages=0), INVALID),
        "width=0": (dict(width=0), INVALID), "page=24": (dict(page=24), UNSUPPORTED), "page=0": (dict(page=0), INVALID),
        "page=256": (dict(page=256), UNSUPPORTED), "pool too large": (dict(pages=1 << 27), INVALID),
        "rows too long": (dict(width=1 << 27), INVALID), "overflow": (dict(B=1 << 40, width=1 << 26), INVALID),
        "null lengths": (dict(lengths=None), INVALID), "null ring": (dict(ring=None), INVALID),
        "null granted": (dict(granted=None), INVALID), "odd slots": (dict(slots=P(6) + 2), MISALIGNED),
        "lengths_out near lengths": (dict(lengths_out=P(0) + 4), INVALID),
        "held_out near held": (dict(held_out=P(2) + 8), INVALID), "slots on positions": (dict(positions=P(6)), INVALID),
        "granted on add": (dict(granted=P(1)), INVALID), "ring on table": (dict(ring=P(4) + 64), INVALID),
        "lengths_out on held": (dict(lengths_out=P(2)), INVALID), "state out on lengths": (dict(ring_state_out=P(0)), INVALID),
    },
    rotary: {
        "B=0": (dict(B=0), INVALID), "D=0": (dict(D=0), INVALID), "Hk=0": (dict(Hk=0), INVALID),
        "R odd": (dict(R=31), INVALID), "R > D": (dict(R=66), INVALID), "R=0": (dict(R=0), INVALID),
        "R large": (dict(R=8194, D=8200), UNSUPPORTED), "dtype": (dict(dtype=3), UNSUPPORTED), "layout": (dict(layout=2), INVALID),
        "null q": (dict(q=None), INVALID), "null positions": (dict(positions=None), INVALID),
        "k without k_out": (dict(k_out=None), INVALID), "k_out without k": (dict(k=None), INVALID),
        "odd q": (dict(q=P(0) + 1), MISALIGNED), "odd inv_freq": (dict(inv_freq=P(3) + 2), MISALIGNED),
        "rows overlap": (dict(strides=(768, 255, 384, 128, 768, 256, 384, 128)), INVALID),
        "out rows overlap": (dict(strides=(768, 256, 384, 128, 767, 256, 384, 128)), INVALID),
        "negative stride": (dict(strides=(768, -256, 384, 128, 768, 256, 384, 128)), INVALID),
        "shifted in place": (dict(q_out=P(0) + 64), INVALID), "q_out on k": (dict(q_out=P(1)), INVALID),
        "in place, other strides": (dict(q_out=P(0), strides=(768, 256, 384, 128, 1024, 300, 384, 128)), INVALID),
        "q_out on k_out": (dict(k_out=P(4) + 512), INVALID), "q_out on positions": (dict(positions=P(4)), INVALID),
        "heads overflow": (dict(Hq=1 << 30), INVALID), "overflow": (dict(B=1 << 40, T=1 << 30), INVALID),
    },
    append: {
        "B=0": (dict(B=0), INVALID), "T=0": (dict(T=0), INVALID), "H=0": (dict(H=0), INVALID), "D=96": (dict(D=96), UNSUPPORTED),
        "page=8": (dict(page=8), UNSUPPORTED), "pages=0": (dict(pages=0), INVALID), "dtype": (dict(dtype=-1), UNSUPPORTED),
        "too many slots": (dict(pages=1 << 27), INVALID), "null k": (dict(k=None), INVALID), "null cache": (dict(cache=None), INVALID),
        "null slots": (dict(slots=None), INVALID), "cache alignment": (dict(cache=P(3) + 8), MISALIGNED),
        "scale alignment": (dict(ks=P(4) + 1), MISALIGNED), "odd v": (dict(v=P(1) + 1), MISALIGNED),
        "k rows": (dict(kst=255), INVALID), "v rows": (dict(vsb=700), INVALID), "k on cache": (dict(k=P(3) + 128), INVALID),
        "slots on cache": (dict(slots=P(3)), INVALID), "overflow": (dict(B=1 << 40, T=1 << 40), INVALID),
    },
    read: {
        "N=0": (dict(N=0), INVALID), "D=32": (dict(D=32), UNSUPPORTED), "page=48": (dict(page=48), UNSUPPORTED),
        "null v": (dict(v=None), INVALID), "odd k": (dict(k=P(0) + 1), MISALIGNED), "k on v": (dict(v=P(0)), INVALID),
        "k on cache": (dict(k=P(3)), INVALID), "dtype": (dict(dtype=7), UNSUPPORTED), "overflow": (dict(N=1 << 58), INVALID),
    },
    attend: {
        "B=0": (dict(B=0), INVALID), "T=0": (dict(T=0), INVALID), "Hq%H": (dict(Hq=6), INVALID), "D=80": (dict(D=80), UNSUPPORTED),
        "page=1": (dict(page=1), UNSUPPORTED), "width=0": (dict(width=0), INVALID), "window=-1": (dict(window=-1), INVALID),
        "window": (dict(window=1 << 31), INVALID), "scale inf": (dict(scale=math.inf), INVALID),
        "scale nan": (dict(scale=math.nan), INVALID), "dtype": (dict(dtype=9), UNSUPPORTED), "null q": (dict(q=None), INVALID),
        "null table": (dict(table=None), INVALID), "null lengths": (dict(lengths=None), INVALID), "null y": (dict(y=None), INVALID),
        "no workspace": (dict(ws=None), INVALID), "short workspace": (dict(ws_bytes=1000), INVALID),
        "workspace alignment": (dict(ws=P(9) + 8), MISALIGNED), "cache alignment": (dict(cache=P(1) + 4), MISALIGNED),
        "odd y": (dict(y=P(7) + 1), MISALIGNED), "odd lse": (dict(lse=P(8) + 2), MISALIGNED), "q rows": (dict(st=511), INVALID),
        "too many slots": (dict(pages=1 << 27), INVALID), "rows too long": (dict(width=1 << 27), INVALID),
        "too many rows": (dict(T=1 << 31, sb=1 << 41, st=512), INVALID), "y on q": (dict(y=P(0)), INVALID),
        "y on cache": (dict(y=P(1) + 64), INVALID), "lse on y": (dict(lse=P(7)), INVALID), "workspace on y": (dict(ws=P(7)), INVALID),
        "lse on lengths": (dict(lse=P(3)), INVALID),
    },
}


@pytest.mark.parametrize("call,name", [(c, n) for c, cases in CASES.items() for n in cases],
                         ids=lambda v: v if isinstance(v, str) else v.__name__)
def test_refusals(lib, call, name):
    change, status = CASES[call][name]
    assert call(lib, **change) == status, lib.gdn_last_error()
    assert lib.gdn_last_error()


@pytest.mark.parametrize("call", list(CASES), ids=lambda c: c.__name__)
def test_good_arguments_reach_the_launch(lib, call):
    """The arguments that the cases above change are good: they pass every check,
    up to the forced failure in front of the device."""
    gdn.force_launch_failures(1)
    try:
        assert call(lib) == CUDA
    finally:
        gdn.force_launch_failures(0)


def test_in_place_is_allowed(lib):
    for call, change in ((slots, dict(lengths_out=P(0), held_out=P(2), ring_state_out=P(3))), (slots, dict(add=None)),
                         (rotary, dict(q_out=P(0), k_out=P(1))), (rotary, dict(k=None, k_out=None, Hk=0)),
                         # q and k of the same rows, both in place
                         (rotary, dict(k=P(0) + 512, q_out=P(0), k_out=P(0) + 512,
                                       strides=(1152, 384, 1152, 384, 1152, 384, 1152, 384))),
                         (attend, dict(fresh=None, lse=None, ks=None, vs=None)),
                         (attend, dict(T=4096, sb=4096 * 512, ws=None, ws_bytes=0, B=8, fresh=None))):
        gdn.force_launch_failures(1)
        try:
            assert call(lib, **change) == CUDA, lib.gdn_last_error()
        finally:
            gdn.force_launch_failures(0)


def test_workspace_size(lib):
    assert gdn.gdn_kv_attention_workspace_size(0, 1, 8, 2, 128) == 0
    assert gdn.gdn_kv_attention_workspace_size(1, 1, 7, 2, 128) == 0
    assert gdn.gdn_kv_attention_workspace_size(1, 1, 8, 2, 100) == 0
    assert gdn.gdn_kv_attention_workspace_size(1, 1, 8, 2, 128) > 16


def test_bindings_refuse():
    """Metadata is checked before the library is called; CPU tensors go nowhere."""
    t = torch.zeros(2, 3, 4, 64, dtype=torch.bfloat16)
    i = torch.zeros(2, 3, dtype=torch.int32)
    cache = gdn.gdn_kv_cache(4, 4, 16, 64, device="cpu")
    assert cache.shape == (4, 4, 16, 72) and not cache.any()
    for wrong in (lambda: gdn.gdn_kv_cache(4, 4, 20, 64, device="cpu"), lambda: gdn.gdn_kv_cache(4, 4, 16, 96, device="cpu"),
                  lambda: gdn.gdn_rotary(t, i, torch.zeros(8)), lambda: gdn.gdn_kv_append(t, t, i, cache),
                  lambda: gdn.gdn_kv_read(cache, i), lambda: gdn.gdn_kv_attention(t, cache, i, i[:, 0]),
                  lambda: gdn.gdn_page_slots(i[:, 0], None, i[:, 0], i[0, :2], i, i[0], T=1, page=16),
                  lambda: gdn.gdn_rotary(t.double(), i, torch.zeros(8))):
        with pytest.raises(ValueError):
            wrong()
    for wrong in (lambda: gdn.gdn_rotary(None, i, torch.zeros(8)), lambda: gdn.gdn_kv_read(cache, [1, 2]),
                  lambda: gdn.gdn_page_slots([1], None, i, i, i, i, T=1, page=16)):
        with pytest.raises(TypeError):
            wrong()


def test_rotary_frequencies():
    f, scale = gdn.rotary_frequencies(64)
    assert f.dtype == torch.float32 and f.shape == (32,) and scale == 1.0
    assert torch.equal(f, (10000.0 ** -(torch.arange(0, 64, 2, dtype=torch.float64) / 64)).float())
    lin, _ = gdn.rotary_frequencies(64, scaling="linear", factor=4.0)
    assert torch.allclose(lin * 4, f, rtol=2e-7)
    base, _ = gdn.rotary_frequencies(64, scaling="base", factor=8.0)
    assert base[0] == 1.0 and abs(float(base[-1] * 8 / f[-1]) - 1) < 1e-6
    parts, s = gdn.rotary_frequencies(64, scaling="parts", factor=8.0, trained=8192, low=1.0, high=4.0)
    turns = 8192 * f.double() / (2 * math.pi)
    assert s == 1.0 and torch.equal(parts[turns > 4], f[turns > 4])
    assert torch.allclose(parts[turns < 1] * 8, f[turns < 1], rtol=2e-7) and bool((parts[1:] <= parts[:-1]).all())
    scaled, s = gdn.rotary_frequencies(64, scaling="parts_scaled", factor=8.0, trained=8192)
    assert abs(s - (1 + 0.1 * math.log(8))) < 1e-12 and scaled[0] == f[0] and abs(float(scaled[-1] * 8 / f[-1]) - 1) < 1e-6
    for wrong in (dict(R=3), dict(R=0), dict(R=8, scaling="other"), dict(R=8, scaling="parts", factor=2.0),
                  dict(R=8, scaling="linear", factor=0.5)):
        with pytest.raises(ValueError):
            gdn.rotary_frequencies(**wrong)


def test_outputs_of_the_same_rows(lib):
    """q_out and k_out may be slices of one wider row (in either order), not of each other."""
    good = (dict(q_out=P(4), k_out=P(4) + 512, strides=(768, 256, 384, 128, 1152, 384, 1152, 384)),
            dict(q_out=P(4) + 256, k_out=P(4), strides=(768, 256, 384, 128, 1152, 384, 1152, 384)),
            dict(q_out=P(4), k_out=P(4) + 512, strides=(768, 256, 384, 128, 400, 800, 400, 800)))
    bad = (dict(q_out=P(4), k_out=P(4) + 510, strides=(768, 256, 384, 128, 1152, 384, 1152, 384)),
           dict(q_out=P(4), k_out=P(4) + 514, strides=(768, 256, 384, 128, 1152, 384, 1152, 384)),
           dict(q_out=P(4), k_out=P(4) + 512, strides=(768, 256, 384, 128, 1152, 384, 1155, 385)),
           # in place, but k lies on q
           dict(q=P(0), k=P(0), q_out=P(0), k_out=P(0), strides=(1152, 384, 1152, 384, 1152, 384, 1152, 384)),
           dict(q=P(0), k=P(0) + 256, q_out=P(0), k_out=P(0) + 256, strides=(1152, 384, 1152, 384, 1152, 384, 1152, 384)))
    gdn.force_launch_failures(1000)
    try:
        for change in good:
            assert rotary(lib, **change) == CUDA, lib.gdn_last_error()
        for change in bad:
            assert rotary(lib, **change) == INVALID, change
    finally:
        gdn.force_launch_failures(0)


# wider rows [q | k | rest] of 4 + 2 heads of 64 and 64 more, and their slices' strides
ROWS = (3 * 448, 448)


@pytest.mark.parametrize("change", [
    # q in place, the keys on its rows or partly on them, k_out apart
    dict(q=P(0), k=P(0), q_out=P(0), strides=(768, 256, 384, 128, 768, 256, 384, 128)),
    dict(q=P(0), k=P(0) + 256, q_out=P(0), strides=(768, 256, 768, 256, 768, 256, 384, 128)),
    dict(q=P(0), k=P(0) + 510, q_out=P(0), strides=ROWS * 3 + (384, 128)),
    dict(q=P(0), k=P(0) - 254, q_out=P(0), strides=ROWS * 3 + (384, 128)),
    # keys between the queries' rows, whose rows do not keep to the gaps
    dict(q=P(0), k=P(0) + 512, q_out=P(0), strides=ROWS + (3 * 500, 500) + ROWS + (384, 128)),
    # and the other way round: k in place, the queries on its rows, q_out apart
    dict(k=P(1), q=P(1), k_out=P(1), strides=(768, 256, 768, 256, 768, 256, 768, 256)),
    dict(k=P(1), q=P(1) - 256, k_out=P(1), strides=(768, 256, 768, 256, 768, 256, 768, 256)),
    dict(k=P(1), q=P(1) + 254, k_out=P(1), strides=ROWS * 2 + (768, 256) + ROWS),
    dict(k=P(1), q=P(1) + 256, k_out=P(1), strides=(3 * 500, 500) + ROWS + (768, 256) + ROWS),
])
def test_one_in_place_on_the_other_input(lib, change):
    """Of q and k the one that is turned in place may not lie on the other one, which
    is read at the same time."""
    gdn.force_launch_failures(1)
    try:
        assert rotary(lib, **change) == INVALID
    finally:
        gdn.force_launch_failures(0)


@pytest.mark.parametrize("change", [
    dict(q=P(0), k=P(0) + 512, q_out=P(0), strides=ROWS * 3 + (384, 128)),
    dict(q=P(0) + 256, k=P(0), q_out=P(0) + 256, strides=ROWS * 3 + (384, 128)),
    dict(k=P(1) + 512, q=P(1), k_out=P(1) + 512, strides=ROWS * 2 + (768, 256) + ROWS),
    dict(k=P(1), q=P(1) + 256, k_out=P(1), strides=ROWS * 2 + (768, 256) + ROWS),
])
def test_one_in_place_of_slices_of_the_same_rows(lib, change):
    gdn.force_launch_failures(1)
    try:
        assert rotary(lib, **change) == CUDA, lib.gdn_last_error()
    finally:
        gdn.force_launch_failures(0)


def neighbours(values):
    """The values, every midpoint between neighbours, and one float32 step on either side
    of all of them (at least 0), with the index of the nearest value: of a midpoint the
    even one."""
    x, want = [], []
    for i, v in enumerate(values):
        x.append(v)
        want.append(i)
        if i + 1 < len(values):
            x.append((v + values[i + 1]) / 2)
            want.append(i if i % 2 == 0 else i + 1)
    x, want = torch.tensor(x, dtype=torch.float64), torch.tensor(want)
    exact = x.float()
    assert torch.equal(exact.double(), x)
    up, down = (torch.nextafter(exact, torch.full_like(exact, s)) for s in (math.inf, 0.0))
    i = torch.arange(len(x)) // 2
    return torch.cat([exact, up, down]), torch.cat([want, torch.where(torch.arange(len(x)) % 2 == 1, i + 1, i), i])


def test_reference_of_scales():
    """The tests' quantiser gives each scale byte where its value, a midpoint or a float
    beside one says so, as torch's own e4m3 does."""
    import attention_reference as ref
    assert torch.equal(torch.tensor(ref.E4M3), torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).float())
    top, want = neighbours([6 * v for v in ref.E4M3])  # a group's largest, whose sixth the scale is
    u = torch.zeros(len(top), 1, 16)
    u[:, 0, 3] = top
    byte = ref.quantise(u, None)[1][:, 0, 0]
    assert torch.equal(byte, want)
    sixth = (top.double() / 6).float()
    exact = sixth.double() * 6 == top.double()
    assert int(exact.sum()) >= 2 * 127 - 1
    assert torch.equal(byte[exact].to(torch.uint8), sixth[exact].to(torch.float8_e4m3fn).view(torch.uint8))
    assert int(ref.quantise(torch.full((1, 1, 16), 1e9), None)[1]) == 126  # the largest scale, no further


@pytest.mark.parametrize("byte", [1, 8, 56, 61, 126])
def test_reference_of_codes(byte):
    """... and each code, of both signs, under scales that are subnormal, one, odd and the largest."""
    import attention_reference as ref
    s = ref.E4M3[byte]
    table = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    x, want = neighbours([v * s for v in table])
    keep = x <= 6 * s
    x, want = x[keep], want[keep]
    u = torch.zeros(2, len(x), 1, 16)
    u[..., 0] = 6 * s  # fixes the group's scale
    u[0, :, 0, 5], u[1, :, 0, 5] = x, -x
    code, sb = ref.quantise(u, None)
    assert bool((sb == byte).all())
    code = code[..., 0, 5]
    assert torch.equal(code[0], want) and torch.equal(code[1] % 8, want) and bool((code[1] >= 8)[x > 0].all())
    assert torch.equal(ref.values(ref.quantise(u, None)[0], sb, None)[0, :, 0, 5],
                       torch.tensor(table, dtype=torch.float64)[want] * s)


def test_reference_of_infinities():
    """A NaN is held as zero, an infinity as the largest value of the largest scale."""
    import attention_reference as ref
    u = torch.tensor([math.nan, math.inf, -math.inf, 1.0] + [0.0] * 12).view(1, 1, 16)
    code, byte = ref.quantise(u, None)
    assert code[0, 0, :4].tolist() == [0, 7, 15, 0] and int(byte) == 126


@pytest.mark.parametrize("wrong", [
    dict(base=0.0), dict(base=-2.0), dict(base=math.nan), dict(base=1.0, scaling="parts_scaled", factor=2.0, trained=100),
    dict(scaling="parts", factor=2.0, trained=-5), dict(scaling="parts_scaled", factor=2.0, trained=-5),
    dict(scaling="parts", factor=2.0, trained=100, low=4.0, high=2.0), dict(scaling="linear", factor=math.nan)])
def test_rotary_frequencies_refuse(wrong):
    with pytest.raises(ValueError, match="must be|needs"):
        gdn.rotary_frequencies(64, **wrong)
