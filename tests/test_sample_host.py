"""The sampling kernel's own source, run on the host (host_cuda.h), against
the float64 form: its cuts through groups of equal logits, rows over one block
and over clusters, and every shared and row access inside its memory.
"""
from __future__ import annotations

import ctypes

import numpy as np
import pytest

import host_cuda
import layer_reference as ref
from sample_cases import TIED_CUTS, bracket_edge, tied_cut

torch = pytest.importorskip("torch")

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
CODES = {"f32": 0, "bf16": 1, "f16": 2}

ENTRY = r"""
extern "C" const char *host_sample(int dtype, const void *logits, const float *noise, const float *temperature,
                                   const int32_t *top_k, const float *top_p, const float *min_p, int32_t *token,
                                   float *logprob, int64_t R, int64_t V, int64_t logits_st, int64_t noise_st, int sms) {
    gdn::SampleArgs a{};
    a.logits = logits, a.noise = noise, a.temperature = temperature, a.top_k = top_k, a.top_p = top_p, a.min_p = min_p;
    a.token = token, a.logprob = logprob, a.R = R, a.V = V, a.logits_st = logits_st, a.noise_st = noise_st;
    const uintptr_t l = (uintptr_t)logits, n = (uintptr_t)noise;
    // (a row's first and last piece may reach past its tokens, and are not read whole)
    host::m.ranges = {{l, l + ((R - 1) * logits_st + V) * (dtype ? 2 : 4)}, {n, n + ((R - 1) * noise_st + V) * 4}};
    const cudaError_t e = gdn::launch_sample((gdn::DType)dtype, a, sms, nullptr);
    if (e == cudaErrorLaunchFailure) return host::m.error;
    return e == cudaSuccess ? "" : "not launched";
}
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    path = host_cuda.compile_unit(["layer.h", "pieces.cuh", "sample.cu"], ENTRY, str(tmp_path_factory.mktemp("host")),
                                  "sample")
    lib = ctypes.CDLL(path)
    lib.host_sample.argtypes = [ctypes.c_int] + [ctypes.c_void_p] * 8 + [ctypes.c_int64] * 4 + [ctypes.c_int]
    lib.host_sample.restype = ctypes.c_char_p
    return lib


def sample(lib, logits, noise, dtype, sms, pad=0, off=0, **settings):
    """Tokens and log probabilities of float64 rows; `sms` decides over how many
    blocks a row goes.  Also the rows as the type holds them."""
    R, V = logits.shape
    wide = torch.full((R, off + V + pad), 7.0, dtype=TYPES[dtype])
    l = wide[:, off:off + V]
    l.copy_(torch.from_numpy(logits))
    one = dict(temperature=1.0, top_k=0, top_p=1.0, min_p=0.0) | settings
    s = {k: np.ascontiguousarray(np.broadcast_to(v, R), np.int32 if k == "top_k" else np.float32) for k, v in one.items()}
    noise = np.ascontiguousarray(noise, np.float32)
    token, logprob = np.full(R, -7, np.int32), np.full(R, np.nan, np.float32)
    p = lambda a: a.ctypes.data  # noqa: E731
    error = lib.host_sample(CODES[dtype], l.data_ptr(), p(noise), p(s["temperature"]), p(s["top_k"]), p(s["top_p"]),
                            p(s["min_p"]), p(token), p(logprob), R, V, off + V + pad, V, sms)
    assert not error, error.decode()
    return token, logprob, l.double().numpy(), s


def hold(lib, logits, noise, dtype, sms, **kw):
    token, logprob, l64, s = sample(lib, logits, noise, dtype, sms, **kw)
    want = [ref.sample(l64[r], noise[r].astype(np.float32), *(s[k][r] for k in ("temperature", "top_k", "top_p", "min_p")))
            for r in range(len(l64))]
    assert token.tolist() == [t for t, _ in want]
    lp = np.array([v for _, v in want])
    fine = np.isfinite(lp)
    assert np.array_equal(fine, np.isfinite(logprob))
    assert (np.abs(logprob[fine] - lp[fine]) <= 2e-5 + 4 * ref.U * np.abs(lp[fine])).all()


@pytest.mark.parametrize("sms", [1, 4, 152], ids=["one block", "two", "cluster"])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_settings(lib, dtype, sms):
    """Every cut and their combinations on ordinary rows at an odd stride."""
    rng = np.random.default_rng(sms)
    R, V = 7, 9001
    logits = 2.5 * rng.standard_normal((R, V))
    logits[:, rng.integers(0, V, 90)] = -np.inf
    logits[5, ::3] = np.nan
    noise = rng.standard_exponential((R, V))
    hold(lib, logits, noise, dtype, sms, pad=2, off=1, temperature=[1, .7, 1.3, 1, .9, 1, 0],
         top_k=[0, 50, 0, 300, 0, 20, 5], top_p=[1, 1, .9, .8, 1, .95, .5], min_p=[0, 0, 0, 0, .02, .01, 0])


@pytest.mark.parametrize("V", [1, 3, 17, 1003])
def test_short_rows(lib, V):
    rng = np.random.default_rng(V)
    noise = rng.standard_exponential((4, V))
    for dtype in TYPES:
        logits = rng.standard_normal((4, V))
        logits[2] = -np.inf
        hold(lib, logits, noise, dtype, 152, pad=3, off=2, top_k=[0, 2, 2, 0], top_p=[1, 1, .9, .9])


@pytest.mark.parametrize("sms", [1, 4, 152], ids=["one block", "two", "cluster"])
@pytest.mark.parametrize("name", list(TIED_CUTS))
def test_top_p_stays_inside_top_k(lib, name, sms):
    """A token that top-k removed by its index stays out, however top-p ends."""
    for dtype in ("bf16", "f32") if sms != 4 else ("f16",):
        l, s, noise = tied_cut(name)
        hold(lib, l[None], noise[None], dtype, sms, **s)


@pytest.mark.parametrize("seed", [2, 3, 7, 15, 22, 23, 30])
def test_nucleus_at_the_edge_of_its_bracket(lib, seed):
    """Rows whose running masses pass the bracket's first value in the rounding
    between one thread's sum and the next one's: the cut is found all the same
    (noise lets every token past it win, were it left)."""
    l, p = bracket_edge(seed)
    ps = (p.view(np.int32) + np.arange(-2, 3, dtype=np.int32)).view(np.float32)
    full = np.argsort(-l, kind="stable")
    noise = np.ones((5, len(l)), np.float32)
    for r in range(5):
        n = len(ref.kept_order(l, 1.0, 0, ps[r], 0.0)[0])
        assert 1490 < n < 1510
        noise[r, full[n:]] = 1e-25
        noise[r, full[n - 1]] = 1e-10
    hold(lib, np.repeat(l[None], 5, 0), noise, "f32", 1, top_p=ps)


@pytest.mark.parametrize("sms", [1, 152], ids=["one block", "cluster"])
def test_extreme_settings(lib, sms):
    """Temperatures at both ends, nuclei of next to nothing and next to all."""
    rng = np.random.default_rng(3)
    R, V = 12, 5001
    logits = 3 * rng.standard_normal((R, V))
    logits[:, ::7] = -np.inf
    logits[8:, 3:] = -np.inf
    noise = rng.standard_exponential((R, V))
    hold(lib, logits, noise, "f32", sms,
         temperature=[3e38, 3e38, 1e30, 1e-30, 1e-45, 1, 1, 1, 3e38, 1e-30, 1, 1],
         top_k=[0, 300, 20, 0, 0, 0, 0, 2000, 0, 0, 300, 2],
         top_p=[.4, .4, .9, .9, 1, 1e-30, .9999999, .9999999, .6, .6, .9999999, .9],
         min_p=[0, 0, .5, 0, 1e-30, 0, 0, 0, 1, 0, 0, 1e-40])
