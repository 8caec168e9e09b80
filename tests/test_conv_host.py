"""The convolution's own source on the host (host_cuda.h): its float64 form, and
single blocks of a call of more steps than 32 bits count."""
from __future__ import annotations

import ctypes
import subprocess
import sys

import numpy as np
import pytest

import host_cuda
import layer_reference as ref

ENTRY = r"""
extern "C" int host_conv(const float *x, const float *w, const float *bias, const float *state, const int32_t *lengths,
                         float *y, float *state_out, int64_t B, int64_t T, int64_t C, int64_t x_sb, int64_t x_st, int W,
                         int vec, int sms) {
    gdn::ConvArgs a{x, w, bias, state, lengths, y, state_out, B, T, C, x_sb, x_st, W, true, vec != 0};
    return gdn::launch_causal_conv(gdn::DType::F32, a, sms, nullptr);
}

// One channel of bf16 over T steps of which the sequence has `length`: the
// blocks of the first run, of the run at `mid` and of the last.  Only the first
// block's pages of y are writable.
extern "C" int host_conv_far(int64_t T, int32_t length, int64_t mid) {
    auto map = [](int64_t bytes, int how) {
        void *p = mmap(nullptr, bytes, how, MAP_PRIVATE | MAP_ANONYMOUS | MAP_NORESERVE, -1, 0);
        if (p == MAP_FAILED) exit(3);
        return p;
    };
    auto *x = static_cast<__nv_bfloat16 *>(map(T * 2, PROT_READ));
    auto *y = static_cast<__nv_bfloat16 *>(map(T * 2, PROT_READ));
    mprotect(y, 4096, PROT_READ | PROT_WRITE);
    __nv_bfloat16 w[4] = {}, bias[1] = {{0x3f80}}, state_out[3];
    gdn::ConvArgs a{x, w, bias, nullptr, &length, y, state_out, 1, T, 1, T, 1, 4, false, false};
    constexpr int run = 64;
    const int64_t runs = (T + run - 1) / run;
    blockDim = dim3(128);
    threadIdx = {0, 0, 0};
    for (int64_t r : {(int64_t)0, mid / run, runs - 1}) {
        blockIdx = {(unsigned)r, 0, 0};
        gdn::conv_kernel<__nv_bfloat16, 1, 4>(a, run, runs, 1);
    }
    for (int t = 0; t < 2048; ++t)
        if (y[t].bits != (t < length ? 0x3f80 : 0)) return 1;
    return 0;
}
"""


@pytest.fixture(scope="module")
def path(tmp_path_factory):
    return host_cuda.compile_unit(["layer.h", "pieces.cuh", "causal_conv.cu"], ENTRY,
                                  str(tmp_path_factory.mktemp("host")), "conv")


@pytest.mark.parametrize("B,T,C,W,pad,sms", [(2, 1, 8, 4, 0, 152), (3, 70, 12, 4, 4, 1), (2, 200, 5, 8, 2, 1),
                                             (1, 9, 4, 2, 0, 152)])
def test_conv(path, B, T, C, W, pad, sms):
    rng = np.random.default_rng(T)
    f32 = lambda *s: rng.standard_normal(s).astype(np.float32)  # noqa: E731
    wide, w, bias, st = f32(B, T, C + pad), f32(C, W), f32(C), f32(B, W - 1, C)
    n = rng.integers(0, T + 1, B).astype(np.int32)
    y, so = np.full((B, T, C), np.nan, np.float32), np.full((B, W - 1, C), np.nan, np.float32)
    p = lambda a: ctypes.c_void_p(a.ctypes.data)  # noqa: E731
    vec = C % 4 == 0 and (C + pad) % 4 == 0
    assert ctypes.CDLL(path).host_conv(
        p(wide), p(w), p(bias), p(st), p(n), p(y), p(so), *(ctypes.c_int64(v) for v in (B, T, C, T * (C + pad), C + pad)),
        W, int(vec), sms) == 0
    want, bound, s_want, on = ref.conv(wide[..., :C].astype(np.float64), *(a.astype(np.float64) for a in (w, bias, st)), n)
    assert np.array_equal(so, s_want)
    assert (np.abs(y - want)[on] <= bound[on]).all() and np.isnan(y[~on]).all()


@pytest.mark.parametrize("T", [(1 << 31) + 640, (1 << 32) + 192, (1 << 33) + 64])
def test_more_steps_than_32_bits(path, T):
    """Blocks past the end of a short sequence write nothing, however far."""
    code = f"import ctypes, sys; f = ctypes.CDLL({path!r}).host_conv_far; " \
           f"sys.exit(f(ctypes.c_int64({T}), 5, ctypes.c_int64({(1 << 31) + 128})))"
    assert subprocess.run([sys.executable, "-c", code]).returncode == 0
