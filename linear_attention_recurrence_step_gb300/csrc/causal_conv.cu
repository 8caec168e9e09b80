// causal_conv.cu -- the short depthwise causal convolution in front of a
// recurrence, with the last W-1 inputs of a sequence as its state:
//     y[b,t,c] = act(bias[c] + sum_j weight[c,j] in[b, t-W+1+j, c])
// where in[b,t] is x[b,t] for t >= 0 and state_in[b, W-1+t] before it.
//
// Bound by memory: every input is read once and every output written once
// (2 W + 4 operations per element).  A thread owns one 16-byte piece of
// channels and a run of consecutive steps; the window of W-1 earlier inputs
// stays in its registers, so a run re-reads only the W-1 steps before it.
// Sums are f32 and rounded once.
//
// Measured (4096 steps of 8192 bf16 channels, width 4): 27.4 us, 4.9 TB/s of
// the bytes it cannot do without; the inputs read again at the start of a run
// come from L2.  16 x 8 steps: 4.6 us, one step of 32 sequences: 3.5 us, which
// are a launch and two dependent loads.
#include "pieces.cuh"
#include "layer.h"

namespace gdn {

namespace {

constexpr int kConvThreads = 128;
// Steps whose loads are issued together.
template <int VEC> struct ConvBatch { static constexpr int value = VEC == 1 ? 8 : 4; };

// blockIdx.x: (sequence, run of steps, block of channel pieces), channels
// innermost.
template <typename T, int VEC, int W>
__global__ void __launch_bounds__(kConvThreads, W <= 4 ? 4 : 2) conv_kernel(const ConvArgs a, int run, int64_t runs,
                                                            int64_t cblocks) {
    constexpr int BATCH = ConvBatch<VEC>::value;
    pdl_trigger();
    pdl_wait();
    const int64_t blk = blockIdx.x;
    const int64_t cb = blk % cblocks, rb = blk / cblocks;
    const int64_t r = rb % runs, b = rb / runs;
    const int64_t c = (cb * kConvThreads + threadIdx.x) * VEC;
    if (c >= a.C) return;
    const T *x = static_cast<const T *>(a.x) + b * a.x_sb + c;
    const T *sin = a.state_in ? static_cast<const T *>(a.state_in) + b * (W - 1) * a.C + c : nullptr;
    int64_t len = a.T;
    if (a.lengths) {
        const int64_t n = a.lengths[b];
        len = n < 0 ? 0 : (n < a.T ? n : a.T);
    }
    const int64_t t0 = r * run;
    const int64_t t1 = t0 + run < len ? t0 + run : len;

    constexpr int NP = kPairs<VEC>;
    float2 w[W][NP], bias[NP];
    {
        const T *wp = static_cast<const T *>(a.weight) + c * W;
        float taps[W * VEC];  // VEC * W consecutive taps, VEC at a time
#pragma unroll
        for (int p = 0; p < W; ++p) {
            float piece[VEC];
            load_piece<T, VEC>(piece, wp + p * VEC);
#pragma unroll
            for (int i = 0; i < VEC; ++i) taps[p * VEC + i] = piece[i];
        }
#pragma unroll
        for (int j = 0; j < W; ++j)
#pragma unroll
            for (int i = 0; i < NP; ++i)
                w[j][i] = make_float2(taps[2 * i * W + j], 2 * i + 1 < VEC ? taps[(2 * i + 1) % VEC * W + j] : 0.f);
#pragma unroll
        for (int i = 0; i < NP; ++i) bias[i] = make_float2(0.f, 0.f);
        if (a.bias) widen2<T, VEC>(bias, load_raw<T, VEC>(static_cast<const T *>(a.bias) + c));
    }

    // win[j]: the input W-1-j steps before the current one
    float2 win[W - 1][NP];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
        const int64_t t = t0 - (W - 1) + j;
        if (t >= 0) widen2<T, VEC>(win[j], load_raw<T, VEC>(x + t * a.x_st));
        else if (sin) widen2<T, VEC>(win[j], load_raw<T, VEC>(sin + (W - 1 + t) * a.C));
        else
#pragma unroll
            for (int i = 0; i < NP; ++i) win[j][i] = make_float2(0.f, 0.f);
    }
    // the first run's thread also writes the new state, a copy of inputs: it
    // alone reads state_in at its channels and has done so before it writes,
    // so state_out may be state_in
    if (a.state_out && r == 0) {
        T *so = static_cast<T *>(a.state_out) + b * (W - 1) * a.C + c;
        RawPiece<T, VEC> next[W - 1];
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
            const int64_t t = len - (W - 1) + j;
            if (t >= 0) next[j] = load_raw<T, VEC>(x + t * a.x_st);
            else if (sin) next[j] = load_raw<T, VEC>(sin + (W - 1 + t) * a.C);
            else next[j] = RawPiece<T, VEC>{};
        }
#pragma unroll
        for (int j = 0; j < W - 1; ++j) store_raw<T, VEC>(so + j * a.C, next[j]);
    }
    if (!a.y) return;
    // the next batch of steps is on its way while one is worked on
    if (t1 <= t0) return;
    int left = (int)(t1 - t0);  // run at most
    const T *px = x + t0 * a.x_st;
    T *py = static_cast<T *>(a.y) + (b * a.T + t0) * a.C + c;
    RawPiece<T, VEC> raw[BATCH];
    auto fetch = [&](int n) {
        if (n >= BATCH) {
#pragma unroll
            for (int k = 0; k < BATCH; ++k) raw[k] = load_raw<T, VEC>(px + k * a.x_st);
        } else {
#pragma unroll
            for (int k = 0; k < BATCH; ++k)
                if (k < n) raw[k] = load_raw<T, VEC>(px + k * a.x_st);
        }
        px += BATCH * a.x_st;
    };
    auto step = [&](const RawPiece<T, VEC> &now) {
        float2 in[NP], out[NP];
        widen2<T, VEC>(in, now);
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            float2 s = bias[i];
#pragma unroll
            for (int j = 0; j < W - 1; ++j) s = ffma2(w[j][i], win[j][i], s);
            s = ffma2(w[W - 1][i], in[i], s);
            out[i] = a.silu ? silu2(s) : s;
        }
        store_piece2<T, VEC>(py, out);
        py += a.C;
#pragma unroll
        for (int i = 0; i < NP; ++i) {
#pragma unroll
            for (int j = 0; j < W - 2; ++j) win[j][i] = win[j + 1][i];
            win[W - 2][i] = in[i];
        }
    };
    fetch(left);
    for (; left >= BATCH; left -= BATCH) {
        RawPiece<T, VEC> now[BATCH];
#pragma unroll
        for (int k = 0; k < BATCH; ++k) now[k] = raw[k];
        fetch(left - BATCH);
#pragma unroll
        for (int k = 0; k < BATCH; ++k) step(now[k]);
    }
#pragma unroll
    for (int k = 0; k < BATCH; ++k)
        if (k < left) step(raw[k]);
}

template <typename T, int VEC, int W>
cudaError_t launch_w(const ConvArgs &a, int sm_count, cudaStream_t s) {
    const int64_t cblocks = (a.C + (int64_t)kConvThreads * VEC - 1) / ((int64_t)kConvThreads * VEC);
    // Steps per thread: up to 64, fewer while there are not three blocks per SM.
    // 4096 steps of 8192 channels: 27.4 us by 64, 29.5 by 32, 34.0 by 16, 40.9 by
    // 8; 512 steps: 9.6 us by 32, 5.7 by 8.
    int run = 64;
    const int64_t want = 3 * (int64_t)(sm_count > 0 ? sm_count : 152);
    if (!a.y || a.T <= 8) run = 8;
    while (run > 8 && a.B * cblocks * ((a.T + run - 1) / run) < want) run /= 2;
    const int64_t runs = a.y ? (a.T + run - 1) / run : 1;
    const int64_t blocks = a.B * runs * cblocks;
    if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
    return launch_dependent(conv_kernel<T, VEC, W>, (unsigned)blocks, kConvThreads, 0, s, a, run, runs, cblocks);
}

template <typename T, int VEC>
cudaError_t launch_v(const ConvArgs &a, int sm_count, cudaStream_t s) {
    switch (a.W) {
    case 2: return launch_w<T, VEC, 2>(a, sm_count, s);
    case 3: return launch_w<T, VEC, 3>(a, sm_count, s);
    case 4: return launch_w<T, VEC, 4>(a, sm_count, s);
    case 5: return launch_w<T, VEC, 5>(a, sm_count, s);
    case 6: return launch_w<T, VEC, 6>(a, sm_count, s);
    case 7: return launch_w<T, VEC, 7>(a, sm_count, s);
    case 8: return launch_w<T, VEC, 8>(a, sm_count, s);
    }
    return cudaErrorInvalidValue;
}

template <typename T>
cudaError_t launch_t(const ConvArgs &a, int sm_count, cudaStream_t s) {
    return a.vec ? launch_v<T, 16 / sizeof(T)>(a, sm_count, s) : launch_v<T, 1>(a, sm_count, s);
}

}  // namespace

cudaError_t launch_causal_conv(DType dt, const ConvArgs &a, int sm_count, cudaStream_t s) {
    switch (dt) {
    case DType::F32: return launch_t<float>(a, sm_count, s);
    case DType::BF16: return launch_t<__nv_bfloat16>(a, sm_count, s);
    case DType::F16: return launch_t<__half>(a, sm_count, s);
    }
    return cudaErrorInvalidValue;
}

}  // namespace gdn
