// layer_abi.cu -- C entry points of the operators around the recurrence
// (declared in include/gdn.h): argument checks and dispatch.  Checks run on
// the host, before any CUDA call, under the rules of abi.cu.
#include <algorithm>
#include <cmath>
#include <utility>

#include "abi_util.h"
#include "layer.h"

using namespace gdn::abi;

extern "C" {

gdn_status gdn_causal_conv(const void *x, const void *weight, const void *bias, const void *state_in,
                           const int32_t *lengths, void *y, void *state_out, int64_t B, int64_t T, int64_t C,
                           int64_t W, int64_t x_stride_b, int64_t x_stride_t, gdn_activation activation,
                           gdn_dtype dtype, gdn_stream_t stream) {
    const char *fn = "gdn_causal_conv";
    const int eb = elem_bytes(dtype);
    if (eb == 0) return fail(GDN_ERR_UNSUPPORTED, "%s: unknown dtype %d", fn, (int)dtype);
    if (B <= 0 || T <= 0 || C <= 0 || W <= 0)
        return fail(GDN_ERR_INVALID_ARGUMENT, "%s: B, T, C, W must all be > 0", fn);
    if (W < 2 || W > 8) return fail(GDN_ERR_UNSUPPORTED, "%s: W (%lld) must be 2 to 8", fn, (long long)W);
    if (activation != GDN_ACT_NONE && activation != GDN_ACT_SILU)
        return fail(GDN_ERR_INVALID_ARGUMENT, "%s: unknown activation %d", fn, (int)activation);
    if (!x || !weight) return fail(GDN_ERR_INVALID_ARGUMENT, "%s: x and weight must be non-NULL", fn);
    if (!y && !state_out) return fail(GDN_ERR_INVALID_ARGUMENT, "%s: y and state_out are both NULL", fn);
    const int64_t x_b = scaled(extent(B, x_stride_b, T, x_stride_t, C), eb);
    const int64_t y_b = nbytes({B, T, C}, eb), s_b = nbytes({B, W - 1, C}, eb), w_b = nbytes({C, W}, eb);
    if (y_b < 0 || s_b < 0 || w_b < 0) return fail(GDN_ERR_INVALID_ARGUMENT, "%s: tensor sizes overflow int64", fn);
    if (x_b < 0)
        return fail(GDN_ERR_INVALID_ARGUMENT, "%s: x strides (%lld, %lld) overlap its rows or overflow", fn,
                    (long long)x_stride_b, (long long)x_stride_t);
    for (const void *p : {x, weight, bias, state_in, (const void *)y, (const void *)state_out})
        if (!aligned(p, eb)) return fail(GDN_ERR_MISALIGNED, "%s: a tensor is not aligned to its element size", fn);
    if (!aligned(lengths, 4)) return fail(GDN_ERR_MISALIGNED, "%s: lengths must be 4-byte aligned", fn);
    if (state_in && state_out && state_in != state_out && overlap(state_in, s_b, state_out, s_b))
        return fail(GDN_ERR_INVALID_ARGUMENT, "%s: state_out overlaps state_in without being the same buffer", fn);
    if (over(y, y_b, x, x_b) || over(y, y_b, state_in, s_b) || over(y, y_b, state_out, s_b) ||
        over(state_out, s_b, x, x_b))
        return fail(GDN_ERR_INVALID_ARGUMENT, "%s: an output overlaps another tensor", fn);
    for (const auto &[o, o_b] : {std::pair<const void *, int64_t>(y, y_b), {state_out, s_b}})
        if (over(o, o_b, weight, w_b) || over(o, o_b, bias, C * eb) || over(o, o_b, lengths, B * 4))
            return fail(GDN_ERR_INVALID_ARGUMENT, "%s: an output overlaps weight, bias or lengths", fn);

    if (take_forced_failure()) return forced_failure(fn);
    cudaError_t e;
    const int sms = current_sm_count(&e);
    if (e != cudaSuccess) return cuda_fail(fn, "device query", e);
    gdn::ConvArgs a{};
    a.x = x;
    a.weight = weight;
    a.bias = bias;
    a.state_in = state_in;
    a.lengths = lengths;
    a.y = y;
    a.state_out = state_out;
    a.B = B;
    a.T = T;
    a.C = C;
    a.x_sb = x_stride_b;
    a.x_st = x_stride_t;
    a.W = (int)W;
    a.silu = activation == GDN_ACT_SILU;
    a.vec = C * eb % 16 == 0 && (B == 1 || x_stride_b * eb % 16 == 0) && (T == 1 || x_stride_t * eb % 16 == 0) &&
            aligned(x, 16) && aligned(weight, 16) && aligned(bias, 16) && aligned(state_in, 16) && aligned(y, 16) &&
            aligned(state_out, 16);
    e = gdn::launch_causal_conv(static_cast<gdn::DType>(dtype), a, sms, reinterpret_cast<cudaStream_t>(stream));
    if (e == cudaErrorInvalidConfiguration) return fail(GDN_ERR_INVALID_ARGUMENT, "%s: grid too large", fn);
    if (e != cudaSuccess) return cuda_fail(fn, "launch", e);
    return ok();
}

size_t gdn_selective_scan_workspace_size(int64_t B, int64_t T, int64_t H, int64_t P, int64_t N) {
    if (B <= 0 || T <= 0 || H <= 0 || P <= 0 || !gdn::scan_supported_n(N)) return 0;
    // whichever form the call takes
    const gdn::ScanPlan p = gdn::scan_plan(B, T, H, P, N, false), q = gdn::scan_plan(B, T, H, P, N, true);
    return p.bytes < 0 || q.bytes < 0 ? 0 : (size_t)std::max<int64_t>(std::max(p.bytes, q.bytes), 16);
}

gdn_status gdn_selective_scan(const void *x, const void *dt, const float *A, const void *Bm, const void *Cm,
                              const float *D, const float *dt_bias, const float *state_in, const int32_t *lengths,
                              void *y, float *state_out, int64_t B, int64_t T, int64_t H, int64_t P, int64_t G,
                              int64_t N, const gdn_scan_strides *strides, int softplus, void *workspace,
                              size_t workspace_bytes, gdn_dtype dtype, gdn_stream_t stream) {
    const char *fn = "gdn_selective_scan";
    const int eb = elem_bytes(dtype);
    if (eb == 0) return fail(GDN_ERR_UNSUPPORTED, "%s: unknown dtype %d", fn, (int)dtype);
    if (B <= 0 || T <= 0 || H <= 0 || P <= 0 || G <= 0 || N <= 0)
        return fail(GDN_ERR_INVALID_ARGUMENT, "%s: B, T, H, P, G, N must all be > 0", fn);
    if (H % G != 0)
        return fail(GDN_ERR_INVALID_ARGUMENT, "%s: H (%lld) must be a multiple of G (%lld)", fn, (long long)H,
                    (long long)G);
    if (!gdn::scan_supported_n(N))
        return fail(GDN_ERR_UNSUPPORTED, "%s: N (%lld) must be 16, 32, 64, 128 or 256", fn, (long long)N);
    if (!x || !dt || !A || !Bm || !Cm)
        return fail(GDN_ERR_INVALID_ARGUMENT, "%s: x, dt, A, B and C must be non-NULL", fn);
    if (!y && !state_out) return fail(GDN_ERR_INVALID_ARGUMENT, "%s: y and state_out are both NULL", fn);
    const int64_t y_b = nbytes({B, T, H, P}, eb), st_b = nbytes({B, H, P, N}, 4), bc_d = nbytes({B, T, G, N}, eb);
    if (y_b < 0 || st_b < 0 || bc_d < 0) return fail(GDN_ERR_INVALID_ARGUMENT, "%s: tensor sizes overflow int64", fn);
    gdn_scan_strides st{T * H * P, H * P, T * H, H, T * G * N, G * N, T * G * N, G * N};
    if (strides) st = *strides;
    const int64_t x_b = scaled(extent(B, st.x_b, T, st.x_t, H * P), eb), dt_b = scaled(extent(B, st.dt_b, T, st.dt_t, H), eb);
    const int64_t b_b = scaled(extent(B, st.B_b, T, st.B_t, G * N), eb), c_b = scaled(extent(B, st.C_b, T, st.C_t, G * N), eb);
    if (x_b < 0 || dt_b < 0 || b_b < 0 || c_b < 0)
        return fail(GDN_ERR_INVALID_ARGUMENT, "%s: strides of x, dt, B or C overlap their rows or overflow", fn);
    for (const void *p : {x, dt, Bm, Cm, (const void *)y})
        if (!aligned(p, eb)) return fail(GDN_ERR_MISALIGNED, "%s: a tensor is not aligned to its element size", fn);
    if (!aligned(A, 4) || !aligned(D, 4) || !aligned(dt_bias, 4) || !aligned(lengths, 4))
        return fail(GDN_ERR_MISALIGNED, "%s: A, D, dt_bias and lengths must be 4-byte aligned", fn);
    if (!aligned(state_in, 16) || !aligned(state_out, 16) || !aligned(workspace, 16))
        return fail(GDN_ERR_MISALIGNED, "%s: state_in, state_out and workspace must be 16-byte aligned", fn);
    if (state_in && state_out && state_in != state_out && overlap(state_in, st_b, state_out, st_b))
        return fail(GDN_ERR_INVALID_ARGUMENT, "%s: state_out overlaps state_in without being the same buffer", fn);
    const bool rows16 = aligned(x, 16) && aligned(Bm, 16) && aligned(Cm, 16) && aligned(y, 16) && st.x_t % 8 == 0 &&
                        st.B_t % 8 == 0 && st.C_t % 8 == 0 &&
                        (B == 1 || (st.x_b % 8 == 0 && st.B_b % 8 == 0 && st.C_b % 8 == 0));
    const bool chunked = rows16 && gdn::scan_chunk_sizes(static_cast<gdn::DType>(dtype), T, P, N);
    const gdn::ScanPlan plan = gdn::scan_plan(B, T, H, P, N, chunked);
    if (plan.bytes < 0) return fail(GDN_ERR_INVALID_ARGUMENT, "%s: tensor sizes overflow int64", fn);
    if (plan.bytes > 0 && (!workspace || workspace_bytes < (size_t)plan.bytes))
        return fail(GDN_ERR_INVALID_ARGUMENT, "%s: workspace too small: need %lld bytes, have %llu", fn,
                    (long long)plan.bytes, (unsigned long long)(workspace ? workspace_bytes : 0));
    const void *outs[3] = {y, state_out, plan.bytes > 0 ? workspace : nullptr};
    const int64_t out_b[3] = {y_b, st_b, plan.bytes};
    for (int i = 0; i < 3; ++i) {
        if (over(outs[i], out_b[i], x, x_b) || over(outs[i], out_b[i], dt, dt_b) || over(outs[i], out_b[i], Bm, b_b) ||
            over(outs[i], out_b[i], Cm, c_b) || (i != 1 && over(outs[i], out_b[i], state_in, st_b)))
            return fail(GDN_ERR_INVALID_ARGUMENT, "%s: an output overlaps an input", fn);
        if (over(outs[i], out_b[i], A, H * 4) || over(outs[i], out_b[i], D, H * 4) ||
            over(outs[i], out_b[i], dt_bias, H * 4) || over(outs[i], out_b[i], lengths, B * 4))
            return fail(GDN_ERR_INVALID_ARGUMENT, "%s: an output overlaps A, D, dt_bias or lengths", fn);
        for (int j = 0; j < i; ++j)
            if (over(outs[i], out_b[i], outs[j], out_b[j]))
                return fail(GDN_ERR_INVALID_ARGUMENT, "%s: two outputs overlap", fn);
    }

    if (take_forced_failure()) return forced_failure(fn);
    cudaError_t e;
    const int sms = current_sm_count(&e);
    if (e != cudaSuccess) return cuda_fail(fn, "device query", e);
    gdn::ScanArgs a{};
    a.x = x;
    a.dt = dt;
    a.Bm = Bm;
    a.Cm = Cm;
    a.A = A;
    a.D = D;
    a.dt_bias = dt_bias;
    a.state_in = state_in;
    a.lengths = lengths;
    a.y = y;
    a.state_out = state_out;
    a.workspace = static_cast<float *>(workspace);
    a.B = B;
    a.T = T;
    a.H = H;
    a.P = P;
    a.G = G;
    a.x_sb = st.x_b;
    a.x_st = st.x_t;
    a.dt_sb = st.dt_b;
    a.dt_st = st.dt_t;
    a.b_sb = st.B_b;
    a.b_st = st.B_t;
    a.c_sb = st.C_b;
    a.c_st = st.C_t;
    a.N = (int)N;
    a.softplus = softplus != 0;
    a.vec_bc = aligned(Bm, 16) && aligned(Cm, 16) && (T == 1 || (st.B_t * eb % 16 == 0 && st.C_t * eb % 16 == 0)) &&
               (B == 1 || (st.B_b * eb % 16 == 0 && st.C_b * eb % 16 == 0));
    a.vec_x = aligned(x, 16) && P * eb % 16 == 0 && (T == 1 || st.x_t * eb % 16 == 0) &&
              (B == 1 || st.x_b * eb % 16 == 0);
    a.chunked = chunked;
    a.segments = plan.segments;
    a.seg_steps = plan.seg_steps;
    e = gdn::launch_selective_scan(static_cast<gdn::DType>(dtype), a, sms, reinterpret_cast<cudaStream_t>(stream));
    if (e == cudaErrorInvalidConfiguration) return fail(GDN_ERR_INVALID_ARGUMENT, "%s: grid too large", fn);
    if (e != cudaSuccess) return cuda_fail(fn, "launch", e);
    return ok();
}

gdn_status gdn_gated_norm(const void *x, const void *weight, const void *gate, const void *residual, void *y,
                          void *residual_out, int64_t M, int64_t K, int64_t D, int64_t x_stride_m,
                          int64_t gate_stride_m, int64_t weight_rows, int gate_first, float residual_scale, float eps,
                          gdn_dtype dtype, gdn_stream_t stream) {
    const char *fn = "gdn_gated_norm";
    const int eb = elem_bytes(dtype);
    if (eb == 0) return fail(GDN_ERR_UNSUPPORTED, "%s: unknown dtype %d", fn, (int)dtype);
    if (M <= 0 || K <= 0 || D <= 0) return fail(GDN_ERR_INVALID_ARGUMENT, "%s: M, K, D must all be > 0", fn);
    if (weight_rows != 1 && weight_rows != K)
        return fail(GDN_ERR_INVALID_ARGUMENT, "%s: weight_rows (%lld) must be 1 or K (%lld)", fn,
                    (long long)weight_rows, (long long)K);
    if (!(eps >= 0.f) || std::isinf(eps)) return fail(GDN_ERR_INVALID_ARGUMENT, "%s: eps must be finite and >= 0", fn);
    if (!x || !weight || !y) return fail(GDN_ERR_INVALID_ARGUMENT, "%s: x, weight and y must be non-NULL", fn);
    if ((residual == nullptr) != (residual_out == nullptr))
        return fail(GDN_ERR_INVALID_ARGUMENT, "%s: residual and residual_out go together", fn);
    const int64_t n_b = nbytes({M, K, D}, eb), w_b = nbytes({weight_rows, D}, eb);
    if (n_b < 0) return fail(GDN_ERR_INVALID_ARGUMENT, "%s: tensor sizes overflow int64", fn);
    const int64_t x_b = scaled(extent(1, 0, M, x_stride_m, K * D), eb);
    const int64_t g_b = gate ? scaled(extent(1, 0, M, gate_stride_m, K * D), eb) : 0;
    if (x_b < 0 || g_b < 0)
        return fail(GDN_ERR_INVALID_ARGUMENT, "%s: a token stride overlaps its rows or overflows", fn);
    for (const void *p : {x, weight, gate, residual, (const void *)y, (const void *)residual_out})
        if (!aligned(p, eb)) return fail(GDN_ERR_MISALIGNED, "%s: a tensor is not aligned to its element size", fn);
    const bool x_dense = M == 1 || x_stride_m == K * D, g_dense = M == 1 || gate_stride_m == K * D;
    // an output may be an input's own dense buffer (each element is read
    // before it is written, by the thread that writes it)
    for (const void *o : {(const void *)y, (const void *)residual_out}) {
        if (over(o, n_b, weight, w_b) || (over(o, n_b, x, x_b) && !(o == x && x_dense)) ||
            (over(o, n_b, gate, g_b) && !(o == gate && g_dense)) || (over(o, n_b, residual, n_b) && o != residual))
            return fail(GDN_ERR_INVALID_ARGUMENT, "%s: an output overlaps an input without being the same buffer", fn);
    }
    if (over(y, n_b, residual_out, n_b)) return fail(GDN_ERR_INVALID_ARGUMENT, "%s: y and residual_out overlap", fn);

    if (take_forced_failure()) return forced_failure(fn);
    cudaError_t e;
    const int sms = current_sm_count(&e);
    if (e != cudaSuccess) return cuda_fail(fn, "device query", e);
    gdn::NormArgs a{};
    a.x = x;
    a.weight = weight;
    a.gate = gate;
    a.residual = residual;
    a.y = y;
    a.residual_out = residual_out;
    a.M = M;
    a.K = K;
    a.D = D;
    a.x_st = x_stride_m;
    a.gate_st = gate_stride_m;
    a.weight_rows = weight_rows;
    a.scale = residual_scale;
    a.eps = eps;
    a.gate_first = gate_first != 0;
    const bool bases = aligned(x, 16) && aligned(weight, 16) && aligned(gate, 16) && aligned(residual, 16) &&
                       aligned(y, 16) && aligned(residual_out, 16);
    a.vec = bases && D * eb % 16 == 0 && (M == 1 || x_stride_m * eb % 16 == 0) &&
            (!gate || M == 1 || gate_stride_m * eb % 16 == 0);
    a.shift = bases && !a.vec && x_dense && (!gate || g_dense);
    const auto launch = dtype == GDN_DTYPE_F32    ? gdn::launch_norm_f32
                        : dtype == GDN_DTYPE_BF16 ? gdn::launch_norm_bf16
                                                  : gdn::launch_norm_f16;
    e = launch(a, sms, reinterpret_cast<cudaStream_t>(stream));
    if (e == cudaErrorInvalidConfiguration) return fail(GDN_ERR_INVALID_ARGUMENT, "%s: grid too large", fn);
    if (e != cudaSuccess) return cuda_fail(fn, "launch", e);
    return ok();
}

gdn_status gdn_sample(const void *logits, const float *noise, const float *temperature, const int32_t *top_k,
                      const float *top_p, const float *min_p, float temperature_all, int32_t top_k_all,
                      float top_p_all, float min_p_all, int32_t *token, float *logprob, int64_t R, int64_t V,
                      int64_t logits_stride, int64_t noise_stride, gdn_dtype dtype, gdn_stream_t stream) {
    const char *fn = "gdn_sample";
    const int eb = elem_bytes(dtype);
    if (eb == 0) return fail(GDN_ERR_UNSUPPORTED, "%s: unknown dtype %d", fn, (int)dtype);
    if (R <= 0 || V <= 0) return fail(GDN_ERR_INVALID_ARGUMENT, "%s: R and V must be > 0", fn);
    if (V > (1 << 22)) return fail(GDN_ERR_UNSUPPORTED, "%s: V (%lld) must be at most 2^22", fn, (long long)V);
    if (!logits || !noise || !token)
        return fail(GDN_ERR_INVALID_ARGUMENT, "%s: logits, noise and token must be non-NULL", fn);
    const int64_t l_b = scaled(extent(1, 0, R, logits_stride, V), eb), n_b = scaled(extent(1, 0, R, noise_stride, V), 4);
    if (l_b < 0 || n_b < 0) return fail(GDN_ERR_INVALID_ARGUMENT, "%s: a row stride is below V or overflows", fn);
    if (!aligned(logits, eb)) return fail(GDN_ERR_MISALIGNED, "%s: logits are not aligned to their element size", fn);
    for (const void *p : {(const void *)noise, (const void *)temperature, (const void *)top_k, (const void *)top_p,
                          (const void *)min_p, (const void *)token, (const void *)logprob})
        if (!aligned(p, 4)) return fail(GDN_ERR_MISALIGNED, "%s: a tensor is not aligned to its element size", fn);
    for (const void *o : {(const void *)token, (const void *)logprob})
        if (over(o, R * 4, logits, l_b) || over(o, R * 4, noise, n_b) || over(o, R * 4, temperature, R * 4) ||
            over(o, R * 4, top_k, R * 4) || over(o, R * 4, top_p, R * 4) || over(o, R * 4, min_p, R * 4))
            return fail(GDN_ERR_INVALID_ARGUMENT, "%s: an output overlaps an input", fn);
    if (over(token, R * 4, logprob, R * 4)) return fail(GDN_ERR_INVALID_ARGUMENT, "%s: token and logprob overlap", fn);

    if (take_forced_failure()) return forced_failure(fn);
    cudaError_t e;
    const int sms = current_sm_count(&e);
    if (e != cudaSuccess) return cuda_fail(fn, "device query", e);
    gdn::SampleArgs a{};
    a.logits = logits;
    a.noise = noise;
    a.temperature = temperature;
    a.top_k = top_k;
    a.top_p = top_p;
    a.min_p = min_p;
    a.temperature_v = temperature_all;
    a.top_k_v = top_k_all;
    a.top_p_v = top_p_all;
    a.min_p_v = min_p_all;
    a.token = token;
    a.logprob = logprob;
    a.R = R;
    a.V = V;
    a.logits_st = logits_stride;
    a.noise_st = noise_stride;
    e = gdn::launch_sample(static_cast<gdn::DType>(dtype), a, sms, reinterpret_cast<cudaStream_t>(stream));
    if (e == cudaErrorInvalidConfiguration) return fail(GDN_ERR_INVALID_ARGUMENT, "%s: grid too large", fn);
    if (e != cudaSuccess) return cuda_fail(fn, "launch", e);
    return ok();
}

}  // extern "C"
