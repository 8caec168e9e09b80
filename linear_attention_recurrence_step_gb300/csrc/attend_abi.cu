// attend_abi.cu -- C entry points of the operators of an attention layer
// (declared in include/gdn.h): argument checks and dispatch.  Checks run on
// the host, before any CUDA call, under the rules of abi.cu.
#include <algorithm>
#include <cmath>
#include <utility>

#include "abi_util.h"
#include "attend.h"

using namespace gdn::abi;

namespace {

struct Tensor {
    const void *p;
    int64_t bytes;
};

// Whether any of the outputs lies on another tensor of the call.
bool clash(std::initializer_list<Tensor> outputs, std::initializer_list<Tensor> inputs) {
    for (const Tensor *o = outputs.begin(); o != outputs.end(); ++o) {
        for (const Tensor *n = o + 1; n != outputs.end(); ++n)
            if (over(o->p, o->bytes, n->p, n->bytes)) return true;
        for (const Tensor &i : inputs)
            if (over(o->p, o->bytes, i.p, i.bytes)) return true;
    }
    return false;
}
// An output on its input: the same buffer or apart from it.
bool apart_or_same(const void *o, const void *i, int64_t bytes) { return o == i || !over(o, bytes, i, bytes); }

// Whether two [B,T,row] tensors of elements of `eb` bytes are slices of the same wider
// rows, apart from one another: same strides, and a row of both, one behind the other,
// still does not reach the next one.
bool slices(const void *p, int64_t sb_p, int64_t st_p, int64_t row_p, const void *q, int64_t sb_q, int64_t st_q,
            int64_t row_q, int64_t B, int64_t T, int eb) {
    if ((B > 1 && sb_p != sb_q) || (T > 1 && st_p != st_q)) return false;
    const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q), d = a < b ? b - a : a - b;
    const int64_t apart = (int64_t)(d / eb), first = a < b ? row_p : row_q, second = a < b ? row_q : row_p;
    return d % eb == 0 && apart >= first && apart <= INT64_MAX - second &&
           extent(B, sb_p, T, st_p, apart + second) >= 0;
}

int shift_of(int64_t page) {
    int s = 0;
    while (((int64_t)1 << s) < page) ++s;
    return s;
}
bool page_ok(int64_t page) { return page == 16 || page == 32 || page == 64 || page == 128; }
bool head_ok(int64_t D) { return D == 64 || D == 128 || D == 256; }

// Tokens of a sequence: places counted in tiles do not pass 31 bits.
constexpr int64_t kMaxRow = INT32_MAX - 4096;

// The sizes of a cache that slots of int32 can name, in bytes, or -1.
int64_t cache_bytes(int64_t pages, int64_t H, int64_t page, int64_t D) {
    int64_t slots;
    if (!mul_ok(pages, page, &slots) || slots > INT32_MAX || H > 65535) return -1;
    return nbytes({pages, H}, gdn::kv_block_bytes(page, D));
}

gdn_status launched(const char *fn, cudaError_t e) {
    if (e == cudaErrorInvalidConfiguration) return fail(GDN_ERR_INVALID_ARGUMENT, "%s: grid too large", fn);
    if (e != cudaSuccess) return cuda_fail(fn, "launch", e);
    return ok();
}

// What gdn_kv_append and gdn_kv_read share.
gdn_status check_kv(const char *fn, const void *cache, const int32_t *slots, const float *k_scale,
                    const float *v_scale, int64_t tokens, int64_t H, int64_t D, int64_t page, int64_t pages,
                    int64_t *bytes) {
    if (tokens <= 0 || H <= 0 || D <= 0 || page <= 0 || pages <= 0)
        return fail(GDN_ERR_INVALID_ARGUMENT, "%s: every size must be > 0", fn);
    if (!head_ok(D)) return fail(GDN_ERR_UNSUPPORTED, "%s: D (%lld) must be 64, 128 or 256", fn, (long long)D);
    if (!page_ok(page))
        return fail(GDN_ERR_UNSUPPORTED, "%s: page (%lld) must be 16, 32, 64 or 128", fn, (long long)page);
    if (!cache || !slots) return fail(GDN_ERR_INVALID_ARGUMENT, "%s: cache and slots must be non-NULL", fn);
    *bytes = cache_bytes(pages, H, page, D);
    if (*bytes < 0)
        return fail(GDN_ERR_INVALID_ARGUMENT, "%s: the cache's sizes overflow (2^31 - 1 slots, 65535 heads)", fn);
    if (!aligned(cache, 16)) return fail(GDN_ERR_MISALIGNED, "%s: cache must be 16-byte aligned", fn);
    if (!aligned(slots, 4) || !aligned(k_scale, 4) || !aligned(v_scale, 4))
        return fail(GDN_ERR_MISALIGNED, "%s: slots, k_scale and v_scale must be 4-byte aligned", fn);
    return GDN_OK;
}

}  // namespace

extern "C" {

gdn_status gdn_page_slots(const int32_t *lengths, const int32_t *add, const int32_t *held, const int32_t *ring_state,
                          int32_t *block_table, int32_t *ring, int32_t *slots, int32_t *positions, int32_t *granted,
                          int32_t *lengths_out, int32_t *held_out, int32_t *ring_state_out, int64_t B, int64_t T,
                          int64_t width, int64_t pages, int64_t page, gdn_stream_t stream) {
    const char *fn = "gdn_page_slots";
    if (B <= 0 || T <= 0 || width <= 0 || pages <= 0 || page <= 0)
        return fail(GDN_ERR_INVALID_ARGUMENT, "%s: B, T, width, pages, page must all be > 0", fn);
    if (!page_ok(page))
        return fail(GDN_ERR_UNSUPPORTED, "%s: page (%lld) must be 16, 32, 64 or 128", fn, (long long)page);
    for (const void *p : {(const void *)lengths, (const void *)held, (const void *)ring_state,
                          (const void *)block_table, (const void *)ring, (const void *)slots, (const void *)positions,
                          (const void *)granted, (const void *)lengths_out, (const void *)held_out,
                          (const void *)ring_state_out})
        if (!p) return fail(GDN_ERR_INVALID_ARGUMENT, "%s: only add may be NULL", fn);
    for (const void *p : {(const void *)lengths, (const void *)add, (const void *)held, (const void *)ring_state,
                          (const void *)block_table, (const void *)ring, (const void *)slots, (const void *)positions,
                          (const void *)granted, (const void *)lengths_out, (const void *)held_out,
                          (const void *)ring_state_out})
        if (!aligned(p, 4)) return fail(GDN_ERR_MISALIGNED, "%s: a tensor is not 4-byte aligned", fn);
    const int64_t b_b = nbytes({B}, 4), bt_b = nbytes({B, T}, 4), table_b = nbytes({B, width}, 4);
    int64_t slots_all, row_all;
    if (b_b < 0 || bt_b < 0 || table_b < 0 || !mul_ok(pages, page, &slots_all) || slots_all > INT32_MAX ||
        !mul_ok(width, page, &row_all) || row_all > kMaxRow || T > kMaxRow || B > INT32_MAX)
        return fail(GDN_ERR_INVALID_ARGUMENT, "%s: sizes overflow (pages * page and width * page fit int32)", fn);
    const int64_t ring_b = pages * 4;
    if (!apart_or_same(lengths_out, lengths, b_b) || !apart_or_same(held_out, held, b_b) ||
        !apart_or_same(ring_state_out, ring_state, 8))
        return fail(GDN_ERR_INVALID_ARGUMENT, "%s: an output overlaps its input without being the same buffer", fn);
    if (clash({{block_table, table_b}, {ring, ring_b}, {slots, bt_b}, {positions, bt_b}, {granted, b_b},
               {lengths_out, b_b}, {held_out, b_b}, {ring_state_out, 8}},
              {{add, b_b}}) ||
        clash({{block_table, table_b}, {ring, ring_b}, {slots, bt_b}, {positions, bt_b}, {granted, b_b}},
              {{lengths, b_b}, {held, b_b}, {ring_state, 8}}) ||
        over(lengths_out, b_b, held, b_b) || over(lengths_out, b_b, ring_state, 8) ||
        over(held_out, b_b, lengths, b_b) || over(held_out, b_b, ring_state, 8) ||
        over(ring_state_out, 8, lengths, b_b) || over(ring_state_out, 8, held, b_b))
        return fail(GDN_ERR_INVALID_ARGUMENT, "%s: an output overlaps another tensor", fn);

    if (take_forced_failure()) return forced_failure(fn);
    gdn::SlotsArgs a{};
    a.lengths = lengths;
    a.add = add;
    a.held = held;
    a.ring_state = ring_state;
    a.table = block_table;
    a.ring = ring;
    a.slots = slots;
    a.positions = positions;
    a.granted = granted;
    a.lengths_out = lengths_out;
    a.held_out = held_out;
    a.ring_state_out = ring_state_out;
    a.B = B;
    a.T = T;
    a.width = (int)width;
    a.pages = (int)pages;
    a.page_shift = shift_of(page);
    return launched(fn, gdn::launch_page_slots(a, reinterpret_cast<cudaStream_t>(stream)));
}

gdn_status gdn_rotary(const void *q, const void *k, const int32_t *positions, const float *inv_freq, void *q_out,
                      void *k_out, int64_t B, int64_t T, int64_t Hq, int64_t Hk, int64_t D, int64_t R,
                      const gdn_rotary_strides *strides, gdn_rotary_layout layout, float scale, int inverse,
                      gdn_dtype dtype, gdn_stream_t stream) {
    const char *fn = "gdn_rotary";
    const int eb = elem_bytes(dtype);
    if (eb == 0) return fail(GDN_ERR_UNSUPPORTED, "%s: unknown dtype %d", fn, (int)dtype);
    if (B <= 0 || T <= 0 || Hq <= 0 || D <= 0 || R <= 0 || (k && Hk <= 0))
        return fail(GDN_ERR_INVALID_ARGUMENT, "%s: B, T, Hq, Hk, D, R must all be > 0", fn);
    if (R % 2 != 0 || R > D)
        return fail(GDN_ERR_INVALID_ARGUMENT, "%s: R (%lld) must be even and at most D (%lld)", fn, (long long)R,
                    (long long)D);
    if (layout != GDN_ROTARY_HALF && layout != GDN_ROTARY_INTERLEAVED)
        return fail(GDN_ERR_INVALID_ARGUMENT, "%s: unknown layout %d", fn, (int)layout);
    if (!q || !q_out || !positions || !inv_freq || !k != !k_out)
        return fail(GDN_ERR_INVALID_ARGUMENT, "%s: a tensor is NULL (k and k_out only together)", fn);
    if (!k) Hk = 0;
    // (a quarter of 2^31, so that four tokens' elements still count in 31 bits)
    int64_t row;
    if (!mul_ok(Hq + Hk, D, &row) || Hq > INT32_MAX || Hk > INT32_MAX || row > (INT32_MAX >> 2) || R / 2 > 4096)
        return fail(R / 2 > 4096 ? GDN_ERR_UNSUPPORTED : GDN_ERR_INVALID_ARGUMENT,
                    "%s: heads of a token overflow, or R (%lld) is above 8192", fn, (long long)R);
    const int64_t qd = Hq * D, kd = Hk * D;
    gdn_rotary_strides st{T * qd, qd, T * kd, kd, T * qd, qd, T * kd, kd};
    if (strides) st = *strides;
    const int64_t q_b = scaled(extent(B, st.q_b, T, st.q_t, qd), eb), qo_b = scaled(extent(B, st.q_out_b, T, st.q_out_t, qd), eb);
    const int64_t k_b = k ? scaled(extent(B, st.k_b, T, st.k_t, kd), eb) : 0;
    const int64_t ko_b = k ? scaled(extent(B, st.k_out_b, T, st.k_out_t, kd), eb) : 0;
    const int64_t bt_b = nbytes({B, T}, 4);
    if (nbytes({B, T, qd + kd}, eb) < 0 || bt_b < 0)
        return fail(GDN_ERR_INVALID_ARGUMENT, "%s: tensor sizes overflow int64", fn);
    if (q_b < 0 || qo_b < 0 || k_b < 0 || ko_b < 0)
        return fail(GDN_ERR_INVALID_ARGUMENT, "%s: strides overlap a tensor's rows or overflow", fn);
    for (const void *p : {q, k, (const void *)q_out, (const void *)k_out})
        if (!aligned(p, eb)) return fail(GDN_ERR_MISALIGNED, "%s: a tensor is not aligned to its element size", fn);
    if (!aligned(positions, 4) || !aligned(inv_freq, 4))
        return fail(GDN_ERR_MISALIGNED, "%s: positions and inv_freq must be 4-byte aligned", fn);
    // An output lies on its input's own rows (in place) or apart from it; on the other
    // input only where it is in place and the two are slices of the same rows (a block
    // writes its rows of the one while others read theirs of the other); on the other
    // output as slices of the same rows.
    const bool q_in = q_out == q && st.q_out_b == st.q_b && st.q_out_t == st.q_t;
    const bool k_in = k && k_out == k && st.k_out_b == st.k_b && st.k_out_t == st.k_t;
    if ((!q_in && over(q_out, qo_b, q, q_b)) || (!k_in && over(k_out, ko_b, k, k_b)) ||
        (over(q_out, qo_b, k, k_b) &&
         !(q_in && slices(q, st.q_b, st.q_t, qd, k, st.k_b, st.k_t, kd, B, T, eb))) ||
        (over(k_out, ko_b, q, q_b) &&
         !(k_in && slices(k, st.k_b, st.k_t, kd, q, st.q_b, st.q_t, qd, B, T, eb))) ||
        (over(q_out, qo_b, k_out, ko_b) &&
         !slices(q_out, st.q_out_b, st.q_out_t, qd, k_out, st.k_out_b, st.k_out_t, kd, B, T, eb)))
        return fail(GDN_ERR_INVALID_ARGUMENT, "%s: an output overlaps another tensor without being in place", fn);
    for (const auto &[o, o_b] : {std::pair<const void *, int64_t>(q_out, qo_b), {k_out, ko_b}})
        if (over(o, o_b, positions, bt_b) || over(o, o_b, inv_freq, R * 2))
            return fail(GDN_ERR_INVALID_ARGUMENT, "%s: an output overlaps positions or inv_freq", fn);

    if (take_forced_failure()) return forced_failure(fn);
    cudaError_t e;
    const int sms = current_sm_count(&e);
    if (e != cudaSuccess) return cuda_fail(fn, "device query", e);
    gdn::RotaryArgs a{};
    a.q = q;
    a.k = k;
    a.positions = positions;
    a.inv_freq = inv_freq;
    a.q_out = q_out;
    a.k_out = k_out;
    a.B = B;
    a.T = T;
    a.Hq = (int)Hq;
    a.Hk = (int)Hk;
    a.D = (int)D;
    a.R = (int)R;
    a.q_sb = st.q_b;
    a.q_st = st.q_t;
    a.k_sb = st.k_b;
    a.k_st = st.k_t;
    a.qo_sb = st.q_out_b;
    a.qo_st = st.q_out_t;
    a.ko_sb = st.k_out_b;
    a.ko_st = st.k_out_t;
    a.scale = scale;
    a.half = layout == GDN_ROTARY_HALF;
    a.inverse = inverse != 0;
    const int64_t vec = 16 / eb;
    auto rows16 = [&](const void *p, int64_t sb, int64_t s_t) {
        return !p || (aligned(p, 16) && (B == 1 || sb % vec == 0) && (T == 1 || s_t % vec == 0));
    };
    a.vec = D % vec == 0 && R % (a.half ? 2 * vec : vec) == 0 && rows16(q, st.q_b, st.q_t) &&
            rows16(k, st.k_b, st.k_t) && rows16(q_out, st.q_out_b, st.q_out_t) && rows16(k_out, st.k_out_b, st.k_out_t);
    return launched(fn, gdn::launch_rotary(static_cast<gdn::DType>(dtype), a, sms, reinterpret_cast<cudaStream_t>(stream)));
}

gdn_status gdn_kv_append(const void *k, const void *v, const int32_t *slots, void *cache, const float *k_scale,
                         const float *v_scale, int64_t B, int64_t T, int64_t H, int64_t D, int64_t page, int64_t pages,
                         int64_t k_stride_b, int64_t k_stride_t, int64_t v_stride_b, int64_t v_stride_t,
                         gdn_dtype dtype, gdn_stream_t stream) {
    const char *fn = "gdn_kv_append";
    const int eb = elem_bytes(dtype);
    if (eb == 0) return fail(GDN_ERR_UNSUPPORTED, "%s: unknown dtype %d", fn, (int)dtype);
    if (B <= 0 || T <= 0) return fail(GDN_ERR_INVALID_ARGUMENT, "%s: every size must be > 0", fn);
    int64_t tokens, c_b;
    if (!mul_ok(B, T, &tokens)) return fail(GDN_ERR_INVALID_ARGUMENT, "%s: tensor sizes overflow int64", fn);
    const gdn_status st = check_kv(fn, cache, slots, k_scale, v_scale, tokens, H, D, page, pages, &c_b);
    if (st != GDN_OK) return st;
    if (!k || !v) return fail(GDN_ERR_INVALID_ARGUMENT, "%s: k and v must be non-NULL", fn);
    if (nbytes({B, T, H, D}, 2 * eb) < 0)
        return fail(GDN_ERR_INVALID_ARGUMENT, "%s: tensor sizes overflow int64", fn);
    const int64_t k_b = scaled(extent(B, k_stride_b, T, k_stride_t, H * D), eb);
    const int64_t v_b = scaled(extent(B, v_stride_b, T, v_stride_t, H * D), eb);
    if (k_b < 0 || v_b < 0)
        return fail(GDN_ERR_INVALID_ARGUMENT, "%s: strides of k or v overlap their rows or overflow", fn);
    if (!aligned(k, eb) || !aligned(v, eb))
        return fail(GDN_ERR_MISALIGNED, "%s: a tensor is not aligned to its element size", fn);
    if (clash({{cache, c_b}}, {{k, k_b}, {v, v_b}, {slots, tokens * 4}, {k_scale, H * 4}, {v_scale, H * 4}}))
        return fail(GDN_ERR_INVALID_ARGUMENT, "%s: the cache overlaps another tensor", fn);

    if (take_forced_failure()) return forced_failure(fn);
    gdn::KvArgs a{};
    a.k_in = k;
    a.v_in = v;
    a.slots = slots;
    a.k_scale = k_scale;
    a.v_scale = v_scale;
    a.cache = static_cast<unsigned char *>(cache);
    a.B = B;
    a.T = T;
    a.pages = pages;
    a.H = (int)H;
    a.D = (int)D;
    a.page_shift = shift_of(page);
    a.k_sb = k_stride_b;
    a.k_st = k_stride_t;
    a.v_sb = v_stride_b;
    a.v_st = v_stride_t;
    const int64_t vec = 16 / eb;
    a.vec = aligned(k, 16) && aligned(v, 16) &&
            (B == 1 || (k_stride_b % vec == 0 && v_stride_b % vec == 0)) &&
            (T == 1 || (k_stride_t % vec == 0 && v_stride_t % vec == 0));
    return launched(fn, gdn::launch_kv_append(static_cast<gdn::DType>(dtype), a, reinterpret_cast<cudaStream_t>(stream)));
}

gdn_status gdn_kv_read(const void *cache, const int32_t *slots, const float *k_scale, const float *v_scale, void *k,
                       void *v, int64_t N, int64_t H, int64_t D, int64_t page, int64_t pages, gdn_dtype dtype,
                       gdn_stream_t stream) {
    const char *fn = "gdn_kv_read";
    const int eb = elem_bytes(dtype);
    if (eb == 0) return fail(GDN_ERR_UNSUPPORTED, "%s: unknown dtype %d", fn, (int)dtype);
    int64_t c_b;
    const gdn_status st = check_kv(fn, cache, slots, k_scale, v_scale, N, H, D, page, pages, &c_b);
    if (st != GDN_OK) return st;
    if (!k || !v) return fail(GDN_ERR_INVALID_ARGUMENT, "%s: k and v must be non-NULL", fn);
    const int64_t o_b = nbytes({N, H, D}, eb);
    if (o_b < 0 || nbytes({N, H, D}, 2 * eb) < 0)
        return fail(GDN_ERR_INVALID_ARGUMENT, "%s: tensor sizes overflow int64", fn);
    if (!aligned(k, eb) || !aligned(v, eb))
        return fail(GDN_ERR_MISALIGNED, "%s: a tensor is not aligned to its element size", fn);
    if (clash({{k, o_b}, {v, o_b}}, {{cache, c_b}, {slots, N * 4}, {k_scale, H * 4}, {v_scale, H * 4}}))
        return fail(GDN_ERR_INVALID_ARGUMENT, "%s: an output overlaps another tensor", fn);

    if (take_forced_failure()) return forced_failure(fn);
    gdn::KvArgs a{};
    a.k_out = k;
    a.v_out = v;
    a.slots = slots;
    a.k_scale = k_scale;
    a.v_scale = v_scale;
    a.cache = const_cast<unsigned char *>(static_cast<const unsigned char *>(cache));
    a.B = 1;
    a.T = N;
    a.pages = pages;
    a.H = (int)H;
    a.D = (int)D;
    a.page_shift = shift_of(page);
    a.vec = aligned(k, 16) && aligned(v, 16);
    return launched(fn, gdn::launch_kv_read(static_cast<gdn::DType>(dtype), a, reinterpret_cast<cudaStream_t>(stream)));
}

size_t gdn_kv_attention_workspace_size(int64_t B, int64_t T, int64_t Hq, int64_t H, int64_t D) {
    if (B <= 0 || T <= 0 || Hq <= 0 || H <= 0 || Hq % H != 0 || !head_ok(D)) return 0;
    const int64_t n = gdn::attend_workspace_bytes(B, T, Hq, H, D);
    return n < 0 ? 0 : (size_t)std::max<int64_t>(n, 16);
}

gdn_status gdn_kv_attention(const void *q, const void *cache, const int32_t *block_table, const int32_t *lengths,
                            const int32_t *fresh, const float *k_scale, const float *v_scale, void *y, float *lse,
                            int64_t B, int64_t T, int64_t Hq, int64_t H, int64_t D, int64_t width, int64_t page,
                            int64_t pages, int64_t q_stride_b, int64_t q_stride_t, float scale, int64_t window,
                            void *workspace, size_t workspace_bytes, gdn_dtype dtype, gdn_stream_t stream) {
    const char *fn = "gdn_kv_attention";
    const int eb = elem_bytes(dtype);
    if (eb == 0) return fail(GDN_ERR_UNSUPPORTED, "%s: unknown dtype %d", fn, (int)dtype);
    if (B <= 0 || T <= 0 || Hq <= 0 || H <= 0 || D <= 0 || width <= 0 || page <= 0 || pages <= 0)
        return fail(GDN_ERR_INVALID_ARGUMENT, "%s: every size must be > 0", fn);
    if (Hq % H != 0)
        return fail(GDN_ERR_INVALID_ARGUMENT, "%s: Hq (%lld) must be a multiple of H (%lld)", fn, (long long)Hq,
                    (long long)H);
    if (!head_ok(D)) return fail(GDN_ERR_UNSUPPORTED, "%s: D (%lld) must be 64, 128 or 256", fn, (long long)D);
    if (!page_ok(page))
        return fail(GDN_ERR_UNSUPPORTED, "%s: page (%lld) must be 16, 32, 64 or 128", fn, (long long)page);
    if (window < 0 || window > INT32_MAX)
        return fail(GDN_ERR_INVALID_ARGUMENT, "%s: window (%lld) must be 0 (none) to 2^31 - 1", fn, (long long)window);
    if (!q || !cache || !block_table || !lengths || !y)
        return fail(GDN_ERR_INVALID_ARGUMENT, "%s: q, cache, block_table, lengths and y must be non-NULL", fn);
    if (!std::isfinite(scale)) return fail(GDN_ERR_INVALID_ARGUMENT, "%s: scale must be finite", fn);
    const int64_t y_b = nbytes({B, T, Hq, D}, eb), l_b = nbytes({B, T, Hq}, 4), t_b = nbytes({B, width}, 4);
    const int64_t c_b = cache_bytes(pages, H, page, D);
    int64_t row_all;
    if (y_b < 0 || l_b < 0 || t_b < 0 || c_b < 0 || !mul_ok(width, page, &row_all) || row_all > kMaxRow ||
        B > INT32_MAX || gdn::attend_workspace_bytes(B, T, Hq, H, D) < 0)
        return fail(GDN_ERR_INVALID_ARGUMENT,
                    "%s: sizes overflow (pages * page, width * page and the query rows fit int32, H 16 bits)", fn);
    const int64_t q_b = scaled(extent(B, q_stride_b, T, q_stride_t, Hq * D), eb);
    if (q_b < 0) return fail(GDN_ERR_INVALID_ARGUMENT, "%s: strides of q overlap its rows or overflow", fn);
    if (!aligned(q, eb) || !aligned(y, eb))
        return fail(GDN_ERR_MISALIGNED, "%s: a tensor is not aligned to its element size", fn);
    if (!aligned(block_table, 4) || !aligned(lengths, 4) || !aligned(fresh, 4) || !aligned(k_scale, 4) ||
        !aligned(v_scale, 4) || !aligned(lse, 4))
        return fail(GDN_ERR_MISALIGNED, "%s: block_table, lengths, new, the scales and lse must be 4-byte aligned", fn);
    const size_t need = gdn_kv_attention_workspace_size(B, T, Hq, H, D);
    const bool ws = need > 16;
    if (ws && (!workspace || workspace_bytes < need))
        return fail(GDN_ERR_INVALID_ARGUMENT, "%s: workspace of %zu bytes needed, %zu given", fn, need,
                    workspace ? workspace_bytes : 0);
    if (!aligned(cache, 16) || (ws && !aligned(workspace, 16)))
        return fail(GDN_ERR_MISALIGNED, "%s: cache and workspace must be 16-byte aligned", fn);
    if (clash({{y, y_b}, {lse, l_b}, {ws ? workspace : nullptr, (int64_t)need}},
              {{q, q_b}, {cache, c_b}, {block_table, t_b}, {lengths, B * 4}, {fresh, B * 4}, {k_scale, H * 4},
               {v_scale, H * 4}}))
        return fail(GDN_ERR_INVALID_ARGUMENT, "%s: an output or the workspace overlaps another tensor", fn);

    if (take_forced_failure()) return forced_failure(fn);
    gdn::AttendArgs a{};
    a.q = q;
    a.cache = static_cast<const unsigned char *>(cache);
    a.table = block_table;
    a.lengths = lengths;
    a.fresh = fresh;
    a.k_scale = k_scale;
    a.v_scale = v_scale;
    a.y = y;
    a.lse = lse;
    a.workspace = static_cast<float *>(workspace);
    a.B = B;
    a.T = T;
    a.pages = pages;
    a.q_sb = q_stride_b;
    a.q_st = q_stride_t;
    a.Hq = (int)Hq;
    a.H = (int)H;
    a.D = (int)D;
    a.width = (int)width;
    a.page_shift = shift_of(page);
    a.scale = scale;
    a.window = (int)window;
    a.vec_y = aligned(y, 16);
    const int64_t vec = 16 / eb;
    a.vec_q = aligned(q, 16) && (B == 1 || q_stride_b % vec == 0) && (T == 1 || q_stride_t % vec == 0);
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const gdn::DType dt = static_cast<gdn::DType>(dtype);
    if (gdn::attend_takes_tc(dt, a)) return launched(fn, gdn::launch_attend_tc(dt, a, s));
    return launched(fn, dtype == GDN_DTYPE_F32    ? gdn::launch_attend_f32(a, s)
                        : dtype == GDN_DTYPE_BF16 ? gdn::launch_attend_bf16(a, s)
                                                  : gdn::launch_attend_f16(a, s));
}

}  // extern "C"
