// page_slots.cu -- block tables and slot maps from the requests' lengths.
//
// Sequence b needs n_b = max(0, ceil((len + add) / page) - held) further
// pages.  An inclusive sum of the n_b over the batch, in order, says which
// sequences are served (sum <= free pages) and where in the ring of free pages
// each one's begin; a second sum places the pages of sequences that end behind
// the ring's last.  The ring's live places are only read and the places behind
// them only written, so takers and givers need no order between them.
//
// The sums take one block (two barriers for 1024 sequences); what bounds a
// decode step is its chain of dependent loads (state, sums, ring, table): 4.1 us for
// 64 requests, 6.2 with 1024 threads for them.  Runs of pages go to a warp each, and
// a thread of the second kernel writes four tokens (64 prompts of up to 4096: 7.4 us,
// 18.6 with a thread per run and token).
#include "attend.h"
#include "common.cuh"

namespace gdn {

namespace {

constexpr int kSlotsThreads = 1024;
// Up to so many slots the block of the sums writes slots and positions too; beyond, a
// second kernel over the whole GPU does, and waits for the first: 2048 slots 6.4 us in
// one kernel, 6.6 in two; 4096 7.5 and 7.1; 8192 9.0 and 7.1; 65536 27 and 7.6.
constexpr int64_t kSlotsOneBlock = 2048;

struct Pair {
    int64_t need, back;
};

__device__ __forceinline__ Pair warp_scan(Pair v) {
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const int64_t n = __shfl_up_sync(0xffffffffu, v.need, d), k = __shfl_up_sync(0xffffffffu, v.back, d);
        if ((int)(threadIdx.x & 31) >= d) {
            v.need += n;
            v.back += k;
        }
    }
    return v;
}

__device__ __forceinline__ int ring_place(int64_t i, int pages) { return (int)(i % pages); }

// Slot and position of token t of a sequence; its pages are in the table.
__device__ __forceinline__ void put_token(const SlotsArgs &a, int64_t b, int64_t t, int first, int granted) {
    int slot = -1, pos = -1;
    if (t < granted) {
        pos = first + (int)t;
        const int p = a.table[b * a.width + (pos >> a.page_shift)];
        if (p >= 0 && p < a.pages) slot = (p << a.page_shift) + (pos & ((1 << a.page_shift) - 1));
    }
    a.slots[b * a.T + t] = slot;
    a.positions[b * a.T + t] = pos;
}

__global__ void __launch_bounds__(kSlotsThreads) slots_plan_kernel(const SlotsArgs a, bool tokens) {
    __shared__ Pair part[32];
    __shared__ int run[kSlotsThreads], run_at[kSlotsThreads], run_ring[kSlotsThreads];  // pages taken (or given back), where
    pdl_trigger();
    pdl_wait();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int page = 1 << a.page_shift;
    // (held in range whatever the caller's memory says)
    const int head = (int)(((int64_t)a.ring_state[0] % a.pages + a.pages) % a.pages);
    const int count = min(max(a.ring_state[1], 0), a.pages);
    Pair carry{0, 0};
    int64_t taken = 0;
    for (int64_t b0 = 0; b0 < a.B; b0 += blockDim.x) {
        const int64_t b = b0 + tid;
        int len = 0, add = 0, held = 0, more = 0, back = 0;
        bool ends = false, fits = false;
        if (b < a.B) {
            len = max(a.lengths[b], 0);
            held = min(max(a.held[b], 0), a.width);
            const int64_t want = a.add ? a.add[b] : a.T;
            ends = want < 0;
            add = (int)min(max(want, (int64_t)0), a.T);
            const int64_t total = (int64_t)len + add;
            fits = !ends && total <= ((int64_t)a.width << a.page_shift);
            if (fits) more = max((int)((total + page - 1) >> a.page_shift) - held, 0);
            if (ends) back = held;
        }
        Pair sum = warp_scan(Pair{more, back});
        if (lane == 31) part[warp] = sum;
        __syncthreads();
        if (warp == 0) {
            const Pair all = warp_scan(lane < (int)blockDim.x / 32 ? part[lane] : Pair{0, 0});
            part[lane] = all;
        }
        __syncthreads();
        if (warp > 0) {
            sum.need += part[warp - 1].need;
            sum.back += part[warp - 1].back;
        }
        sum.need += carry.need;
        sum.back += carry.back;
        const Pair total{carry.need + part[31].need, carry.back + part[31].back};
        const bool served = fits && (more == 0 || sum.need <= count);
        if (!served) more = 0;
        const int granted = served ? add : 0;
        int64_t from = sum.need - more;               // of the ring's free pages, from its head on
        int64_t to = (int64_t)count + sum.back - back;  // behind them
        if (b < a.B) {
            a.granted[b] = granted;
            a.lengths_out[b] = ends ? 0 : len + granted;
            a.held_out[b] = ends ? 0 : held + more;
        }
        // a sequence's page by its own thread, longer runs by a warp each
        int32_t *row = a.table + b * a.width;
        const bool runs = more > 1 || back > 0;
        if (more == 1) row[held] = a.ring[ring_place(head + from, a.pages)];
        if (runs) {
            run[tid] = more > 1 ? more : -back;
            run_at[tid] = more > 1 ? held : 0;
            run_ring[tid] = ring_place(head + (more > 1 ? from : to), a.pages);
            // (a ring that is full already takes no more)
            if (back > 0) run[tid] = -(int)max(min((int64_t)back, a.pages - to), (int64_t)0);
        } else {
            run[tid] = 0;
        }
        if (__syncthreads_or(runs)) {
            const int warps = (int)blockDim.x / 32, mine = run[warp + warps * lane];
            for (unsigned m = __ballot_sync(0xffffffffu, mine != 0); m; m &= m - 1) {
                const int q = warp + warps * (__ffs(m) - 1), n = run[q];
                int32_t *r = a.table + (b0 + q) * a.width + run_at[q];
                for (int i = lane; i < (n < 0 ? -n : n); i += 32) {
                    const int at = run_ring[q] + i, place = at < a.pages ? at : at - a.pages;
                    if (n > 0) r[i] = a.ring[place];
                    else a.ring[place] = r[i];
                }
            }
        }
        // the pages taken so far: the sum up to the last sequence that took one
        int64_t mine = more > 0 ? sum.need : 0;
#pragma unroll
        for (int d = 16; d; d /= 2) mine = max(mine, __shfl_xor_sync(0xffffffffu, mine, d));
        __syncthreads();
        if (lane == 0) part[warp].need = mine;
        __syncthreads();
        for (int w = 0; w < (int)blockDim.x / 32; ++w) taken = max(taken, part[w].need);
        carry = total;
        __syncthreads();
    }
    if (tid == 0) {
        a.ring_state_out[0] = ring_place(head + taken, a.pages);
        a.ring_state_out[1] = (int)min((int64_t)count - taken + carry.back, (int64_t)a.pages);
    }
    if (tokens)
        for (int64_t i = tid; i < a.B * a.T; i += blockDim.x) {
            const int64_t b = i / a.T;
            const int granted = a.granted[b];
            put_token(a, b, i - b * a.T, a.lengths_out[b] - granted, granted);
        }
}

// Four neighbouring tokens per thread; VECTOR: rows of whole int4.
template <bool VECTOR>
__global__ void __launch_bounds__(256) slots_tokens_kernel(const SlotsArgs a, int per_row) {
    pdl_trigger();
    pdl_wait();
    const int64_t b = blockIdx.x / per_row, t0 = ((int64_t)(blockIdx.x - b * per_row) * 256 + threadIdx.x) * 4;
    if (t0 >= a.T) return;
    const int granted = a.granted[b], first = a.lengths_out[b] - granted;
    int slot[4], pos[4], page = -1, entry = -1;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        slot[i] = pos[i] = -1;
        if (t0 + i < granted) {
            pos[i] = first + (int)t0 + i;
            if (pos[i] >> a.page_shift != page) {
                page = pos[i] >> a.page_shift;
                entry = a.table[b * a.width + page];
            }
            if (entry >= 0 && entry < a.pages) slot[i] = (entry << a.page_shift) + (pos[i] & ((1 << a.page_shift) - 1));
        }
    }
    const int64_t at = b * a.T + t0;
    if (VECTOR) {
        *reinterpret_cast<int4 *>(a.slots + at) = make_int4(slot[0], slot[1], slot[2], slot[3]);
        *reinterpret_cast<int4 *>(a.positions + at) = make_int4(pos[0], pos[1], pos[2], pos[3]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (t0 + i < a.T) {
                a.slots[at + i] = slot[i];
                a.positions[at + i] = pos[i];
            }
    }
}

}  // namespace

cudaError_t launch_page_slots(const SlotsArgs &a, cudaStream_t s) {
    const int64_t n = a.B * a.T;
    const bool one = n <= kSlotsOneBlock;
    const unsigned threads = a.B <= 256 && n <= 256 ? 256 : kSlotsThreads;
    cudaError_t e = launch_dependent(slots_plan_kernel, 1, threads, 0, s, a, one);
    if (e != cudaSuccess || one) return e;
    const int64_t per_row = (a.T + 1023) / 1024, blocks = a.B * per_row;
    if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
    const bool vec = a.T % 4 == 0 && ((reinterpret_cast<uintptr_t>(a.slots) | reinterpret_cast<uintptr_t>(a.positions)) & 15) == 0;
    return vec ? launch_dependent(slots_tokens_kernel<true>, (unsigned)blocks, 256, 0, s, a, (int)per_row)
               : launch_dependent(slots_tokens_kernel<false>, (unsigned)blocks, 256, 0, s, a, (int)per_row);
}

}  // namespace gdn
