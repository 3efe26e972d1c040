// slots.cuh — block tables and slot maps of a paged cache, built on the GPU
// from what a verify step leaves there.
//
// Before the scorer runs, every request needs a cache slot for each of the
// rows it will score (its last token and its drafts, or the nodes of its
// tree): position p of a request lies in slot table[p / bs] bs + p % bs.  The
// accepted length of the last verify step (vLLM page, section 1: a step gains
// the accepted drafts and one token) moves the sequence on; pages are granted
// from a ring of free pages in request order, and those of released requests
// go back to it.
//
// plan_tables_kernel: lengths, page counts, prefix sums of the pages asked
// for, the tables' new entries and the ring.  plan_slots_kernel: positions
// and slots of the rows.
#pragma once

#include <cuda_runtime.h>
#include <limits.h>
#include <stdint.h>

#include "device_utils.cuh"
#include "verify_common.cuh"

namespace specdec {

constexpr int kPlanThreads = 1024;

struct PlanParams {
    const int32_t* seq_lens;    // [B]
    const int32_t* accept_len;  // [B] or null
    const int32_t* release;     // [B] or null
    const int32_t* offsets;     // [B + 1] or null: k drafts per request
    int B, k;
    int64_t total;              // packed layout: drafts laid out
    int block_size;
    int32_t* tables;
    int64_t table_stride;
    int max_blocks;
    const int32_t* held;        // [B]
    int32_t* ring;
    int capacity;
    const int32_t* ring_state;  // [2] head, count
    int32_t* seq_out;
    int32_t* held_out;
    int32_t* ring_out;
    int64_t* positions;         // [rows]
    int64_t* slots;             // [rows]
};

struct PlanRows {
    int64_t row0;
    int64_t n;  // rows of the request; 0 where its offsets are invalid
};
__device__ __forceinline__ PlanRows plan_rows(const PlanParams& P, int64_t b) {
    PlanRows r;
    if (P.offsets == nullptr) {
        r.n = P.k + 1;
        r.row0 = b * r.n;
        return r;
    }
    const int64_t o0 = __ldg(&P.offsets[b]), o1 = __ldg(&P.offsets[b + 1]), tot = __ldg(&P.offsets[P.B]);
    const bool ok = o0 >= 0 && o0 <= o1 && o1 <= tot && o1 <= P.total && o1 - o0 <= P.k;
    r.n = ok ? o1 - o0 + 1 : 0;
    r.row0 = o0 + b;
    return r;
}

// A request's new length, the pages it holds, and what it asks for.
struct PlanNeed {
    int64_t len;
    int held, grow, back;
};
__device__ __forceinline__ PlanNeed plan_need(const PlanParams& P, int64_t b) {
    PlanNeed q;
    const int h = __ldg(&P.held[b]);
    q.held = h < 0 ? 0 : (h < P.max_blocks ? h : P.max_blocks);
    q.grow = q.back = 0;
    q.len = 0;
    if (P.release != nullptr && __ldg(&P.release[b]) != 0) {
        q.back = q.held;
        return q;
    }
    const int l = P.seq_lens[b];
    q.len = l < 0 ? 0 : l;
    if (P.accept_len != nullptr) {
        const int a = __ldg(&P.accept_len[b]);
        if (a >= 0) q.len += static_cast<int64_t>(a) + 1;
    }
    if (q.len > INT_MAX) q.len = INT_MAX;
    const int64_t n = plan_rows(P, b).n;
    const int64_t need = n > 0 ? (q.len + n + P.block_size - 1) / P.block_size : 0;
    if (need <= P.max_blocks && need > q.held) q.grow = static_cast<int>(need) - q.held;
    return q;
}

// CTA-wide exclusive prefix sums of two counts in thread order.
struct PlanScan {
    int64_t grow, back;
};
__device__ __forceinline__ PlanScan plan_scan(PlanScan v, PlanScan* red, PlanScan* total) {
    const int lane = threadIdx.x & 31, wp = threadIdx.x >> 5;
    PlanScan incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t g = __shfl_up_sync(FULL_MASK, incl.grow, o), k = __shfl_up_sync(FULL_MASK, incl.back, o);
        if (lane >= o) {
            incl.grow += g;
            incl.back += k;
        }
    }
    if (lane == 31) red[wp] = incl;
    __syncthreads();
    PlanScan before = {0, 0}, all = {0, 0};
    for (int w = 0; w < kPlanThreads / 32; ++w) {
        if (w < wp) {
            before.grow += red[w].grow;
            before.back += red[w].back;
        }
        all.grow += red[w].grow;
        all.back += red[w].back;
    }
    __syncthreads();
    *total = all;
    PlanScan ex;
    ex.grow = before.grow + incl.grow - v.grow;
    ex.back = before.back + incl.back - v.back;
    return ex;
}

__device__ __forceinline__ int64_t wrap(int64_t x, int64_t cap) { return x % cap; }

__global__ void __launch_bounds__(kPlanThreads) plan_tables_kernel(const PlanParams P) {
    __shared__ PlanScan red[kPlanThreads / 32];
    __shared__ int64_t taken_s;
    const int lane = threadIdx.x & 31;
    grid_dependency_wait();
    grid_launch_dependents();
    int64_t head = P.ring_state[0], count = P.ring_state[1];
    if (head < 0 || head >= P.capacity) head = 0;
    if (count < 0) count = 0;
    if (count > P.capacity) count = P.capacity;
    if (threadIdx.x == 0) taken_s = 0;
    __syncthreads();
    PlanScan carry = {0, 0};
    int64_t most = 0;  // pages granted up to the last request of this thread that got its pages
    for (int64_t b0 = 0; b0 < P.B; b0 += kPlanThreads) {
        const int64_t b = b0 + threadIdx.x;
        PlanNeed q = {0, 0, 0, 0};
        if (b < P.B) q = plan_need(P, b);
        PlanScan v = {q.grow, q.back}, total;
        const PlanScan ex = plan_scan(v, red, &total);
        const int64_t first = carry.grow + ex.grow, ret = carry.back + ex.back;
        carry.grow += total.grow;
        carry.back += total.back;
        int got = first + q.grow <= count ? q.grow : 0;
        if (got > 0) most = first + got;
        if (b < P.B) {
            P.seq_out[b] = static_cast<int32_t>(q.len);
            P.held_out[b] = q.back > 0 || (P.release != nullptr && __ldg(&P.release[b]) != 0) ? 0 : q.held + got;
        }
        // New table entries and returned pages, a warp at a time: the lanes of
        // the warp share each request's pages.
        const int moves = got > 0 ? got : q.back;
        for (unsigned m = __ballot_sync(FULL_MASK, moves > 0); m != 0u; m &= m - 1u) {
            const int l = __ffs(m) - 1;
            const int64_t rb = __shfl_sync(FULL_MASK, b, l);
            const int g = __shfl_sync(FULL_MASK, got, l), h = __shfl_sync(FULL_MASK, q.held, l);
            const int64_t f = __shfl_sync(FULL_MASK, first, l), rt = __shfl_sync(FULL_MASK, ret, l);
            int32_t* row = P.tables + rb * P.table_stride;
            if (g > 0) {
                for (int i = lane; i < g; i += 32) row[h + i] = P.ring[wrap(head + f + i, P.capacity)];
            } else {
                for (int i = lane; i < h; i += 32)
                    if (count + rt + i < P.capacity) P.ring[wrap(head + count + rt + i, P.capacity)] = row[i];
            }
        }
    }
    if (most > 0) atomicMax(reinterpret_cast<unsigned long long*>(&taken_s), static_cast<unsigned long long>(most));
    __syncthreads();
    if (threadIdx.x == 0) {
        const int64_t taken = taken_s;
        const int64_t back = carry.back < P.capacity - count ? carry.back : P.capacity - count;
        P.ring_out[0] = static_cast<int32_t>(wrap(head + taken, P.capacity));
        P.ring_out[1] = static_cast<int32_t>(count - taken + back);
    }
}

// Slots of one request's rows first, first + step, ...
__device__ __forceinline__ void write_slots(const PlanParams& P, int64_t b, int64_t first, int64_t end, int64_t step) {
    const PlanRows r = plan_rows(P, b);
    const bool gone = P.release != nullptr && __ldg(&P.release[b]) != 0;
    const int64_t len = __ldcg(&P.seq_out[b]);
    const int held = __ldcg(&P.held_out[b]);
    const int32_t* row = P.tables + b * P.table_stride;
    if (end > r.n) end = r.n;
    for (int64_t j = first; j < end; j += step) {
        const int64_t p = len + j;
        const int64_t page = p / P.block_size;
        int64_t slot = -1;
        if (!gone && page < held) {
            const int block = __ldcg(&row[page]);
            if (block >= 0) slot = static_cast<int64_t>(block) * P.block_size + (p - page * P.block_size);
        }
        P.positions[r.row0 + j] = gone ? -1 : p;
        P.slots[r.row0 + j] = slot;
    }
}

constexpr int kSlotTile = 1024;  // rows of a request per warp

__global__ void __launch_bounds__(NT) plan_slots_kernel(const PlanParams P) {
    grid_dependency_wait();
    grid_launch_dependents();
    const int64_t b = static_cast<int64_t>(blockIdx.x) * NWARPS + (threadIdx.x >> 5);
    if (b >= P.B) return;
    const int64_t r0 = static_cast<int64_t>(blockIdx.y) * kSlotTile;
    write_slots(P, b, r0 + (threadIdx.x & 31), r0 + kSlotTile, 32);
}

}  // namespace specdec
