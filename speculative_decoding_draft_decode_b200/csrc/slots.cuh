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
// plan_tables_kernel: lengths, page counts, prefix sums of the pages asked for
// and returned, the tables' new entries and the ring.  One cluster of up to 8
// CTAs, a thread per request (several beyond 8192): the CTAs' totals go
// through distributed shared memory, so the whole batch is scanned in one
// launch.  Bound by the latency of its few dependent reads, not by bytes: 64
// requests of 6 rows 4.5 us, 4096 with 0 to 8 drafts each 9.6 us (two launches).
// A batch that one CTA holds and whose rows are few gets its positions and
// slots in the same launch; otherwise plan_slots_kernel writes them.
#pragma once

#include <cooperative_groups.h>
#include <cuda_runtime.h>
#include <limits.h>
#include <stdint.h>

#include "device_utils.cuh"
#include "verify_common.cuh"

namespace specdec {

constexpr int kPlanThreads = 1024;
constexpr int kPlanFew = 256;        // threads for batches of at most so many requests with few rows
constexpr int kPlanCtas = 8;         // CTAs of the cluster at most (the portable cluster size)
constexpr int kPlanFusedRows = 8192; // rows that plan_tables_kernel maps itself (one CTA)

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
    bool gone;
};
__device__ __forceinline__ PlanNeed plan_need(const PlanParams& P, int64_t b, const PlanRows& rows) {
    PlanNeed q;
    const int h = P.held[b], l = P.seq_lens[b];  // plain loads: the outputs may be the same arrays
    const int a = P.accept_len != nullptr ? __ldg(&P.accept_len[b]) : -1;
    q.gone = P.release != nullptr && __ldg(&P.release[b]) != 0;
    q.held = h < 0 ? 0 : (h < P.max_blocks ? h : P.max_blocks);
    q.grow = q.back = 0;
    q.len = 0;
    if (q.gone) {
        q.back = q.held;
        return q;
    }
    q.len = l < 0 ? 0 : l;
    if (a >= 0) q.len += static_cast<int64_t>(a) + 1;
    if (q.len > INT_MAX) q.len = INT_MAX;
    // len + n + block_size stays below 2^32
    const unsigned need = rows.n > 0 ? (static_cast<unsigned>(q.len + rows.n - 1)) / static_cast<unsigned>(P.block_size) + 1u : 0u;
    if (need <= static_cast<unsigned>(P.max_blocks) && static_cast<int>(need) > q.held) q.grow = static_cast<int>(need) - q.held;
    return q;
}

// Prefix sums of pages asked for and returned.
struct PlanScan {
    int64_t grow, back;
};
__device__ __forceinline__ PlanScan warp_inclusive(PlanScan v, bool backs) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t g = __shfl_up_sync(FULL_MASK, v.grow, o);
        if (lane >= o) v.grow += g;
    }
    if (backs) {
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t k = __shfl_up_sync(FULL_MASK, v.back, o);
            if (lane >= o) v.back += k;
        }
    }
    return v;
}

// Slot of position p of a request that holds `held` pages.
__device__ __forceinline__ int64_t plan_slot(const PlanParams& P, const int32_t* table, unsigned p, int held) {
    const unsigned page = p / static_cast<unsigned>(P.block_size);
    if (page >= static_cast<unsigned>(held)) return -1;
    const int block = __ldcg(&table[page]);
    return block >= 0 ? static_cast<int64_t>(block) * P.block_size + (p - page * static_cast<unsigned>(P.block_size)) : -1;
}

// One request's page moves: new table entries from the ring's head, or the
// pages it held back behind the tail.  Indexes stay below 2 capacities.
struct PlanMove {
    int64_t b, first, ret;
    int got, held;
};
__device__ __forceinline__ void plan_move(const PlanParams& P, const PlanMove& m, int64_t head, int64_t count, int i0,
                                          int step) {
    int32_t* row = P.tables + m.b * P.table_stride;
    if (m.got > 0) {
        for (int i = i0; i < m.got; i += step) {
            int64_t at = head + m.first + i;
            if (at >= P.capacity) at -= P.capacity;
            row[m.held + i] = P.ring[at];
        }
    } else {
        for (int i = i0; i < m.held && count + m.ret + i < P.capacity; i += step) {
            int64_t at = head + count + m.ret + i;
            if (at >= P.capacity) at -= P.capacity;
            P.ring[at] = row[i];
        }
    }
}

// Pages that a thread takes or returns by itself, one after another; the few
// longer moves (prompts, released requests) are shared by its warp.
constexpr int kPlanTake = 12, kPlanReturn = 4;

template <int THREADS>
struct PlanSmem {
    PlanScan warp[32];
    PlanScan cta[kPlanCtas];        // written by the cluster's CTAs
    unsigned long long taken[kPlanCtas];
    unsigned long long most;
    // one CTA that also maps the rows
    unsigned len[THREADS];
    int held[THREADS];              // -1: released
    int64_t row0[THREADS];
    uint16_t request[kPlanFusedRows];
};

template <bool FUSED, int THREADS>
__global__ void __launch_bounds__(THREADS) plan_tables_kernel(const PlanParams P) {
    namespace cg = cooperative_groups;
    __shared__ PlanSmem<THREADS> sm;
    const int t = threadIdx.x, lane = t & 31, wp = t >> 5;
    const int ctas = static_cast<int>(gridDim.x), rank = static_cast<int>(blockIdx.x);  // one cluster
    grid_dependency_wait();
    grid_launch_dependents();
    // Waited for before the first remote write: by then every CTA of the cluster runs.
    if (!FUSED && ctas > 1) cg::this_cluster().barrier_arrive();
    const int per = (P.B + ctas * THREADS - 1) / (ctas * THREADS);  // requests of a thread, consecutive
    const int64_t b0 = (static_cast<int64_t>(rank) * THREADS + t) * per;
    const bool backs = P.release != nullptr;
    int64_t head = P.ring_state[0], count = P.ring_state[1];
    const int64_t rows = FUSED ? (P.offsets == nullptr ? static_cast<int64_t>(P.B) * (P.k + 1) : P.B + P.total) : 0;
    if (FUSED && P.offsets != nullptr)
        for (int i = t; i < rows; i += THREADS) sm.request[i] = 0xffffu;
    PlanScan mine = {0, 0};
    PlanNeed q = {0, 0, 0, 0, false};
    PlanRows pr = {0, 0};
    for (int i = 0; i < per; ++i)
        if (b0 + i < P.B) {
            pr = plan_rows(P, b0 + i);
            q = plan_need(P, b0 + i, pr);
            mine.grow += q.grow;
            mine.back += q.back;
        }
    if (head < 0 || head >= P.capacity) head = 0;
    if (count < 0) count = 0;
    if (count > P.capacity) count = P.capacity;
    if (t == 0) sm.most = 0ull;
    PlanScan incl = warp_inclusive(mine, backs);
    if (lane == 31) sm.warp[wp] = incl;
    __syncthreads();
    PlanScan w = {0, 0};
    if (lane < THREADS / 32) w = sm.warp[lane];
    w = warp_inclusive(w, backs);  // over the warps, in every warp
    PlanScan all = {__shfl_sync(FULL_MASK, w.grow, 31), __shfl_sync(FULL_MASK, w.back, 31)};
    PlanScan before = {__shfl_sync(FULL_MASK, w.grow, (wp + 31) & 31), __shfl_sync(FULL_MASK, w.back, (wp + 31) & 31)};
    if (wp == 0) before = {0, 0};
    PlanScan at = {before.grow + incl.grow - mine.grow, before.back + incl.back - mine.back};
    if (!FUSED && ctas > 1) {
        cg::cluster_group cluster = cg::this_cluster();
        cluster.barrier_wait();
        if (t < ctas) cluster.map_shared_rank(&sm, t)->cta[rank] = all;
        cluster.sync();
        PlanScan total = {0, 0};
        for (int i = 0; i < ctas; ++i) {
            const PlanScan c = sm.cta[i];
            if (i < rank) {
                at.grow += c.grow;
                at.back += c.back;
            }
            total.grow += c.grow;
            total.back += c.back;
        }
        all = total;
    }
    // Requests whose pages the ring holds get them.
    int64_t most = 0;  // pages taken up to this thread's last such request
    for (int i = 0; i < per; ++i) {
        const int64_t b = b0 + i;
        PlanMove m = {b, at.grow, at.back, 0, 0};
        if (b < P.B) {
            if (per > 1) {
                pr = plan_rows(P, b);
                q = plan_need(P, b, pr);
            }
            if (at.grow + q.grow <= count) m.got = q.grow;
            m.held = q.held;
            if (m.got > 0) most = at.grow + m.got;
            at.grow += q.grow;
            at.back += q.back;
            const int held = q.gone ? 0 : q.held + m.got;
            P.seq_out[b] = static_cast<int32_t>(q.len);
            P.held_out[b] = held;
            if (FUSED) {
                sm.len[t] = static_cast<unsigned>(q.len);
                sm.held[t] = q.gone ? -1 : held;
                sm.row0[t] = pr.row0;
                if (P.offsets != nullptr)
                    for (int64_t j = pr.row0; j < pr.row0 + pr.n; ++j) sm.request[j] = static_cast<uint16_t>(t);
            }
        }
        const int pages = b < P.B ? (m.got > 0 ? m.got : q.back) : 0;
        const bool own = pages <= (m.got > 0 ? kPlanTake : kPlanReturn);
        if (pages > 0 && own) plan_move(P, m, head, count, 0, 1);
        for (unsigned long_ones = __ballot_sync(FULL_MASK, !own); long_ones != 0u; long_ones &= long_ones - 1u) {
            const int l = __ffs(long_ones) - 1;
            PlanMove x;
            x.b = __shfl_sync(FULL_MASK, m.b, l);
            x.first = __shfl_sync(FULL_MASK, m.first, l);
            x.ret = __shfl_sync(FULL_MASK, m.ret, l);
            x.got = __shfl_sync(FULL_MASK, m.got, l);
            x.held = __shfl_sync(FULL_MASK, m.held, l);
            plan_move(P, x, head, count, lane, 32);
        }
    }
    // The ring after this call.  Everything asked for was there, or what the last
    // granted request took up to.  (Every CTA read the ring's state before the
    // cluster's barrier above; the outputs may replace it.)
    int64_t taken = all.grow;
    if (all.grow > count) {  // the same in every CTA
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) most = max(most, __shfl_xor_sync(FULL_MASK, most, o));
        if (lane == 0 && most > 0) atomicMax(&sm.most, static_cast<unsigned long long>(most));
        __syncthreads();
        taken = static_cast<int64_t>(sm.most);
        if (!FUSED && ctas > 1) {
            cg::cluster_group cluster = cg::this_cluster();
            if (t == 0) cluster.map_shared_rank(&sm, 0)->taken[rank] = sm.most;
            cluster.sync();
            if (rank == 0)
                for (int i = 0; i < ctas; ++i) taken = max(taken, static_cast<int64_t>(sm.taken[i]));
        }
    }
    __syncthreads();
    if (rank == 0 && t == 0) {
        const int64_t back = all.back < P.capacity - count ? all.back : P.capacity - count;
        int64_t h = head + taken;
        if (h >= P.capacity) h -= P.capacity;
        P.ring_out[0] = static_cast<int32_t>(h);
        P.ring_out[1] = static_cast<int32_t>(count - taken + back);
    }
    if (FUSED) {  // a thread per row; the tables' entries were written by this CTA before the barrier
        for (int i = t; i < rows; i += THREADS) {
            const unsigned b = P.offsets == nullptr ? static_cast<unsigned>(i) / static_cast<unsigned>(P.k + 1) : sm.request[i];
            if (b == 0xffffu) continue;
            const int held = sm.held[b];
            const unsigned p = sm.len[b] + static_cast<unsigned>(i - sm.row0[b]);
            P.positions[i] = held < 0 ? -1 : static_cast<int64_t>(p);
            P.slots[i] = held < 0 ? -1 : plan_slot(P, P.tables + b * P.table_stride, p, held);
        }
    }
}

constexpr int kSlotTile = 1024;  // rows of a request per warp

// A warp per request and tile of its rows.
__global__ void __launch_bounds__(NT) plan_slots_kernel(const PlanParams P) {
    grid_dependency_wait();
    grid_launch_dependents();
    const int64_t b = static_cast<int64_t>(blockIdx.x) * NWARPS + (threadIdx.x >> 5);
    if (b >= P.B) return;
    const int lane = threadIdx.x & 31;
    const int64_t first = static_cast<int64_t>(blockIdx.y) * kSlotTile;
    const PlanRows r = plan_rows(P, b);
    const bool gone = P.release != nullptr && __ldg(&P.release[b]) != 0;
    const unsigned len = static_cast<unsigned>(__ldcg(&P.seq_out[b]));
    const int held = __ldcg(&P.held_out[b]);
    const int64_t end = min(r.n, first + kSlotTile);
    for (int64_t j = first + lane; j < end; j += 32) {
        const unsigned p = len + static_cast<unsigned>(j);
        P.positions[r.row0 + j] = gone ? -1 : static_cast<int64_t>(p);
        P.slots[r.row0 + j] = gone ? -1 : plan_slot(P, P.tables + b * P.table_stride, p, held);
    }
}

}  // namespace specdec
