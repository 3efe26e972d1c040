// beam_select.cuh — one step of beam search or draft-tree expansion: the K
// best continuations of every request's W beams over the vocabulary.
//
// Handbook page, "EAGLE" (EAGLE-2 grows its draft tree by the cumulative
// probability of the branches) and "Medusa" (candidates form a tree): the
// level's candidates are every (beam w, token v) with
//   c = s_w + l_wv - log sum_v' exp(l_wv'),
// and the K largest are kept, equal values in order of w V + v.  A row adds
// the same number to all its logits, so a row's K best are its K largest
// logits (lowest index first among equals), whatever its sum turns out to be:
// the logits are read once.
//
// beam_pass_kernel: one CTA per (row, chunk of up to kU 16-byte vectors per
// thread).  The chunk stays in registers: its maximum, a threshold that at
// least K of its elements reach, sum exp(l - max), and its K best keys.
// beam_merge_kernel: one CTA per request: the rows' sums, a bound that K
// candidates reach, and the order of the candidates above it in fp64.
// Nothing is shared between CTAs but the partials, and every sum has a fixed
// order: the results do not vary from run to run.
#pragma once

#include <cuda_runtime.h>
#include <float.h>
#include <limits.h>
#include <stdint.h>

#include "device_utils.cuh"
#include "verify_common.cuh"
#include "verify_pass1.cuh"

namespace specdec {

constexpr int kMaxBeams = 32;    // beams per request, and beams selected
constexpr int kBeamMerge = 1024;  // candidates of a request held in shared memory

struct BeamStat {
    double M;  // a value near the chunk's largest logit
    double S;  // sum exp(l - M) over the chunk; NaN for a NaN or +inf logit
};

struct BeamParams {
    const void* logits;
    int64_t row_stride;
    const float* scores;      // [B, W] cumulative log probabilities; -inf: no hypothesis
    const int32_t* finished;  // [B, W] or null
    int B, W, K, V;
    int eos;
    int cpr;             // chunks per row
    BeamStat* stats;     // [B W, cpr]
    uint64_t* keys;      // [B W, cpr, K] the chunks' best, descending, 0 past the end
    float* out_scores;   // [B, K]
    int32_t* out_parents;
    int32_t* out_tokens;
};

// Rows that are streamed: a hypothesis with a finite score that is not
// finished.
__device__ __forceinline__ bool beam_streams(const BeamParams& P, int64_t r) {
    const float s = __ldg(&P.scores[r]);
    if (!(s > -INFINITY && s < INFINITY)) return false;
    return P.finished == nullptr || __ldg(&P.finished[r]) == 0;
}

// The vectors of a row: elements before the first 16-byte boundary (the
// head), nv full vectors, and the elements behind them (the tail).  Rows need
// no alignment beyond their element's.
struct RowCut {
    int head, nv, tail;
};
template <class Tag, int VEC>
__device__ __forceinline__ RowCut cut_row(const typename Tag::storage* row, int V) {
    constexpr int es = sizeof(typename Tag::storage);
    RowCut c;
    c.head = static_cast<int>((16 - (reinterpret_cast<uintptr_t>(row) & 15)) & 15) / es;
    if (c.head > V) c.head = V;
    c.nv = (V - c.head) / VEC;
    c.tail = V - c.head - c.nv * VEC;
    return c;
}

template <class Tag>
__device__ __forceinline__ uint4 minus_inf_vec() {
    const uint32_t x = sizeof(typename Tag::storage) == 2 ? 0xff80ff80u : 0xff800000u;
    return make_uint4(x, x, x, x);
}

// A value that at least K of the CTA's threads reach, from one ordered value
// per thread (INT_MIN: none): the K-th largest of the 32 values that the
// warps' 32 / warps largest lanes make up.  pool holds 32 words; one CTA
// barrier.  x: the bound (INT_MIN if fewer than K values are there), y: the
// largest value.
__device__ __forceinline__ int2 cta_kth(int v, int K, int warps, int* pool) {
    const int lane = threadIdx.x & 31, wp = threadIdx.x >> 5;
    const int m = 32 / warps;
    int mine = INT_MIN;
    for (int i = 0; i < m; ++i) {
        const int x = __reduce_max_sync(FULL_MASK, v);
        if (lane == i) mine = x;
        const unsigned who = __ballot_sync(FULL_MASK, v == x);
        if (lane == __ffs(who) - 1) v = INT_MIN;
    }
    if (lane < m) pool[wp * m + lane] = mine;
    __syncthreads();
    int p = pool[lane];
    int2 r;
    r.y = __reduce_max_sync(FULL_MASK, p);
    if (K <= 16) {  // take the K - 1 largest out
        r.x = r.y;
        for (int i = 1; i < K; ++i) {
            const unsigned who = __ballot_sync(FULL_MASK, p == r.x);
            if (lane == __ffs(who) - 1) p = INT_MIN;
            r.x = __reduce_max_sync(FULL_MASK, p);
        }
    } else {  // take the 32 - K least out
        r.x = __reduce_min_sync(FULL_MASK, p);
        for (int i = K; i < 32; ++i) {
            const unsigned who = __ballot_sync(FULL_MASK, p == r.x);
            if (lane == __ffs(who) - 1) p = INT_MAX;
            r.x = __reduce_min_sync(FULL_MASK, p);
        }
    }
    return r;
}

__device__ __forceinline__ uint32_t max_bf162(uint32_t a, uint32_t b) {
    const __nv_bfloat162 m = __hmax2(as_bf162(a), as_bf162(b));
    uint32_t r;
    memcpy(&r, &m, 4);
    return r;
}

// Two fp32 values in one 64-bit register pair (packed add and fused multiply-add).
__device__ __forceinline__ uint64_t f32x2(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ float2 f32x2_get(uint64_t x) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
    return r;
}
__device__ __forceinline__ uint64_t f32x2_add(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t f32x2_fma(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

#ifndef BEAM_MINB
#define BEAM_MINB 5
#endif
constexpr int kBeamBatch = 4;    // vectors a thread loads at a time, one batch ahead
constexpr int kBeamVecs = 1024;   // vectors of a chunk that may hold candidates
constexpr int kBeamCand = 512;   // candidates of a chunk
constexpr float kLog2e = 1.4426950408889634f;

struct BeamSmem {
    uint4 vec[kBeamVecs];
    int at[kBeamVecs];  // their vector numbers
    uint64_t cand[kBeamCand];
    uint64_t red[NWARPS];
    double S[NWARPS];
    float ref[NWARPS];
    int pool[32];
    int vecs, cands;
};

// What a thread carries through its part of a chunk.
struct BeamThread {
    float th;    // K elements of the chunk reach it
    float hit;   // elements below it are no candidates of the batches to come
    float ref;   // S counts exp(l - beam_ref(ref))
    bool known;  // CTA-uniform: K elements above -inf have been seen
    bool flood;  // many vectors reach the threshold
    double S;
};

// Each term is taken as 2^(l c - E) with one rounding in the exponent: c is
// log2 e in fp32 and E = ref c in fp32, so the terms count from E / c exactly,
// and c's own error (2^-26 relative) only weighs the distance from there.
// Values so large that ref c or l c leaves fp32 take l - ref first.
__device__ __forceinline__ bool beam_far(float ref) { return !(fabsf(ref) < 1e37f); }
__device__ __forceinline__ double beam_ref(float ref) {
    return beam_far(ref) ? static_cast<double>(ref)
                         : static_cast<double>(__fmul_rn(ref, kLog2e)) / static_cast<double>(kLog2e);
}
__device__ __forceinline__ float beam_term(float x, float ref) {
    return ex2_sfu(beam_far(ref) ? (x - ref) * kLog2e : __fmaf_rn(x, kLog2e, -__fmul_rn(ref, kLog2e)));
}

// The sum of a batch's terms, fp32: 2 x 16 (bf16) or 2 x 8 (fp32) of them.
template <class Tag, int VEC>
__device__ __forceinline__ float beam_batch_sum(const uint4 (&w)[kBeamBatch], float ref) {
    if (beam_far(ref)) {
        float s = 0.0f;
#pragma unroll 1
        for (int i = 0; i < kBeamBatch * VEC; ++i) {
            const int u = i / VEC;
            const uint4 x = u == 0 ? w[0] : u == 1 ? w[1] : u == 2 ? w[2] : w[3];
            s += beam_term(VecOps<Tag, VEC>::elem(x, i % VEC), ref);
        }
        return s;
    }
    const float E = __fmul_rn(ref, kLog2e);
    const uint64_t minus = f32x2(-E, -E), scale = f32x2(kLog2e, kLog2e);
    uint64_t s = f32x2(0.0f, 0.0f);
#pragma unroll
    for (int u = 0; u < kBeamBatch; ++u)
#pragma unroll
        for (int q = 0; q < VEC; q += 2) {
            const uint64_t x = f32x2(VecOps<Tag, VEC>::elem(w[u], q), VecOps<Tag, VEC>::elem(w[u], q + 1));
            const float2 e = f32x2_get(f32x2_fma(x, scale, minus));
            s = f32x2_add(s, f32x2(ex2_sfu(e.x), ex2_sfu(e.y)));
        }
    const float2 r = f32x2_get(s);
    return r.x + r.y;
}

// The largest element of a batch (NaN ignored).
template <class Tag, int VEC>
__device__ __forceinline__ float beam_batch_max(const uint4 (&w)[kBeamBatch]) {
    if constexpr (sizeof(typename Tag::storage) == 2) {
        const uint4 m = make_uint4(max_bf162(max_bf162(w[0].x, w[1].x), max_bf162(w[2].x, w[3].x)),
                                   max_bf162(max_bf162(w[0].y, w[1].y), max_bf162(w[2].y, w[3].y)),
                                   max_bf162(max_bf162(w[0].z, w[1].z), max_bf162(w[2].z, w[3].z)),
                                   max_bf162(max_bf162(w[0].w, w[1].w), max_bf162(w[2].w, w[3].w)));
        return VecOps<Tag, VEC>::vmax(m);
    } else {
        return fmaxf(fmaxf(VecOps<Tag, VEC>::vmax(w[0]), VecOps<Tag, VEC>::vmax(w[1])),
                     fmaxf(VecOps<Tag, VEC>::vmax(w[2]), VecOps<Tag, VEC>::vmax(w[3])));
    }
}

// A value above the reference by more than kBeamRaise: the sum goes over to it
// (terms stay below 2^6 and the fp32 sums far from overflow).
constexpr float kBeamRaise = 4.0f;
__device__ __forceinline__ void beam_raise(BeamThread& st, float m) {
    if (m > st.ref + kBeamRaise) {
        st.S *= exp(beam_ref(st.ref) - beam_ref(m));
        st.ref = m;
    }
}

// The least float above x (both zeros count as +0).
__device__ __forceinline__ float next_up(float x) { return x == 0.0f ? __int_as_float(1) : from_ord_i32(ord_i32(x) + 1); }

template <class Tag, int VEC>
__device__ __forceinline__ void beam_batch(BeamThread& st, const uint4 (&w)[kBeamBatch], int j, int K, BeamSmem& sm) {
    const int lane = threadIdx.x & 31;
    const float tm = beam_batch_max<Tag, VEC>(w);
    const bool first = !st.known;
    bool raised = false;
    if (first) {
        __syncthreads();
        const int2 k = cta_kth(ord_i32(tm), K, NWARPS, sm.pool);
        if (k.x >= ord_i32(-FLT_MAX)) {
            st.known = true;
            st.th = st.hit = from_ord_i32(k.x);
            raised = true;
        }
        const float top = from_ord_i32(k.y);  // one reference for the CTA
        if (top > -INFINITY) beam_raise(st, top);
    } else if (__any_sync(FULL_MASK, st.flood)) {
        // Many vectors reach the threshold: raise it to the K-th largest lane
        // maximum of this warp's batch.
        int v = ord_i32(tm), x = INT_MIN;
        for (int i = 0; i < K; ++i) {
            x = __reduce_max_sync(FULL_MASK, v);
            const unsigned who = __ballot_sync(FULL_MASK, v == x);
            if (lane == __ffs(who) - 1) v = INT_MIN;
        }
        if (x >= ord_i32(-FLT_MAX) && from_ord_i32(x) > st.th) {
            st.th = st.hit = from_ord_i32(x);
            raised = true;
        }
    }
    if (tm >= st.hit) {
        beam_raise(st, tm);  // the reference is never below the threshold - kBeamRaise
#pragma unroll
        for (int u = 0; u < kBeamBatch; ++u)
            if (VecOps<Tag, VEC>::vmax(w[u]) >= st.hit) {
                const int at = atomicAdd(&sm.vecs, 1);
                if (at < kBeamVecs) {
                    sm.vec[at] = w[u];
                    sm.at[at] = j + u * NT;
                }
                st.flood |= at > kBeamVecs / 4;
            }
    }
    // The K elements that reach a threshold are in the batch that gave it:
    // elements of later batches that only equal it come behind them.
    if (raised) st.hit = next_up(st.th);
    st.S += static_cast<double>(beam_batch_sum<Tag, VEC>(w, st.ref));
}

// The K best keys of a chunk whose candidates do not fit (runs of equal
// values): the largest key below the last one found, K times, over the
// vectors put aside or, if there were more than kBeamVecs, over the chunk read
// again.  CTA-collective.
template <class Tag, int VEC>
__device__ __noinline__ void beam_chunk_ties(const typename Tag::storage* row, RowCut cut, int v0, int cnt, bool ends,
                                             float th, int K, BeamSmem& sm, uint64_t* out) {
    const int t = threadIdx.x;
    const int vecs = sm.vecs;
    const int first = cut.head + v0 * VEC, n = vecs <= kBeamVecs ? 0 : cnt * VEC;
    const int extra = ends ? cut.head + cut.tail : 0;
    uint64_t last = ~0ull;
    for (int i = 0; i < K; ++i) {
        uint64_t best = 0ull;
        auto offer = [&](float f, int x) {
            if (f >= th) {
                const uint64_t k = make_key(f, x);
                if (k < last && k > best) best = k;
            }
        };
        if (vecs <= kBeamVecs)
            for (int j = t; j < vecs; j += NT) {
                const uint4 w = sm.vec[j];
#pragma unroll
                for (int q = 0; q < VEC; ++q) offer(VecOps<Tag, VEC>::elem(w, q), first + sm.at[j] * VEC + q);
            }
        for (int j = t; j < n + extra; j += NT) {
            int x = first + j;
            if (j >= n) x = j - n < cut.head ? j - n : cut.head + cut.nv * VEC + (j - n - cut.head);
            offer(load_scalar<Tag>(row + x), x);
        }
        best = block_max_u64(best, sm.red);
        if (t == 0) out[i] = best;
        last = best;
    }
}

template <class Tag, int VEC>
__global__ void __launch_bounds__(NT, BEAM_MINB) beam_pass_kernel(const BeamParams P) {
    __shared__ BeamSmem sm;
    using Elem = typename Tag::storage;
    const int t = threadIdx.x, lane = t & 31, wp = t >> 5;
    grid_dependency_wait();
    grid_launch_dependents();
    const int64_t r = blockIdx.x;
    const int sub = blockIdx.y;
    if (!beam_streams(P, r)) return;  // CTA-uniform
    const Elem* row = static_cast<const Elem*>(P.logits) + r * P.row_stride;
    const RowCut cut = cut_row<Tag, VEC>(row, P.V);
    // the row's vectors are dealt evenly over its chunks
    const int per = (cut.nv + P.cpr - 1) / P.cpr;
    const int v0 = min(sub * per, cut.nv), cnt = min(per, cut.nv - v0);
    const Elem* base = row + cut.head + static_cast<int64_t>(v0) * VEC;
    auto load = [&](uint4 (&w)[kBeamBatch], int j) {
        if (j - t + NT * kBeamBatch <= cnt) {  // CTA-uniform: a whole batch
            const Elem* p = base + static_cast<int64_t>(j) * VEC;
#pragma unroll
            for (int u = 0; u < kBeamBatch; ++u) w[u] = ld_stream_v4(p + u * NT * VEC);
            return;
        }
#pragma unroll
        for (int u = 0; u < kBeamBatch; ++u) {
            w[u] = minus_inf_vec<Tag>();
            if (j + u * NT < cnt) w[u] = ld_stream_v4(base + static_cast<int64_t>(j + u * NT) * VEC);
        }
    };
    uint4 wa[kBeamBatch], wb[kBeamBatch];
    load(wa, t);
    // the first chunk also takes the row's head and tail, one element a thread
    float xe = -INFINITY;
    int ie = 0;
    if (sub == 0 && t < cut.head + cut.tail) {
        ie = t < cut.head ? t : cut.head + cut.nv * VEC + (t - cut.head);
        xe = load_scalar<Tag>(row + ie);
    }
    if (t == 0) sm.vecs = sm.cands = 0;
    BeamThread st;
    st.th = st.hit = st.ref = -FLT_MAX;
    st.known = st.flood = false;
    st.S = 0.0;
    constexpr int kStep = NT * kBeamBatch;
    for (int j = t; j - t < max(cnt, 1); j += 2 * kStep) {
        load(wb, j + kStep);
        beam_batch<Tag, VEC>(st, wa, j, P.K, sm);
        if (j - t + kStep >= cnt) break;
        load(wa, j + 2 * kStep);
        beam_batch<Tag, VEC>(st, wb, j + kStep, P.K, sm);
    }
    if (xe > -INFINITY || xe != xe) {
        beam_raise(st, xe);
        st.S += static_cast<double>(beam_term(xe, st.ref));
        if (xe >= st.th) {
            const int at = atomicAdd(&sm.cands, 1);
            sm.cand[at] = make_key(xe, ie);  // at most 14 of these
        }
    }
    // one reference for the warp (the threads' are the same but for spikes)
    const float ref = from_ord_i32(__reduce_max_sync(FULL_MASK, ord_i32(st.ref)));
    double S = st.S;
    if (st.ref != ref && S != 0.0) S *= exp(beam_ref(st.ref) - beam_ref(ref));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) S += __shfl_xor_sync(FULL_MASK, S, o);
    if (lane == 0) {
        sm.S[wp] = S;
        sm.ref[wp] = ref;
    }
    __syncthreads();
    const int64_t chunk = r * P.cpr + sub;
    if (wp == 0) {  // and one for the CTA
        S = lane < NWARPS ? sm.S[lane] : 0.0;
        const float mine = lane < NWARPS ? sm.ref[lane] : -FLT_MAX;
        const float R = from_ord_i32(__reduce_max_sync(FULL_MASK, ord_i32(mine)));
        if (mine != R && S != 0.0) S *= exp(beam_ref(mine) - beam_ref(R));
#pragma unroll
        for (int o = NWARPS / 2; o > 0; o >>= 1) S += __shfl_xor_sync(FULL_MASK, S, o);
        if (lane == 0) {
            BeamStat o;
            o.M = beam_ref(R);
            o.S = S;
            P.stats[chunk] = o;
        }
    }
    uint64_t* out = P.keys + chunk * P.K;
    const int vecs = sm.vecs;
    bool fits = vecs <= kBeamVecs;
    if (fits) {
        for (int i = t; i < vecs; i += NT) {
            const uint4 w = sm.vec[i];
            const int e0 = cut.head + (v0 + sm.at[i]) * VEC;
#pragma unroll
            for (int q = 0; q < VEC; ++q) {
                const float x = VecOps<Tag, VEC>::elem(w, q);
                if (x >= st.th) {
                    const int at = atomicAdd(&sm.cands, 1);
                    if (at < kBeamCand) sm.cand[at] = make_key(x, e0 + q);
                }
            }
        }
        __syncthreads();
        fits = sm.cands <= kBeamCand;
    }
    if (fits) {
        // The keys are distinct: a candidate's rank is its place.
        const int have = sm.cands;
        for (int i = t; i < have; i += NT) {
            const uint64_t key = sm.cand[i];
            int rank = 0;
            for (int j = 0; j < have; ++j) rank += sm.cand[j] > key ? 1 : 0;
            if (rank < P.K) out[rank] = key;
        }
        for (int i = have + t; i < P.K; i += NT) out[i] = 0ull;
    } else {
        beam_chunk_ties<Tag, VEC>(row, cut, v0, cnt, sub == 0, st.th, P.K, sm, out);
    }
}

// ---------------------------------------------------------------------------
// The request's merge: a CTA with a warp per beam (8 warps at least).
// ---------------------------------------------------------------------------
constexpr int kMergeWarps = 32;  // warps of the merge CTA at most (8, 16 or 32)
constexpr int kMergeKeys = 4;    // keys a thread holds in registers

struct BeamMergeSmem {
    double M[kMaxBeams];     // largest logit of the row
    double logS[kMaxBeams];  // log sum exp(l - M)
    double s[kMaxBeams];
    int state[kMaxBeams];    // 0: no candidates, 1: streamed, 2: finished
    double c[kBeamMerge];
    uint32_t flat[kBeamMerge];  // w V + token
    int pool[32];
    double red_c[kMergeWarps];
    uint32_t red_f[kMergeWarps];
    int cnt;
};

// A row's sum from its chunks': 32 chunks at a time, each against the largest
// reference of the 32.  Warp-collective.
__device__ __forceinline__ BeamStat beam_row_sum(const BeamStat* p, int n) {
    const int lane = threadIdx.x & 31;
    BeamStat acc;
    acc.M = -DBL_MAX;
    acc.S = 0.0;
    for (int i0 = 0; i0 < n; i0 += 32) {
        double M = -DBL_MAX, S = 0.0;
        if (i0 + lane < n) {
            M = __ldcg(&p[i0 + lane].M);
            S = __ldcg(&p[i0 + lane].S);
        }
        double top = S != 0.0 ? fmax(M, acc.M) : acc.M;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmax(top, __shfl_xor_sync(FULL_MASK, top, o));
        if (S != 0.0 && M != top) S *= exp(M - top);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) S += __shfl_xor_sync(FULL_MASK, S, o);
        if (acc.S != 0.0) S += acc.M != top ? acc.S * exp(acc.M - top) : acc.S;
        acc.M = top;
        acc.S = S;
    }
    return acc;
}

// c of a key of row w.
__device__ __forceinline__ double beam_value(const BeamMergeSmem& sm, int w, uint64_t key) {
    return (sm.s[w] + (static_cast<double>(key_value(key)) - sm.M[w])) - sm.logS[w];
}

// One candidate of the request: none where state[w] has none.
struct BeamCandidate {
    double c;
    uint32_t flat;
    bool ok;
};
__device__ __forceinline__ BeamCandidate beam_candidate(const BeamMergeSmem& sm, int w, uint64_t key, uint32_t V) {
    BeamCandidate r;
    r.ok = key != 0ull && sm.state[w] == 1;
    r.c = r.ok ? beam_value(sm, w, key) : -INFINITY;
    r.flat = static_cast<uint32_t>(w) * V + static_cast<uint32_t>(key_index(key));
    return r;
}

__device__ __forceinline__ void beam_output(const BeamParams& P, int64_t at, double c, uint32_t flat) {
    P.out_scores[at] = static_cast<float>(c);
    P.out_parents[at] = static_cast<int32_t>(flat / static_cast<uint32_t>(P.V));
    P.out_tokens[at] = static_cast<int32_t>(flat % static_cast<uint32_t>(P.V));
}

// More candidates at the bound than kBeamMerge (runs of equal values over many
// chunks): the best below the last one found, K times.  CTA-collective.
__device__ __noinline__ void beam_merge_ties(const BeamParams& P, int64_t b, BeamMergeSmem& sm) {
    const int t = threadIdx.x, nt = blockDim.x, lane = t & 31, wp = t >> 5;
    const uint32_t V = static_cast<uint32_t>(P.V);
    const int row_keys = P.cpr * P.K, total = P.W * row_keys;
    const uint64_t* keys = P.keys + b * total;
    double lc = INFINITY;
    uint32_t lf = 0u;
    for (int i = 0; i < P.K; ++i) {
        double bc = -INFINITY;
        uint32_t bf = 0xffffffffu;
        auto offer = [&](double c, uint32_t f) {
            const bool below = c < lc || (c == lc && f > lf);
            if (below && (c > bc || (c == bc && f < bf))) {
                bc = c;
                bf = f;
            }
        };
        for (int w = t; w < P.W; w += nt)
            if (sm.state[w] == 2) offer(sm.s[w], static_cast<uint32_t>(w) * V + static_cast<uint32_t>(P.eos));
        for (int j = t; j < total; j += nt) {
            const BeamCandidate q = beam_candidate(sm, j / row_keys, __ldcg(&keys[j]), V);
            if (q.ok) offer(q.c, q.flat);
        }
        auto join = [&](double c, uint32_t f) {
            if (c > bc || (c == bc && f < bf)) {
                bc = c;
                bf = f;
            }
        };
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const double c = __shfl_xor_sync(FULL_MASK, bc, o);
            const uint32_t f = __shfl_xor_sync(FULL_MASK, bf, o);
            join(c, f);
        }
        if (lane == 0) {
            sm.red_c[wp] = bc;
            sm.red_f[wp] = bf;
        }
        __syncthreads();
        for (int q = 0; q < (nt >> 5); ++q) join(sm.red_c[q], sm.red_f[q]);
        __syncthreads();
        lc = bc;
        lf = bf;
        if (t == 0) beam_output(P, b * P.K + i, bc, bf);
    }
}

__global__ void __launch_bounds__(32 * kMergeWarps) beam_merge_kernel(const BeamParams P) {
    __shared__ BeamMergeSmem sm;
    const int t = threadIdx.x, nt = blockDim.x, lane = t & 31, wp = t >> 5, nw = nt >> 5;
    grid_dependency_wait();
    grid_launch_dependents();
    const int64_t b = blockIdx.x;
    const int K = P.K, cpr = P.cpr;
    const uint32_t V = static_cast<uint32_t>(P.V);
    const int row_keys = cpr * K, total = P.W * row_keys;
    const uint64_t* keys = P.keys + b * total;
    // Key j of this thread: every warp gets keys of all rows, chunks and ranks,
    // so that the warps' largest are the request's largest.
    auto at = [&](int j) { return j * nt + lane * nw + ((wp + lane) & (nw - 1)); };
    // The keys' loads go out before the rows' sums are merged.  Rows that were
    // not streamed hold nothing; their keys are read but not used.
    uint64_t kk[kMergeKeys];
#pragma unroll
    for (int j = 0; j < kMergeKeys; ++j) {
        const int i = at(j);
        kk[j] = i < total ? __ldcg(&keys[i]) : 0ull;
    }
    if (t == 0) sm.cnt = 0;
    int bad = 0;
    for (int w = wp; w < P.W; w += nw) {
        const int64_t r = b * P.W + w;
        const float s = __ldg(&P.scores[r]);
        const bool fin = P.finished != nullptr && __ldg(&P.finished[r]) != 0;
        int state = 0;
        double M = 0.0, logS = 0.0;
        if (!(s < INFINITY)) {
            bad = 1;  // NaN or +inf
        } else if (s > -INFINITY) {
            if (fin) {
                state = 2;
            } else {
                const BeamStat a = beam_row_sum(P.stats + r * cpr, cpr);
                if (!(a.S <= DBL_MAX)) {
                    bad = 1;  // a NaN or +inf logit
                } else if (a.S > 0.0) {
                    state = 1;
                    M = a.M;
                    logS = log(a.S);
                }
            }
        }
        if (lane == 0) {
            sm.M[w] = M;
            sm.logS[w] = logS;
            sm.s[w] = static_cast<double>(s);
            sm.state[w] = state;
        }
    }
    if (__syncthreads_or(bad)) {
        for (int i = t; i < K; i += nt) {
            P.out_scores[b * K + i] = __uint_as_float(0x7fc00000u);
            P.out_parents[b * K + i] = -1;
            P.out_tokens[b * K + i] = -1;
        }
        return;
    }
    // A bound that K candidates reach, from each thread's best (rounded down to
    // fp32).
    BeamCandidate q[kMergeKeys];
    double best = -INFINITY;
#pragma unroll
    for (int j = 0; j < kMergeKeys; ++j) {
        const int i = at(j);
        q[j] = beam_candidate(sm, i < total ? i / row_keys : 0, kk[j], V);
        best = fmax(best, q[j].c);
    }
    for (int j = kMergeKeys; j * nt < total; ++j) {
        const int i = at(j);
        if (i < total) best = fmax(best, beam_candidate(sm, i / row_keys, __ldcg(&keys[i]), V).c);
    }
    const int kth = cta_kth(ord_i32(__double2float_rd(best)), K, nw, sm.pool).x;
    const double bound = kth == INT_MIN ? -INFINITY : static_cast<double>(from_ord_i32(kth));
    auto keep = [&](double c, uint32_t flat) {
        const int place = atomicAdd(&sm.cnt, 1);
        if (place < kBeamMerge) {
            sm.c[place] = c;
            sm.flat[place] = flat;
        }
    };
    for (int w = t; w < P.W; w += nt)
        if (sm.state[w] == 2 && sm.s[w] >= bound) keep(sm.s[w], static_cast<uint32_t>(w) * V + static_cast<uint32_t>(P.eos));
#pragma unroll
    for (int j = 0; j < kMergeKeys; ++j)
        if (q[j].ok && q[j].c >= bound) keep(q[j].c, q[j].flat);
    for (int j = kMergeKeys; j * nt < total; ++j) {
        const int i = at(j);
        if (i >= total) continue;
        const BeamCandidate x = beam_candidate(sm, i / row_keys, __ldcg(&keys[i]), V);
        if (x.ok && x.c >= bound) keep(x.c, x.flat);
    }
    __syncthreads();
    const int have = sm.cnt;
    if (have > kBeamMerge) {
        beam_merge_ties(P, b, sm);
        return;
    }
    // The candidates differ in w V + token: a candidate's rank is its place.
    for (int i = t; i < have; i += nt) {
        const double c = sm.c[i];
        const uint32_t f = sm.flat[i];
        int rank = 0;
        for (int j = 0; j < have; ++j) rank += sm.c[j] > c || (sm.c[j] == c && sm.flat[j] < f) ? 1 : 0;
        if (rank < K) beam_output(P, b * K + rank, c, f);
    }
    for (int i = have + t; i < K; i += nt) {
        P.out_scores[b * K + i] = -INFINITY;
        P.out_parents[b * K + i] = -1;
        P.out_tokens[b * K + i] = -1;
    }
}

}  // namespace specdec
