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
constexpr int kBeamCand = 512;   // candidates of a chunk held in shared memory
constexpr int kBeamMerge = 1024;  // candidates of a request held in shared memory

struct BeamStat {
    float M;  // largest logit of the chunk (0 if none is above -inf)
    float pad;
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

struct BeamSmem {
    uint64_t cand[kBeamCand];
    uint64_t red[NWARPS];
    double S[NWARPS];
    float M[NWARPS];
    float th[NWARPS];
    int cnt;
};

template <class Tag, int VEC>
__global__ void __launch_bounds__(NT, 4) beam_pass_kernel(const BeamParams P) {
    __shared__ BeamSmem sm;
    using Elem = typename Tag::storage;
    using Ops = VecOps<Tag, VEC>;
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
    uint4 w[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
        const int j = u * NT + t;
        w[u] = minus_inf_vec<Tag>();
        if (j < cnt) w[u] = ld_stream_v4(row + cut.head + static_cast<int64_t>(v0 + j) * VEC);
    }
    // the first chunk also takes the row's head and tail, one element a thread
    float xe = -INFINITY;
    int ie = 0;
    if (sub == 0 && t < cut.head + cut.tail) {
        ie = t < cut.head ? t : cut.head + cut.nv * VEC + (t - cut.head);
        xe = load_scalar<Tag>(row + ie);
    }
    if (t == 0) sm.cnt = 0;
    float tm = xe;
#pragma unroll
    for (int u = 0; u < kU; ++u) tm = fmaxf(tm, Ops::vmax(w[u]));
    // Threshold: each of the A warps that hold vectors offers its n-th largest
    // lane maximum, n = ceil(K / A); the least of these is reached by at least
    // A n >= K elements.
    const int active = max(1, min(NWARPS, (cnt + 31) >> 5));
    const int n = (P.K + active - 1) / active;
    int v = ord_i32(tm), top = 0, nth = 0;
    for (int i = 0; i < n; ++i) {
        nth = __reduce_max_sync(FULL_MASK, v);
        if (i == 0) top = nth;
        const unsigned who = __ballot_sync(FULL_MASK, v == nth);
        if (lane == __ffs(who) - 1) v = INT_MIN;
    }
    if (lane == 0) {
        sm.M[wp] = from_ord_i32(top);
        sm.th[wp] = nth == INT_MIN ? -INFINITY : from_ord_i32(nth);
    }
    __syncthreads();
    float M = sm.M[0], th = sm.th[0];
#pragma unroll
    for (int i = 1; i < NWARPS; ++i) {
        M = fmaxf(M, sm.M[i]);
        if (i < active) th = fminf(th, sm.th[i]);
    }
    const float Mr = M > -INFINITY ? M : 0.0f;  // a chunk of -inf only sums to 0
    constexpr float kLog2e = 1.4426950408889634f;
    double S = 0.0;
    if (xe > -INFINITY || xe != xe) S = static_cast<double>(ex2_sfu((xe - Mr) * kLog2e));
#pragma unroll
    for (int u = 0; u < kU; ++u) {
        float s = 0.0f;
        bool hit = false;
        float e[VEC];
#pragma unroll
        for (int q = 0; q < VEC; ++q) {
            e[q] = Ops::elem(w[u], q);
            s += ex2_sfu((e[q] - Mr) * kLog2e);
        }
        S += static_cast<double>(s);
        const float m = Ops::vmax(w[u]);
        hit = m >= th && m > -INFINITY;
        if (hit) {
#pragma unroll
            for (int q = 0; q < VEC; ++q)
                if (e[q] >= th && e[q] > -INFINITY) {
                    const int at = atomicAdd(&sm.cnt, 1);
                    if (at < kBeamCand) sm.cand[at] = make_key(e[q], cut.head + (v0 + u * NT + t) * VEC + q);
                }
        }
    }
    if (xe >= th && xe > -INFINITY) {
        const int at = atomicAdd(&sm.cnt, 1);
        if (at < kBeamCand) sm.cand[at] = make_key(xe, ie);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) S += __shfl_xor_sync(FULL_MASK, S, o);
    if (lane == 0) sm.S[wp] = S;
    __syncthreads();
    const int64_t chunk = r * P.cpr + sub;
    if (t == 0) {
        double total = sm.S[0];
        for (int i = 1; i < NWARPS; ++i) total += sm.S[i];
        BeamStat st;
        st.M = Mr;
        st.pad = 0.0f;
        st.S = total;
        P.stats[chunk] = st;
    }
    uint64_t* out = P.keys + chunk * P.K;
    const int have = sm.cnt;
    if (have <= kBeamCand) {
        // The keys are distinct: a candidate's rank is its place.
        for (int i = t; i < have; i += NT) {
            const uint64_t key = sm.cand[i];
            int rank = 0;
            for (int j = 0; j < have; ++j) rank += sm.cand[j] > key ? 1 : 0;
            if (rank < P.K) out[rank] = key;
        }
        for (int i = have + t; i < P.K; i += NT) out[i] = 0ull;
    } else {
        // More elements reach the threshold than fit (long runs of equal
        // values): the largest key below the last one found, K times.
        uint64_t last = ~0ull;
        for (int i = 0; i < P.K; ++i) {
            uint64_t best = 0ull;
            if (xe >= th && xe > -INFINITY) {
                const uint64_t k = make_key(xe, ie);
                if (k < last) best = k;
            }
#pragma unroll
            for (int u = 0; u < kU; ++u)
#pragma unroll
                for (int q = 0; q < VEC; ++q) {
                    const float x = Ops::elem(w[u], q);
                    if (x >= th && x > -INFINITY) {
                        const uint64_t k = make_key(x, cut.head + (v0 + u * NT + t) * VEC + q);
                        if (k < last && k > best) best = k;
                    }
                }
            best = block_max_u64(best, sm.red);
            if (t == 0) out[i] = best;
            last = best;
        }
    }
}

struct BeamMergeSmem {
    double M[kMaxBeams];     // largest logit of the row
    double logS[kMaxBeams];  // log sum exp(l - M)
    double s[kMaxBeams];
    int state[kMaxBeams];    // 0: no candidates, 1: streamed, 2: finished
    double c[kBeamMerge];
    uint32_t flat[kBeamMerge];  // w V + token
    double bound[NWARPS];
    uint64_t red[NWARPS];
    int cnt;
};

// c of a key of row w.
__device__ __forceinline__ double beam_value(const BeamMergeSmem& sm, int w, uint64_t key) {
    return (sm.s[w] + (static_cast<double>(key_value(key)) - sm.M[w])) - sm.logS[w];
}

__global__ void __launch_bounds__(NT) beam_merge_kernel(const BeamParams P) {
    __shared__ BeamMergeSmem sm;
    const int t = threadIdx.x, lane = t & 31, wp = t >> 5;
    grid_dependency_wait();
    grid_launch_dependents();
    const int64_t b = blockIdx.x;
    const int K = P.K, cpr = P.cpr;
    if (t == 0) sm.cnt = 0;
    int bad = 0;
    for (int w = wp; w < P.W; w += NWARPS) {
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
                const MaxSum a = warp_row_maxsum(P.stats + r * cpr, cpr, 1.0);
                if (!(a.S <= DBL_MAX)) bad = 1;  // NaN: a NaN or +inf logit
                else if (a.S > 0.0) {
                    state = 1;
                    M = static_cast<double>(a.M);
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
    bad = __syncthreads_or(bad);
    float* os = P.out_scores + b * K;
    int32_t* op = P.out_parents + b * K;
    int32_t* ot = P.out_tokens + b * K;
    if (bad) {
        for (int i = t; i < K; i += NT) {
            os[i] = __uint_as_float(0x7fc00000u);
            op[i] = -1;
            ot[i] = -1;
        }
        return;
    }
    // A chunk's K-th key is a value that K candidates reach: the largest of
    // these bounds the request's K-th best from below.
    const uint64_t* keys = P.keys + b * P.W * cpr * K;
    double bound = -INFINITY;
    for (int i = t; i < P.W * cpr; i += NT) {
        const int w = i / cpr;
        if (sm.state[w] == 1) {
            const uint64_t k = __ldcg(&keys[static_cast<int64_t>(i) * K + K - 1]);
            if (k != 0ull) bound = fmax(bound, beam_value(sm, w, k));
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) bound = fmax(bound, __shfl_xor_sync(FULL_MASK, bound, o));
    if (lane == 0) sm.bound[wp] = bound;
    __syncthreads();
    for (int i = 0; i < NWARPS; ++i) bound = fmax(bound, sm.bound[i]);
    for (int w = t; w < P.W; w += NT)
        if (sm.state[w] == 2 && sm.s[w] >= bound) {
            const int at = atomicAdd(&sm.cnt, 1);  // W <= kBeamMerge
            sm.c[at] = sm.s[w];
            sm.flat[at] = static_cast<uint32_t>(w) * static_cast<uint32_t>(P.V) + static_cast<uint32_t>(P.eos);
        }
    const int total = P.W * cpr * K;
    for (int i = t; i < total; i += NT) {
        const int w = i / (cpr * K);
        if (sm.state[w] != 1) continue;
        const uint64_t k = __ldcg(&keys[i]);
        if (k == 0ull) continue;
        const double c = beam_value(sm, w, k);
        if (c >= bound) {
            const int at = atomicAdd(&sm.cnt, 1);
            if (at < kBeamMerge) {
                sm.c[at] = c;
                sm.flat[at] = static_cast<uint32_t>(w) * static_cast<uint32_t>(P.V) + static_cast<uint32_t>(key_index(k));
            }
        }
    }
    __syncthreads();
    const int have = sm.cnt;
    if (have <= kBeamMerge) {
        for (int i = t; i < have; i += NT) {
            const double c = sm.c[i];
            const uint32_t f = sm.flat[i];
            int rank = 0;
            for (int j = 0; j < have; ++j) rank += sm.c[j] > c || (sm.c[j] == c && sm.flat[j] < f) ? 1 : 0;
            if (rank < K) {
                os[rank] = static_cast<float>(c);
                op[rank] = static_cast<int32_t>(f / static_cast<uint32_t>(P.V));
                ot[rank] = static_cast<int32_t>(f % static_cast<uint32_t>(P.V));
            }
        }
        for (int i = have + t; i < K; i += NT) {
            os[i] = -INFINITY;
            op[i] = -1;
            ot[i] = -1;
        }
        return;
    }
    // More candidates at the bound than fit (runs of equal values over many
    // chunks): the best below the last one found, K times.
    double lc = INFINITY;
    uint32_t lf = 0u;
    __shared__ double red_c[NWARPS];
    __shared__ uint32_t red_f[NWARPS];
    for (int i = 0; i < K; ++i) {
        double bc = -INFINITY;
        uint32_t bf = 0xffffffffu;
        auto offer = [&](double c, uint32_t f) {
            const bool below = c < lc || (c == lc && f > lf);
            if (below && (c > bc || (c == bc && f < bf))) {
                bc = c;
                bf = f;
            }
        };
        for (int w = t; w < P.W; w += NT)
            if (sm.state[w] == 2)
                offer(sm.s[w], static_cast<uint32_t>(w) * static_cast<uint32_t>(P.V) + static_cast<uint32_t>(P.eos));
        for (int j = t; j < total; j += NT) {
            const int w = j / (cpr * K);
            if (sm.state[w] != 1) continue;
            const uint64_t k = __ldcg(&keys[j]);
            if (k != 0ull)
                offer(beam_value(sm, w, k),
                      static_cast<uint32_t>(w) * static_cast<uint32_t>(P.V) + static_cast<uint32_t>(key_index(k)));
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const double c = __shfl_xor_sync(FULL_MASK, bc, o);
            const uint32_t f = __shfl_xor_sync(FULL_MASK, bf, o);
            if (c > bc || (c == bc && f < bf)) {
                bc = c;
                bf = f;
            }
        }
        if (lane == 0) {
            red_c[wp] = bc;
            red_f[wp] = bf;
        }
        __syncthreads();
        bc = red_c[0];
        bf = red_f[0];
        for (int q = 1; q < NWARPS; ++q)
            if (red_c[q] > bc || (red_c[q] == bc && red_f[q] < bf)) {
                bc = red_c[q];
                bf = red_f[q];
            }
        __syncthreads();
        lc = bc;
        lf = bf;
        if (t == 0) {
            os[i] = static_cast<float>(bc);
            op[i] = static_cast<int32_t>(bf / static_cast<uint32_t>(P.V));
            ot[i] = static_cast<int32_t>(bf % static_cast<uint32_t>(P.V));
        }
    }
}

}  // namespace specdec
