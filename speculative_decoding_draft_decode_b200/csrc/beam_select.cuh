// beam_select.cuh — one step of beam search or draft-tree expansion: the K
// best continuations of every request's W beams over the vocabulary.
//
// Handbook page, "EAGLE" (EAGLE-2 grows its draft tree by the cumulative
// probability of the branches) and "Medusa" (candidates form a tree): the
// level's candidates are every (beam w, token v) with
//   c = s_w + l_wv - log sum_v' exp(l_wv'),
// and the K largest are kept, equal values in order of w V + v.
//
// beam_stream reads the logits once.  A warp takes a segment of a row, tile by
// tile (128 vectors of 16 bytes, 4 a lane), and keeps sum exp(l - ref) and every
// tile's largest logit.  Nothing is selected here, so warps need neither
// thresholds nor one another.  Bound by load latency together with the
// special-function unit: 64 x 8 rows of 128256 bf16 take 26.5 us (5.0 TB/s), the
// same with 4 to 6 CTAs per SM, with a tile loaded ahead, or with part of the
// exponentials as polynomials.
// beam_merge, one CTA per request: the rows' sums, then the K best tiles by (c
// of the largest logit, position).  An element of any other tile has K elements
// before it (the largest ones of these K tiles: greater, or equal and earlier),
// so only K tiles are read again (up to 16 if that many reach the bound).  Values
// are ordered in fp64.  About 5 us, a chain of dependent steps.  Every sum has a
// fixed order: results do not vary from run to run.
#pragma once

#include <cuda_runtime.h>
#include <float.h>
#include <limits.h>
#include <stdint.h>

#include <type_traits>

#include "device_utils.cuh"
#include "verify_common.cuh"
#include "verify_pass1.cuh"

namespace specdec {

constexpr int kMaxBeams = 32;    // beams per request, and beams selected
constexpr int kTileU = 4;        // 16-byte vectors of a tile per lane
constexpr int kTileVecs = 32 * kTileU;

struct BeamStat {
    double M;  // a value near the segment's largest logit
    double S;  // sum exp(l - M) over the segment; NaN for a NaN or +inf logit
};

struct BeamParams {
    const void* logits;
    int64_t row_stride;
    const float* scores;      // [B, W] cumulative log probabilities; -inf: no hypothesis
    const int32_t* finished;  // [B, W] or null
    int B, W, K, V;
    int eos;
    int tiles;        // tiles per row
    int seg_tiles;    // tiles of a segment
    int segs;         // segments per row
    BeamStat* stats;  // [B W, segs]
    float* peaks;     // [B W, tiles] largest logit of each tile (-inf: none above it)
    float* out_scores;  // [B, K]
    int32_t* out_parents;
    int32_t* out_tokens;
};

// Rows that are streamed: a hypothesis with a finite score that is not
// finished.
__device__ __forceinline__ bool beam_streams(const BeamParams& P, int64_t r) {
    const float s = __ldg(&P.scores[r]);
    const int f = P.finished != nullptr ? __ldg(&P.finished[r]) : 0;
    return s > -INFINITY && s < INFINITY && f == 0;
}

// The vectors of a row: elements before the first 16-byte boundary (the
// head), nv full vectors, and the elements behind them (the tail).  Rows need
// no alignment beyond their element's.  The head belongs to the first tile and
// the tail to the last one.
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

// The K-th largest of 32 ordered values in shared memory (INT_MIN: none), for
// every lane of the warp.  Each lane counts the values before its own.
__device__ __forceinline__ int pool_kth(const int* pool, int K) {
    const int lane = threadIdx.x & 31;
    const int p = pool[lane];
    int rank = 0;
#pragma unroll
    for (int i = 0; i < 32; i += 4) {
        const int4 x = *reinterpret_cast<const int4*>(&pool[i]);
        rank += (x.x > p || (x.x == p && i < lane) ? 1 : 0) + (x.y > p || (x.y == p && i + 1 < lane) ? 1 : 0) +
                (x.z > p || (x.z == p && i + 2 < lane) ? 1 : 0) + (x.w > p || (x.w == p && i + 3 < lane) ? 1 : 0);
    }
    const unsigned who = __ballot_sync(FULL_MASK, rank == K - 1);
    return __shfl_sync(FULL_MASK, p, __ffs(who) - 1);
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

constexpr float kLog2e = 1.4426950408889634f;

// A tile as a lane holds it: vectors [j, j + 128) of the row, and in the first
// and last tile one element of the head or tail (xe, number ie; -inf: none).
template <class Tag, int VEC>
struct BeamTile {
    using Elem = typename Tag::storage;
    uint4 w[kTileU];
    __device__ __forceinline__ void load(const Elem* row, const RowCut& cut, int tile) {
        const int lane = threadIdx.x & 31, j = tile * kTileVecs;
        const Elem* p = row + cut.head + static_cast<int64_t>(j + lane) * VEC;
        if (j + kTileVecs <= cut.nv) {
#pragma unroll
            for (int u = 0; u < kTileU; ++u) w[u] = ld_stream_v4(p + u * 32 * VEC);
        } else {
#pragma unroll
            for (int u = 0; u < kTileU; ++u) {
                w[u] = minus_inf_vec<Tag>();
                if (j + u * 32 + lane < cut.nv) w[u] = ld_stream_v4(p + u * 32 * VEC);
            }
        }
    }
    // The largest element (NaN ignored).
    __device__ __forceinline__ float most() const {
        if constexpr (sizeof(Elem) == 2) {
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
};

// This lane's element of the head (first tile) or tail (last tile): its value,
// -inf if it has none, and its number.  Head and tail have at most 7 elements.
template <class Tag>
__device__ __forceinline__ float beam_end(const typename Tag::storage* row, const RowCut& cut, int V, bool first,
                                          bool last, int& ie) {
    const int lane = threadIdx.x & 31;
    ie = -1;
    if (first && lane < cut.head) ie = lane;
    if (last && lane >= 8 && lane < 8 + cut.tail) ie = V - cut.tail + lane - 8;
    return ie >= 0 ? load_scalar<Tag>(row + ie) : -INFINITY;
}

// Each term is taken as 2^(l c - E) with one rounding in the exponent: c is
// log2 e in fp32 and E = ref c in fp32, so the terms count from E / c exactly,
// and c's own error (2^-26 relative) only weighs the distance from there.  The
// largest logit's term is then 2^(at most E's rounding), which must stay near 1:
// below 2^16 that is 2^(2^-8), from 2^31 on it could leave fp32.  From 2^16 on a
// term is 2^((l - ref) c): l - ref is exact for every term that does not vanish
// (l lies between ref / 2 and 2 ref), so there is one rounding here too.
__device__ __forceinline__ bool beam_far(float ref) { return !(fabsf(ref) < 65536.0f); }
__device__ __forceinline__ double beam_ref(float ref) {
    return beam_far(ref) ? static_cast<double>(ref)
                         : static_cast<double>(__fmul_rn(ref, kLog2e)) * (1.0 / static_cast<double>(kLog2e));
}
__device__ __forceinline__ float beam_term(float x, float ref) {
    return ex2_sfu(beam_far(ref) ? (x - ref) * kLog2e : __fmaf_rn(x, kLog2e, -__fmul_rn(ref, kLog2e)));
}

// A reference as the sums use it.
struct BeamRef {
    uint64_t minus;  // -E, or -ref where that is far, twice
    bool far;
    __device__ __forceinline__ explicit BeamRef(float ref) : far(beam_far(ref)) {
        const float x = far ? -ref : -__fmul_rn(ref, kLog2e);
        minus = f32x2(x, x);
    }
};

// The sum of a tile's terms, fp32: 2 x 16 (bf16) or 2 x 8 (fp32) of them.
template <class Tag, int VEC>
__device__ __forceinline__ float beam_sum(const uint4 (&w)[kTileU], const BeamRef& ref) {
    const uint64_t scale = f32x2(kLog2e, kLog2e);
    uint64_t s = f32x2(0.0f, 0.0f);
    auto sum = [&](auto exponent) {
#pragma unroll
        for (int u = 0; u < kTileU; ++u)
#pragma unroll
            for (int q = 0; q < VEC; q += 2) {
                const float2 e = f32x2_get(exponent(f32x2(VecOps<Tag, VEC>::elem(w[u], q), VecOps<Tag, VEC>::elem(w[u], q + 1))));
                s = f32x2_add(s, f32x2(ex2_sfu(e.x), ex2_sfu(e.y)));
            }
    };
    if (ref.far) {
        const uint64_t zero = f32x2(0.0f, 0.0f);
        sum([&](uint64_t x) { return f32x2_fma(f32x2_add(x, ref.minus), scale, zero); });
    } else {
        sum([&](uint64_t x) { return f32x2_fma(x, scale, ref.minus); });
    }
    const float2 r = f32x2_get(s);
    return r.x + r.y;
}

// What a large term misses by the special-function unit and the rounding of its
// exponent.
__device__ __noinline__ double beam_miss(float x, float ref) {
    return exp(static_cast<double>(x) - beam_ref(ref)) - static_cast<double>(beam_term(x, ref));
}

// The same sum without its roundings: every term is split on a grid of 2^-20
// (terms are at most 2^(2^-8) here, so the grid parts add exactly up to 16 and the
// rest is at most 2^-21), and the lane's largest term (of logit `most`), if it is from `from`
// on, is taken in fp64.  A row's sum errs by its few large terms (the many small
// ones average out), so the tiles that hold candidates are summed this way.  Not
// for far references.
template <class Tag, int VEC>
__device__ __forceinline__ double beam_sum_exact(const uint4 (&w)[kTileU], float most, float ref, float from) {
    const float E = __fmul_rn(ref, kLog2e);
    const uint64_t minus = f32x2(-E, -E), scale = f32x2(kLog2e, kLog2e), one = f32x2(-1.0f, -1.0f);
    const uint64_t up = f32x2(12.0f, 12.0f), down = f32x2(-12.0f, -12.0f);
    uint64_t hi = f32x2(0.0f, 0.0f), lo = hi;
#pragma unroll
    for (int u = 0; u < kTileU; ++u) {
#pragma unroll
        for (int q = 0; q < VEC; q += 2) {
            const float2 y = f32x2_get(
                f32x2_fma(f32x2(VecOps<Tag, VEC>::elem(w[u], q), VecOps<Tag, VEC>::elem(w[u], q + 1)), scale, minus));
            const uint64_t e = f32x2(ex2_sfu(y.x), ex2_sfu(y.y));
            const uint64_t h = f32x2_add(f32x2_add(e, up), down);
            hi = f32x2_add(hi, h);
            lo = f32x2_add(lo, f32x2_fma(h, one, e));
        }
    }
    const double miss = most >= from ? beam_miss(most, ref) : 0.0;
    const float2 h = f32x2_get(hi), l = f32x2_get(lo);
    return (static_cast<double>(h.x) + static_cast<double>(h.y)) +
           (static_cast<double>(l.x) + static_cast<double>(l.y)) + miss;
}
constexpr float kBeamLarge = 4.0f;  // how far below a tile's largest logit a term counts as large

__device__ __forceinline__ double warp_sum_f64(double v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(FULL_MASK, v, o);
    return v;
}

// The reference of values up to m: the multiple of 8 from m on, so that most
// segments of a row share it and their sums add as they are.
__device__ __forceinline__ float beam_up(float m) { return beam_far(m) ? fmaxf(m, -FLT_MAX) : 8.0f * ceilf(m * 0.125f); }

// A sum over to another reference.
__device__ __noinline__ double beam_carry(double S, float from, float to) {
    return S == 0.0 ? 0.0 : S * exp(beam_ref(from) - beam_ref(to));
}

// A warp's segment of row r.
template <class Tag, int VEC>
__device__ __forceinline__ void beam_stream(const BeamParams& P, int64_t r, int seg) {
    using Elem = typename Tag::storage;
    const int lane = threadIdx.x & 31;
    const int t0 = seg * P.seg_tiles, t1 = min(t0 + P.seg_tiles, P.tiles);
    const Elem* row = static_cast<const Elem*>(P.logits) + r * P.row_stride;
    const RowCut cut = cut_row<Tag, VEC>(row, P.V);
    float* peaks = P.peaks + r * P.tiles;
    BeamTile<Tag, VEC> a;
    if (!beam_streams(P, r)) return;  // warp-uniform
    a.load(row, cut, t0);
    int ie;
    const float xe = beam_end<Tag>(row, cut, P.V, t0 == 0, t1 == P.tiles, ie);
    // A head element counts to the segment's first tile's largest logit, a tail
    // element to the last one's.
    const bool is_head = ie >= 0 && ie < cut.head;
    const float x0 = is_head ? xe : -INFINITY, x1 = is_head ? -INFINITY : xe;
    auto warp_max = [](float m) { return from_ord_i32(__reduce_max_sync(FULL_MASK, ord_i32(m))); };
    float m = warp_max(fmaxf(fmaxf(a.most(), x0), t0 + 1 == t1 ? x1 : -INFINITY));
    float ref = beam_up(m);
    BeamRef use(ref);
    double S = 0.0;
    for (int t = t0;;) {
        float s = beam_sum<Tag, VEC>(a.w, use);
        if (lane == 0) peaks[t] = m;
        if (m > ref) {  // rare: the terms again, against a new reference
            const float up = beam_up(m);
            S = beam_carry(S, ref, up);
            ref = up;
            use = BeamRef(ref);
            s = beam_sum<Tag, VEC>(a.w, use);
        }
        S += static_cast<double>(s);
        if (++t >= t1) break;
        a.load(row, cut, t);
        m = warp_max(t + 1 == t1 ? fmaxf(a.most(), x1) : a.most());  // on its way while the terms are summed
    }
    if (ie >= 0) S += static_cast<double>(beam_term(xe, ref));
    S = warp_sum_f64(S);
    if (lane == 0) {
        BeamStat st;
        st.M = beam_ref(ref);
        st.S = S;
        P.stats[r * P.segs + seg] = st;
    }
}

// ---------------------------------------------------------------------------
// The request's merge.
// ---------------------------------------------------------------------------
constexpr int kMergePeaks = 8;    // tiles whose largest logit a thread holds in registers
constexpr int kMergeTiles = 512;  // tiles of a request that are ranked in shared memory
constexpr int kMergeCand = 1024;  // candidates of a request that are ranked in shared memory

struct BeamMergeSmem {
    double M[kMaxBeams];     // near the row's largest logit
    double logS[kMaxBeams];  // log sum exp(l - M)
    double s[kMaxBeams];
    double add[kMaxBeams];   // s - M - logS
    double S[kMaxBeams];     // sum exp(l - M)
    float near[kMaxBeams];   // logits nearer to zero may share a value (see beam_near)
    long long fix[kMaxBeams];  // what its roundings are known to have cost, in units of 2^-52
    int state[kMaxBeams];    // 0: no candidates, 1: streamed, 2: finished
    double c[kMergeCand];    // tiles, then candidates
    uint32_t id[kMergeCand];    // their names
    double tile_c[kMaxBeams];   // the K best tiles
    uint32_t tile_id[kMaxBeams];
    __align__(16) int pool[32];
    double red_c[NWARPS];
    uint32_t red_id[NWARPS];
    float red_x[NWARPS];
    int tiles, cands;
    int close;               // a logit that may share its value was seen
};

constexpr double kFixUnit = 4503599627370496.0;  // 2^52: whole numbers add in any order

// c of a logit of row w: one addition, or, where M is so large that s and logS
// would be lost beside it, the difference of the large numbers first.
constexpr double kBeamPlain = 1e6;
__device__ __forceinline__ double beam_value(const BeamMergeSmem& sm, int w, float x) {
    const double M = sm.M[w];
    if (fabs(M) < kBeamPlain) return static_cast<double>(x) + sm.add[w];
    return (sm.s[w] + (static_cast<double>(x) - M)) - sm.logS[w];
}

// Candidates are named (w << 24) + token and tiles (w << 16) + tile: both in
// the order of w V + token.
constexpr int kTokenBits = 24, kTileBits = 16;

// Two logits of a row may have one value in 64 bits: logits next to zero, or
// scores that are large numbers.  They keep the logits' order.  Every step of a
// value rounds by at most 2^-53 of 2 (|s| + |M| + 64 + |x|) (log S is below 32),
// while neighbours of x in fp32 lie 2^-24 |x| apart, so it takes an |x| below
// 2^-22 (|s| + |M| + 64); where none was seen the names alone order equal values.
__device__ __forceinline__ float beam_near(double s, double M) {
    return static_cast<float>((fabs(s) + fabs(M) + 64.0) * 0x1p-22);
}

// Whether a value c of logit x, named id, stands before d of y, named jd.  CLOSE:
// different logits may share a value.  BITS: of an element or a tile in a name.
template <bool CLOSE, int BITS>
__device__ __forceinline__ bool beam_before(double c, uint32_t id, float x, double d, uint32_t jd, float y) {
    if (CLOSE) {
        if (c != d) return c > d;
        return x != y && (id >> BITS) == (jd >> BITS) ? x > y : id < jd;
    }
    return c > d || (c == d && id < jd);
}

// A lane's part of a row's n segments: kSegs of them, 32 apart, from i0 on.
constexpr int kSegs = 4;
struct BeamSegs {
    double M[kSegs], S[kSegs];
    __device__ __forceinline__ void load(const BeamStat* p, int i0, int n) {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int j = 0; j < kSegs; ++j) {
            const int i = i0 + j * 32 + lane;
            M[j] = -DBL_MAX;
            S[j] = 0.0;
            if (i < n) {
                M[j] = __ldcg(&p[i].M);
                S[j] = __ldcg(&p[i].S);
            }
        }
    }
};

// A row's sum from its segments' (x: the first 32 kSegs), each against the
// largest reference of those loaded with it.  Warp-collective.
__device__ __forceinline__ BeamStat beam_row_sum(const BeamStat* p, int n, BeamSegs x) {
    BeamStat acc;
    acc.M = -DBL_MAX;
    acc.S = 0.0;
    for (int i0 = 0;;) {
        double M = -DBL_MAX;  // a segment's reference is an fp32 value's, so fp32 tells them apart
#pragma unroll
        for (int j = 0; j < kSegs; ++j)
            if (x.S[j] != 0.0) M = fmax(M, x.M[j]);
        const int o32 = ord_i32(static_cast<float>(M)), most = __reduce_max_sync(FULL_MASK, o32);
        double top = __shfl_sync(FULL_MASK, M, __ffs(__ballot_sync(FULL_MASK, o32 == most)) - 1);
        if (acc.S != 0.0) top = fmax(top, acc.M);
        double S = 0.0;
#pragma unroll
        for (int j = 0; j < kSegs; ++j)
            if (x.S[j] != 0.0) S += x.M[j] != top ? x.S[j] * exp(x.M[j] - top) : x.S[j];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) S += __shfl_xor_sync(FULL_MASK, S, o);
        if (acc.S != 0.0) S += acc.M != top ? acc.S * exp(acc.M - top) : acc.S;
        acc.M = top;
        acc.S = S;
        i0 += 32 * kSegs;
        if (i0 >= n) return acc;
        x.load(p, i0, n);
    }
}

// The best candidate (or tile) of one per thread, id kBeamNone: none.
// CTA-collective; every thread gets it.
constexpr uint32_t kBeamNone = 0xffffffffu;  // no name: tokens of beam 255
struct BeamBest {
    double c;
    uint32_t id;
    float x;
};
template <bool CLOSE, int BITS>
__device__ __forceinline__ bool beam_before(const BeamBest& a, const BeamBest& b) {
    return beam_before<CLOSE, BITS>(a.c, a.id, a.x, b.c, b.id, b.x);
}
// `x` if it is the best so far behind the last one found.
template <bool CLOSE, int BITS>
__device__ __forceinline__ void beam_next(const BeamBest& last, const BeamBest& x, BeamBest& best) {
    if (beam_before<CLOSE, BITS>(last, x) && beam_before<CLOSE, BITS>(x, best)) best = x;
}
template <bool CLOSE, int BITS>
__device__ __forceinline__ BeamBest beam_block_best(BeamBest x, BeamMergeSmem& sm) {
    const int lane = threadIdx.x & 31, wp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const BeamBest y = {__shfl_xor_sync(FULL_MASK, x.c, o), __shfl_xor_sync(FULL_MASK, x.id, o),
                            __shfl_xor_sync(FULL_MASK, x.x, o)};
        if (beam_before<CLOSE, BITS>(y, x)) x = y;
    }
    if (lane == 0) {
        sm.red_c[wp] = x.c;
        sm.red_id[wp] = x.id;
        sm.red_x[wp] = x.x;
    }
    __syncthreads();
    for (int q = 0; q < NWARPS; ++q) {
        const BeamBest y = {sm.red_c[q], sm.red_id[q], sm.red_x[q]};
        if (beam_before<CLOSE, BITS>(y, x)) x = y;
    }
    __syncthreads();
    return x;
}

__device__ __forceinline__ void beam_output(const BeamParams& P, int64_t at, double c, uint32_t id) {
    P.out_scores[at] = static_cast<float>(c);
    P.out_parents[at] = static_cast<int32_t>(id >> kTokenBits);
    P.out_tokens[at] = static_cast<int32_t>(id & ((1u << kTokenBits) - 1u));
}

// The K best tiles of more than kMergeTiles at the bound (runs of equal
// values): the best one behind the last one found, K times.
template <bool CLOSE>
__device__ __noinline__ int beam_many_tiles(const BeamParams& P, const float* peaks, BeamMergeSmem& sm) {
    const int total = P.W * P.tiles;
    BeamBest last = {INFINITY, 0u, 0.0f};
    for (int i = 0; i < P.K; ++i) {
        BeamBest best = {-INFINITY, kBeamNone, 0.0f};
        for (int j = threadIdx.x; j < total; j += NT) {
            const int w = j / P.tiles;
            const float m = sm.state[w] == 1 ? __ldcg(&peaks[j]) : -INFINITY;
            if (!(m > -INFINITY)) continue;
            const uint32_t id = (static_cast<uint32_t>(w) << kTileBits) + static_cast<uint32_t>(j - w * P.tiles);
            beam_next<CLOSE, kTileBits>(last, {beam_value(sm, w, m), id, m}, best);
        }
        last = beam_block_best<CLOSE, kTileBits>(best, sm);
        if (last.id == kBeamNone) return i;
        if (threadIdx.x == 0) {
            sm.tile_c[i] = last.c;
            sm.tile_id[i] = last.id;
        }
    }
    return P.K;
}

// Rows of at most kMendTiles tiles have their sums mended.  A row of 1000
// logits N(0, 2^2) with one at +8 then errs by 1e-8 (standard deviation) instead
// of 1e-7; one of 128256 errs by 7e-9 without, and mending would cost a merge
// 2.9 us (14.6 against 11.7 us at 16 x 4 rows of 128256 bf16).
constexpr int kMendTiles = 16;
// Bounds taken before that are lowered by more than values can fall with it (a
// sum's error is below 4e-6, and a value's last place moves).
__device__ __forceinline__ double beam_slack(double bound) { return bound - (1e-5 + 1e-14 * fabs(bound)); }

// One of the K best tiles, as a warp reads it again.
template <class Tag, int VEC>
struct BeamPlace {
    using Elem = typename Tag::storage;
    BeamTile<Tag, VEC> a;
    RowCut cut;
    int w, tile, ie;  // ie: this lane's element of the row's head or tail, -1 if it has none
    float xe;
    __device__ __forceinline__ void load(const BeamParams& P, int64_t b, const BeamMergeSmem& sm, int i) {
        w = static_cast<int>(sm.tile_id[i] >> kTileBits);
        tile = static_cast<int>(sm.tile_id[i] & ((1u << kTileBits) - 1u));
        const Elem* row = static_cast<const Elem*>(P.logits) + (b * P.W + w) * P.row_stride;
        cut = cut_row<Tag, VEC>(row, P.V);
        a.load(row, cut, tile);
        xe = beam_end<Tag>(row, cut, P.V, tile == 0, tile == P.tiles - 1, ie);
    }
    // The best value among this lane's elements.
    __device__ __forceinline__ double best(const BeamMergeSmem& sm) const {
        const float m = fmaxf(a.most(), xe);
        return m > -INFINITY ? beam_value(sm, w, m) : -INFINITY;
    }
    // The tile's sum again, exactly, against what the streaming pass added for
    // it: with the reference it had by then, from the peaks of its segment.
    __device__ __forceinline__ void mend(const BeamParams& P, int64_t b, BeamMergeSmem& sm) const {
        const int lane = threadIdx.x & 31;
        const float* peaks = P.peaks + (b * P.W + w) * P.tiles;
        const int t0 = tile - tile % P.seg_tiles;
        const float p = t0 + lane <= tile ? __ldcg(&peaks[t0 + lane]) : -INFINITY;  // seg_tiles <= 4
        const float m = __shfl_sync(FULL_MASK, p, tile - t0);
        const float ref = beam_up(from_ord_i32(__reduce_max_sync(FULL_MASK, ord_i32(p))));
        if (beam_far(ref)) return;
        double d = beam_sum_exact<Tag, VEC>(a.w, a.most(), ref, m - kBeamLarge) - static_cast<double>(beam_sum<Tag, VEC>(a.w, BeamRef(ref)));
        d = warp_sum_f64(d);
        const double at = beam_ref(ref);
        if (at != sm.M[w]) d *= exp(at - sm.M[w]);
        if (lane == 0)
            atomicAdd(reinterpret_cast<unsigned long long*>(&sm.fix[w]),
                      static_cast<unsigned long long>(__double2ll_rn(d * kFixUnit)));
    }
    // Every element of this lane with a value of at least `bound`: f(c, id, x,
    // whether another logit may share the value).
    template <class F>
    __device__ __forceinline__ void look(const BeamMergeSmem& sm, double bound, F f) const {
        const int lane = threadIdx.x & 31;
        // A logit below this has a value below the bound (the margin covers the
        // roundings); what passes is compared in fp64.
        const float at = __double2float_rd(bound - sm.add[w]);
        const float slack = 1e-6f * (fabsf(at) + fabsf(static_cast<float>(bound)) + fabsf(static_cast<float>(sm.add[w])));
        const float low = bound > -INFINITY ? fmaxf(at - slack, -FLT_MAX) : -FLT_MAX;
        auto offer = [&](float x, int e) {
            if (x >= low) {
                const double c = beam_value(sm, w, x);
                if (c >= bound)
                    f(c, (static_cast<uint32_t>(w) << kTokenBits) + static_cast<uint32_t>(e), x, fabsf(x) < sm.near[w]);
            }
        };
        if (ie >= 0) offer(xe, ie);
#pragma unroll
        for (int u = 0; u < kTileU; ++u) {
            if (!(VecOps<Tag, VEC>::vmax(a.w[u]) >= low)) continue;
            const int e0 = cut.head + (tile * kTileVecs + u * 32 + lane) * VEC;
#pragma unroll
            for (int q = 0; q < VEC; ++q) offer(VecOps<Tag, VEC>::elem(a.w[u], q), e0 + q);
        }
    }
};

// A bound that K candidates reach, from the best one of each thread (rounded
// down to fp32): the K-th largest of the 32 values that the warps' 4 best lanes
// make up; -inf if there are fewer.  CTA-collective.
__device__ __forceinline__ double beam_bound(double best, int K, BeamMergeSmem& sm) {
    const int lane = threadIdx.x & 31, wp = threadIdx.x >> 5;
    constexpr int kEach = 32 / NWARPS;
    int o = ord_i32(__double2float_rd(best)), mine = INT_MIN;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int x = __reduce_max_sync(FULL_MASK, o);
        if (lane == i) mine = x;
        const unsigned who = __ballot_sync(FULL_MASK, o == x);
        if (lane == __ffs(who) - 1) o = INT_MIN;
    }
    if (lane < kEach) sm.pool[wp * kEach + lane] = mine;
    __syncthreads();
    const int kth = pool_kth(sm.pool, K);
    __syncthreads();  // the pool may be written again
    return kth == INT_MIN ? -INFINITY : static_cast<double>(from_ord_i32(kth));
}

// This thread's finished beam, if it has one (W <= kMaxBeams <= NT).
__device__ __forceinline__ bool beam_ended(const BeamParams& P, const BeamMergeSmem& sm) {
    return static_cast<int>(threadIdx.x) < P.W && sm.state[threadIdx.x] == 2;
}
template <class F>
__device__ __forceinline__ void beam_look_ended(const BeamParams& P, const BeamMergeSmem& sm, double bound, F f) {
    if (beam_ended(P, sm) && sm.s[threadIdx.x] >= bound)
        f(sm.s[threadIdx.x], (threadIdx.x << kTokenBits) + static_cast<uint32_t>(P.eos), 0.0f, false);
}

// Every candidate of the n best tiles and the finished beams with a value of at
// least `bound`.  A warp per tile.
template <class Tag, int VEC, class F>
__device__ __forceinline__ void beam_visit(const BeamParams& P, int64_t b, int n, double bound, const BeamMergeSmem& sm, F f) {
    BeamPlace<Tag, VEC> x;
    for (int i = threadIdx.x >> 5; i < n; i += NWARPS) {
        x.load(P, b, sm, i);
        x.look(sm, bound, f);
    }
    beam_look_ended(P, sm, bound, f);
}

// The bound of the best candidate of every thread over the n tiles.
template <class Tag, int VEC>
__device__ __noinline__ double beam_visit_bound(const BeamParams& P, int64_t b, int n, BeamMergeSmem& sm) {
    double best = beam_ended(P, sm) ? sm.s[threadIdx.x] : -INFINITY;
    BeamPlace<Tag, VEC> x;
    for (int i = threadIdx.x >> 5; i < n; i += NWARPS) {
        x.load(P, b, sm, i);
        best = fmax(best, x.best(sm));
    }
    return beam_bound(best, P.K, sm);
}

// The outputs of more than kMergeCand candidates: the best one behind the last
// one found, K times.
template <class Tag, int VEC, bool CLOSE>
__device__ __noinline__ void beam_many_candidates(const BeamParams& P, int64_t b, int n, double bound, BeamMergeSmem& sm) {
    BeamBest last = {INFINITY, 0u, 0.0f};
    for (int i = 0; i < P.K; ++i) {
        BeamBest best = {-INFINITY, kBeamNone, 0.0f};
        beam_visit<Tag, VEC>(P, b, n, bound, sm, [&](double c, uint32_t id, float x, bool) {
            beam_next<CLOSE, kTokenBits>(last, {c, id, x}, best);
        });
        last = beam_block_best<CLOSE, kTokenBits>(best, sm);
        if (threadIdx.x == 0) beam_output(P, b * P.K + i, last.c, last.id);
    }
}

// The rows' normalisers: sum(w) is the row's sum.  True (for the whole CTA) if
// the request is undefined; its outputs are then written.
template <class F>
__device__ __forceinline__ bool beam_rows(const BeamParams& P, int64_t b, BeamMergeSmem& sm, F sum) {
    const int lane = threadIdx.x & 31;
    int bad = 0;
    for (int w = threadIdx.x >> 5; w < P.W; w += NWARPS) {
        const float s = __ldg(&P.scores[b * P.W + w]);
        const bool fin = P.finished != nullptr && __ldg(&P.finished[b * P.W + w]) != 0;
        int state = 0;
        double M = 0.0, S = 1.0, logS = 0.0;
        if (!(s < INFINITY)) {
            bad = 1;  // NaN or +inf
        } else if (s > -INFINITY) {
            if (fin) {
                state = 2;
            } else {
                const BeamStat a = sum(w);
                if (!(a.S <= DBL_MAX)) {
                    bad = 1;  // a NaN or +inf logit
                } else if (a.S > 0.0) {
                    state = 1;
                    M = a.M;
                    S = a.S;
                    logS = log(S);
                }
            }
        }
        if (lane == 0) {
            sm.M[w] = M;
            sm.logS[w] = logS;
            sm.s[w] = static_cast<double>(s);
            sm.add[w] = (static_cast<double>(s) - M) - logS;
            sm.S[w] = S;
            sm.near[w] = beam_near(static_cast<double>(s), M);
            sm.fix[w] = 0;
            sm.state[w] = state;
        }
    }
    if (!__syncthreads_or(bad)) return false;
    for (int i = threadIdx.x; i < P.K; i += NT) {
        P.out_scores[b * P.K + i] = __uint_as_float(0x7fc00000u);
        P.out_parents[b * P.K + i] = -1;
        P.out_tokens[b * P.K + i] = -1;
    }
    return true;
}

// The sums of the rows whose tiles have been looked at again.  CTA-collective.
__device__ __forceinline__ void beam_mend_rows(const BeamParams& P, BeamMergeSmem& sm) {
    __syncthreads();
    for (int w = threadIdx.x; w < P.W; w += NT)
        if (sm.state[w] == 1 && sm.fix[w] != 0) {
            const double logS = log(sm.S[w] + static_cast<double>(sm.fix[w]) / kFixUnit);
            sm.logS[w] = logS;
            sm.add[w] = (sm.s[w] - sm.M[w]) - logS;
        }
    __syncthreads();
}

// How many of n candidates (or tiles) in shared memory stand before one.
__device__ __forceinline__ int beam_place(const BeamMergeSmem& sm, int n, double c, uint32_t id) {
    int rank = 0;
#pragma unroll 4
    for (int i = 0; i < n; ++i) rank += beam_before<false, 0>(sm.c[i], sm.id[i], 0.0f, c, id, 0.0f) ? 1 : 0;
    return rank;
}
// The same where different logits may share a value: element i of row w of
// `logits` is that of name (w << BITS) + i.  Keeping the logits beside their
// values instead costs every call more (16 x 4 rows of 128256 bf16 13.0 us instead
// of 12.3).
__device__ __forceinline__ float beam_logit(float x) { return x; }
__device__ __forceinline__ float beam_logit(uint16_t x) { return bf16_bits_to_float(x); }
template <class T, int BITS>
__device__ __noinline__ int beam_place_close(const T* logits, int64_t stride, const BeamMergeSmem& sm, int n, double c,
                                             uint32_t id) {
    auto logit = [&](uint32_t i) { return beam_logit(logits[(i >> BITS) * stride + (i & ((1u << BITS) - 1u))]); };
    int rank = 0;
    for (int i = 0; i < n; ++i) {
        const double d = sm.c[i];
        const uint32_t jd = sm.id[i];
        const bool ask = d == c && jd != id && (jd >> BITS) == (id >> BITS);
        rank += beam_before<true, BITS>(d, jd, ask ? logit(jd) : 0.0f, c, id, ask ? logit(id) : 0.0f) ? 1 : 0;
    }
    return rank;
}

// The outputs from at most kMergeCand candidates in shared memory.
template <class Elem>
__device__ __forceinline__ void beam_rank(const BeamParams& P, int64_t b, BeamMergeSmem& sm, int cands) {
    const int t = threadIdx.x, K = P.K;
    // A candidate's rank is its place.  Among many, those below the bound of
    // the threads' best ones have none.
    double own_c[kMergeCand / NT];
    uint32_t own_id[kMergeCand / NT];
    double e = -INFINITY;
#pragma unroll
    for (int j = 0; j < kMergeCand / NT; ++j) {
        const int i = t + j * NT;
        own_c[j] = -INFINITY;
        own_id[j] = 0u;
        if (i < cands) {
            own_c[j] = sm.c[i];
            own_id[j] = sm.id[i];
            e = fmax(e, own_c[j]);
        }
    }
    int ranked = cands;
    if (cands > 64) {
        const double least = beam_bound(e, K, sm);  // its barriers: every candidate has been read
        if (t == 0) sm.cands = 0;
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kMergeCand / NT; ++j) {
            if (!(own_c[j] >= least)) own_c[j] = -INFINITY;
            if (own_c[j] > -INFINITY) {
                const int at = atomicAdd(&sm.cands, 1);
                sm.c[at] = own_c[j];
                sm.id[at] = own_id[j];
            }
        }
        __syncthreads();
        ranked = sm.cands;
    }
#pragma unroll
    for (int j = 0; j < kMergeCand / NT; ++j) {
        if (!(own_c[j] > -INFINITY)) continue;
        int rank = beam_place(sm, ranked, own_c[j], own_id[j]);
        if (sm.close != 0)
            rank = beam_place_close<Elem, kTokenBits>(static_cast<const Elem*>(P.logits) + b * P.W * P.row_stride,
                                                      P.row_stride, sm, ranked, own_c[j], own_id[j]);
        if (rank < K) beam_output(P, b * K + rank, own_c[j], own_id[j]);
    }
    for (int i = cands + t; i < K; i += NT) {
        P.out_scores[b * K + i] = -INFINITY;
        P.out_parents[b * K + i] = -1;
        P.out_tokens[b * K + i] = -1;
    }
}

// CTA-collective.
template <class Tag, int VEC>
__device__ __forceinline__ void beam_merge(const BeamParams& P, int64_t b, BeamMergeSmem& sm) {
    const int t = threadIdx.x, lane = t & 31, wp = t >> 5;
    const int K = P.K, total = P.W * P.tiles;
    const float* peaks = P.peaks + b * total;
    // Tile j of this thread: every warp gets tiles of all rows, so that the
    // warps' best are the request's best.  The loads go out before the rows'
    // sums are merged; rows that were not streamed hold nothing, what is read
    // there is not used.
    auto nth = [&](int j) { return j * NT + lane * NWARPS + ((wp + lane) & (NWARPS - 1)); };
    BeamSegs first;
    first.load(P.stats + (b * P.W + min(wp, P.W - 1)) * P.segs, 0, P.segs);
    float m[kMergePeaks];
#pragma unroll
    for (int j = 0; j < kMergePeaks; ++j) {
        const int i = nth(j);
        m[j] = j * NT < total && i < total ? __ldcg(&peaks[i]) : -INFINITY;
    }
    if (t == 0) sm.tiles = sm.cands = sm.close = 0;
    if (beam_rows(P, b, sm, [&](int w) {
            const BeamStat* p = P.stats + (b * P.W + w) * P.segs;
            if (w != wp) first.load(p, 0, P.segs);
            return beam_row_sum(p, P.segs, first);
        }))
        return;
    // The tiles' values, and a bound that K of them reach: the K-th largest of
    // the 32 that the warps' 32 / NWARPS largest lanes make up (rounded down to
    // fp32).
    // The row of tile i: the quotient is below 32 and its error below 2^-17, less
    // than half a tile (at most 2^15 tiles a row).
    const float inv = 1.0f / static_cast<float>(P.tiles);
    auto row_of = [&](int i) { return static_cast<int>((static_cast<float>(i) + 0.5f) * inv); };
    auto value = [&](int i, float x) {
        const int w = row_of(i);
        return x > -INFINITY && sm.state[w] == 1 ? beam_value(sm, w, x) : -INFINITY;
    };
    double c[kMergePeaks], best = -INFINITY;
#pragma unroll
    for (int j = 0; j < kMergePeaks; ++j) {
        c[j] = -INFINITY;
        if (j * NT >= total) continue;  // CTA-uniform
        const int i = nth(j);
        if (i < total) c[j] = value(i, m[j]);
        best = fmax(best, c[j]);
    }
    for (int j = kMergePeaks; j * NT < total; ++j) {
        const int i = nth(j);
        if (i < total) best = fmax(best, value(i, __ldcg(&peaks[i])));
    }
    const double floor = beam_bound(best, K, sm);
    auto keep = [&](double v, int i, float x) {
        if (!(v >= floor && v > -INFINITY)) return;
        const int at = atomicAdd(&sm.tiles, 1), w = row_of(i);
        if (fabsf(x) < sm.near[w]) sm.close = 1;
        if (at < kMergeTiles) {
            sm.c[at] = v;
            const uint32_t id = (static_cast<uint32_t>(w) << kTileBits) + static_cast<uint32_t>(i - w * P.tiles);
            sm.id[at] = id;
            if (at < kMaxBeams) sm.tile_id[at] = id;
        }
    };
#pragma unroll
    for (int j = 0; j < kMergePeaks; ++j)
        if (j * NT < total) keep(c[j], nth(j), m[j]);
    for (int j = kMergePeaks; j * NT < total; ++j) {
        const int i = nth(j);
        const float x = i < total ? __ldcg(&peaks[i]) : -INFINITY;
        if (i < total) keep(value(i, x), i, x);
    }
    __syncthreads();
    // Few enough tiles to hold in registers are all taken; of more the K best, a
    // tile's rank being its place.
    const int have = sm.tiles;
    int n = have;
    double bound = floor;
    if (have > 2 * NWARPS) {
        n = min(have, K);
        if (have <= kMergeTiles) {
            for (int i = t; i < have; i += NT) {
                const double v = sm.c[i];
                const uint32_t id = sm.id[i];
                int rank = beam_place(sm, have, v, id);
                if (sm.close != 0) rank = beam_place_close<float, kTileBits>(peaks, P.tiles, sm, have, v, id);
                if (rank < K) {
                    sm.tile_c[rank] = v;
                    sm.tile_id[rank] = id;
                }
            }
        } else {
            n = sm.close != 0 ? beam_many_tiles<true>(P, peaks, sm) : beam_many_tiles<false>(P, peaks, sm);
        }
        __syncthreads();
        bound = n == K ? sm.tile_c[K - 1] : -INFINITY;
    }
    auto take = [&](double v, uint32_t id, float, bool close) {
        if (close) sm.close = 1;
        const int at = atomicAdd(&sm.cands, 1);
        if (at < kMergeCand) {
            sm.c[at] = v;
            sm.id[at] = id;
        }
    };
    // Few tiles to choose from bound the elements badly: the threads' best
    // elements do better.
    const bool few = total < 8 * K;
    if (n <= 2 * NWARPS) {  // two tiles a warp, held in registers
        BeamPlace<Tag, VEC> x, y;
        const bool has_x = wp < n, has_y = wp + NWARPS < n;
        if (has_x) x.load(P, b, sm, wp);
        if (has_y) y.load(P, b, sm, wp + NWARPS);
        if (few) {
            double e = beam_ended(P, sm) ? sm.s[t] : -INFINITY;
            if (has_x) e = fmax(e, x.best(sm));
            if (has_y) e = fmax(e, y.best(sm));
            bound = fmax(bound, beam_bound(e, K, sm));
        }
        if (P.tiles <= kMendTiles) {
            if (has_x) x.mend(P, b, sm);
            if (has_y) y.mend(P, b, sm);
            beam_mend_rows(P, sm);
            bound = beam_slack(bound);
        }
        if (has_x) x.look(sm, bound, take);
        if (has_y) y.look(sm, bound, take);
        beam_look_ended(P, sm, bound, take);
    } else {
        if (P.tiles <= kMendTiles) {
            BeamPlace<Tag, VEC> x;
            for (int i = wp; i < n; i += NWARPS) {
                x.load(P, b, sm, i);
                x.mend(P, b, sm);
            }
            beam_mend_rows(P, sm);
            bound = beam_slack(bound);
        }
        if (few) bound = fmax(bound, beam_visit_bound<Tag, VEC>(P, b, n, sm));
        beam_visit<Tag, VEC>(P, b, n, bound, sm, take);
    }
    __syncthreads();
    int cands = sm.cands;
    if (cands > kMergeCand && !few) {  // the tiles' many elements above the K-th tile's best
        bound = fmax(bound, beam_visit_bound<Tag, VEC>(P, b, n, sm));
        if (t == 0) sm.cands = 0;
        __syncthreads();
        beam_visit<Tag, VEC>(P, b, n, bound, sm, take);
        __syncthreads();
        cands = sm.cands;
    }
    if (cands <= kMergeCand) beam_rank<typename Tag::storage>(P, b, sm, cands);
    else if (sm.close != 0) beam_many_candidates<Tag, VEC, true>(P, b, n, bound, sm);
    else beam_many_candidates<Tag, VEC, false>(P, b, n, bound, sm);
}

// Rows of many tiles: a warp per segment, then a CTA per request.  The second
// kernel's launch overlaps the first one's end.  (One kernel whose last CTA
// per request merges, found by an atomic ticket, is slower: every CTA then
// waits for a memory fence and the ticket before it leaves its place, 38 us
// against 33.5 us at 64 x 8 rows of 128256 bf16.)
template <class Tag, int VEC>
__global__ void __launch_bounds__(NT, 5) beam_pass_kernel(const BeamParams P) {
    grid_dependency_wait();
    grid_launch_dependents();
    const unsigned unit = blockIdx.x * NWARPS + (threadIdx.x >> 5);
    const unsigned r = unit / static_cast<unsigned>(P.segs);
    if (r >= static_cast<unsigned>(P.B * P.W)) return;  // warp-uniform; no CTA barrier below
    beam_stream<Tag, VEC>(P, r, static_cast<int>(unit - r * static_cast<unsigned>(P.segs)));
}

template <class Tag, int VEC>
__global__ void __launch_bounds__(NT, 2) beam_merge_kernel(const BeamParams P) {
    __shared__ BeamMergeSmem sm;
    grid_dependency_wait();
    grid_launch_dependents();
    beam_merge<Tag, VEC>(P, blockIdx.x, sm);
}

// Requests of at most kSmallTiles tiles: one CTA and one launch.  Every tile
// stays in its warp's registers from the first read to the last, so there is
// nothing to select tiles for.
constexpr int kSmallTiles = 2 * NWARPS;

struct BeamSmallSmem : BeamMergeSmem {
    BeamStat stat[kSmallTiles];
};

template <class Tag, int VEC>
__global__ void __launch_bounds__(NT, 2) beam_small_kernel(const BeamParams P) {
    __shared__ BeamSmallSmem sm;
    const int t = threadIdx.x, lane = t & 31, wp = t >> 5;
    grid_dependency_wait();
    grid_launch_dependents();
    const int64_t b = blockIdx.x;
    const int units = P.W * P.tiles;  // unit u: tile u % tiles of beam u / tiles
    if (t == 0) sm.cands = sm.close = 0;
    if (t < kSmallTiles) sm.tile_id[t] = static_cast<uint32_t>(t / P.tiles << kTileBits) + static_cast<uint32_t>(t % P.tiles);
    __syncthreads();
    BeamPlace<Tag, VEC> x, y;
    // Rows that are not streamed are not read.
    auto streams = [&](int u) {
        return u < units && beam_streams(P, b * P.W + static_cast<int>(sm.tile_id[u] >> kTileBits));
    };
    bool has_x = streams(wp), has_y = streams(wp + NWARPS);
    if (has_x) x.load(P, b, sm, wp);
    if (has_y) y.load(P, b, sm, wp + NWARPS);
    auto total = [&](const BeamPlace<Tag, VEC>& p, int u) {
        const float m = from_ord_i32(__reduce_max_sync(FULL_MASK, ord_i32(fmaxf(p.a.most(), p.xe))));
        const float ref = beam_up(m);
        double S = beam_far(ref) ? static_cast<double>(beam_sum<Tag, VEC>(p.a.w, BeamRef(ref)))
                                 : beam_sum_exact<Tag, VEC>(p.a.w, p.a.most(), ref, m - kBeamLarge);
        if (p.ie >= 0) S += static_cast<double>(beam_term(p.xe, ref)) + (p.xe >= m - kBeamLarge && !beam_far(ref) ? beam_miss(p.xe, ref) : 0.0);
        S = warp_sum_f64(S);
        if (lane == 0) {
            sm.stat[u].M = beam_ref(ref);
            sm.stat[u].S = S;
        }
    };
    if (has_x) total(x, wp);
    if (has_y) total(y, wp + NWARPS);
    __syncthreads();
    if (beam_rows(P, b, sm, [&](int w) {
            BeamSegs v;
#pragma unroll
            for (int j = 0; j < kSegs; ++j) {
                v.M[j] = -DBL_MAX;
                v.S[j] = 0.0;
            }
            if (lane < P.tiles) {
                v.M[0] = sm.stat[w * P.tiles + lane].M;
                v.S[0] = sm.stat[w * P.tiles + lane].S;
            }
            return beam_row_sum(nullptr, P.tiles, v);
        }))
        return;
    has_x = has_x && sm.state[x.w] == 1;  // a row of only -inf holds no candidate
    has_y = has_y && sm.state[y.w] == 1;
    double e = beam_ended(P, sm) ? sm.s[t] : -INFINITY;
    if (has_x) e = fmax(e, x.best(sm));
    if (has_y) e = fmax(e, y.best(sm));
    const double bound = beam_bound(e, P.K, sm);
    auto take = [&](double v, uint32_t id, float, bool close) {
        if (close) sm.close = 1;
        const int at = atomicAdd(&sm.cands, 1);
        if (at < kMergeCand) {
            sm.c[at] = v;
            sm.id[at] = id;
        }
    };
    if (has_x) x.look(sm, bound, take);
    if (has_y) y.look(sm, bound, take);
    beam_look_ended(P, sm, bound, take);
    __syncthreads();
    const int cands = sm.cands;
    if (cands <= kMergeCand) {
        beam_rank<typename Tag::storage>(P, b, sm, cands);
        return;
    }
    // Runs of equal values: the best one behind the last one found, K times.
    auto one_by_one = [&](auto close) {
        constexpr bool CLOSE = decltype(close)::value;
        BeamBest last = {INFINITY, 0u, 0.0f};
        for (int i = 0; i < P.K; ++i) {
            BeamBest best = {-INFINITY, kBeamNone, 0.0f};
            auto offer = [&](double c, uint32_t id, float x, bool) { beam_next<CLOSE, kTokenBits>(last, {c, id, x}, best); };
            if (has_x) x.look(sm, bound, offer);
            if (has_y) y.look(sm, bound, offer);
            beam_look_ended(P, sm, bound, offer);
            last = beam_block_best<CLOSE, kTokenBits>(best, sm);
            if (t == 0) beam_output(P, b * P.K + i, last.c, last.id);
        }
    };
    // 8 x 4 rows of 1000 bf16, K = 32 (all candidates are looked at K times): 153 us,
    // 201 us in one loop that may compare logits.
    if (sm.close == 0) one_by_one(std::false_type());
    else one_by_one(std::true_type());
}

}  // namespace specdec
