// states.cuh — moving cached states (keys, values, hidden states) after a
// selection or a verification: pure copies, bound by memory bandwidth.
//
// reorder_states_kernel: beams.  Row (b, i) of every group becomes row
// (b, parents[b, i]).  One thread owns one column (the same 4 to 16 bytes of
// every beam): it loads each parent that moves once and then stores to all of
// its children, so the move is safe in place and a parent is read once
// however many children it has.  16 groups of 8 x 8 beams of up to 1024 x 512
// bf16 (random lengths, mean of three inputs): 168 us for 1.09 GB read and
// written, 6.5 TB/s, as fast as a plain copy; 6 groups and 7 heads of 5 x 5 beams
// of up to 333 x 80 fp32 in place, 14.4 us for 53 MB, 3.7 TB/s.
//
// commit_path_kernel: draft trees (handbook page, "Medusa": the longest
// accepted candidate prefix is kept).  The states of the root and of the
// accepted nodes go to the slots of the request's next positions.  A node of
// depth j has an index >= j, so in place (source and destination rows of one
// cache, addressed by the same slots) row j is written only after every row
// with an index <= j has been read.  A few dependent reads, then a copy: 8
// groups of 256 requests with 1000-byte rows 5.3 us for 20 MB, 3.9 TB/s.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "device_utils.cuh"
#include "verify_common.cuh"

namespace specdec {

constexpr int kMaxReorderBeams = 32;

struct ReorderParams {
    const char* src;
    char* dst;
    const int32_t* parents;  // [B, W]
    const int32_t* lengths;  // [B] or null
    int64_t G, H;
    int B, W;
    int64_t T;
    int64_t row;                            // columns of a position (units of VT)
    int64_t sg, sb, sw, sh, st;             // strides of src in bytes: group, request, beam, head, position
    int64_t dg, db, dw, dh, dt;             // of dst
    int flat;                               // positions follow one another without a gap on both sides
    int narrow;                             // the columns of a (group, head, request) are counted in 32 bits
    int in_place;
};

// CTAs (x: column tiles, y: requests, z: groups and heads), each taking every
// gridDim-th of them.  A request none of whose rows move costs its parents'
// read.
template <class VT, int WT, int C>
__global__ void __launch_bounds__(NT) reorder_states_kernel(const ReorderParams P) {
    const int lane = threadIdx.x & 31;
    grid_dependency_wait();
    grid_launch_dependents();
    for (int b = blockIdx.y; b < P.B; b += gridDim.y) {
        int par = -1;
        if (lane < P.W) {
            par = __ldg(&P.parents[static_cast<int64_t>(b) * P.W + lane]);
            if (par >= P.W || par < 0 || (P.in_place && par == lane)) par = -1;  // row left as it is
        }
        int64_t len = P.T;
        if (P.lengths != nullptr) {
            const int64_t l = __ldg(&P.lengths[b]);
            len = l < 0 ? 0 : (l < len ? l : len);
        }
        if (__ballot_sync(FULL_MASK, par >= 0) == 0u) continue;
        unsigned child[WT];
#pragma unroll
        for (int p = 0; p < WT; ++p) child[p] = __ballot_sync(FULL_MASK, par == p);
        const int64_t cols = len * P.row;
        for (int64_t gh = blockIdx.z; gh < P.G * P.H; gh += gridDim.z) {
            const int64_t g = P.H == 1 ? gh : gh / P.H, h = gh - g * P.H;
            const char* s0 = P.src + g * P.sg + b * P.sb + h * P.sh;
            char* d0 = P.dst + g * P.dg + b * P.db + h * P.dh;
            for (int64_t c0 = static_cast<int64_t>(blockIdx.x) * (NT * C); c0 < cols;
                 c0 += static_cast<int64_t>(gridDim.x) * (NT * C)) {
                VT v[C][WT];
                int64_t dof[C];
                bool ok[C];
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    const int64_t x = c0 + c * NT + threadIdx.x;
                    ok[c] = x < cols;
                    int64_t so;
                    if (P.flat) {
                        so = dof[c] = x * static_cast<int64_t>(sizeof(VT));
                    } else {
                        const int64_t t = P.narrow ? static_cast<int64_t>(static_cast<uint32_t>(x) / static_cast<uint32_t>(P.row))
                                                   : x / P.row;
                        const int64_t e = (x - t * P.row) * static_cast<int64_t>(sizeof(VT));
                        so = t * P.st + e;
                        dof[c] = t * P.dt + e;
                    }
#pragma unroll
                    for (int p = 0; p < WT; ++p)
                        if (child[p] != 0u && ok[c]) v[c][p] = *reinterpret_cast<const VT*>(s0 + p * P.sw + so);
                }
#pragma unroll
                for (int p = 0; p < WT; ++p) {
                    for (unsigned m = child[p]; m != 0u; m &= m - 1u) {
                        char* d = d0 + (__ffs(m) - 1) * P.dw;
#pragma unroll
                        for (int c = 0; c < C; ++c)
                            if (ok[c]) *reinterpret_cast<VT*>(d + dof[c]) = v[c][p];
                    }
                }
            }
        }
    }
}

// Out of place, positions without gaps, but beams whose runs start at any byte
// (odd row sizes): 16-byte stores all the same.  A thread owns 16 aligned bytes
// of every row of dst and puts each together from the two aligned 16-byte words
// of src that hold them (both hold a byte of the run, so no other memory is
// touched; the neighbouring threads' words come from L1).  28 groups of 9 beams
// of 472 x 249 bf16: 21.9 us for 61 MB (2.8 TB/s; two loads for every store, and
// a parent's words once for each of its children), 33.9 us in 2-byte accesses.
__device__ __forceinline__ uint4 shift_words(const uint4& a, const uint4& b, int bytes) {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    uint32_t x[5];
    switch (bytes >> 2) {  // the same for the whole CTA
        case 0:
#pragma unroll
            for (int i = 0; i < 5; ++i) x[i] = w[i];
            break;
        case 1:
#pragma unroll
            for (int i = 0; i < 5; ++i) x[i] = w[i + 1];
            break;
        case 2:
#pragma unroll
            for (int i = 0; i < 5; ++i) x[i] = w[i + 2];
            break;
        default:
#pragma unroll
            for (int i = 0; i < 5; ++i) x[i] = i + 3 < 8 ? w[i + 3] : 0u;
            break;
    }
    const int bits = (bytes & 3) * 8;
    return make_uint4(__funnelshift_r(x[0], x[1], bits), __funnelshift_r(x[1], x[2], bits),
                      __funnelshift_r(x[2], x[3], bits), __funnelshift_r(x[3], x[4], bits));
}

constexpr int kShiftRows = 4;  // rows whose words a thread has on their way

__global__ void __launch_bounds__(NT) reorder_shift_kernel(const ReorderParams P) {  // P.row in bytes
    __shared__ int parent[kMaxReorderBeams];
    grid_dependency_wait();
    grid_launch_dependents();
    const int t = threadIdx.x;
    for (int b = blockIdx.y; b < P.B; b += gridDim.y) {
        __syncthreads();
        if (t < kMaxReorderBeams) {
            int p = t < P.W ? __ldg(&P.parents[static_cast<int64_t>(b) * P.W + t]) : -1;
            parent[t] = p < P.W ? p : -1;
        }
        __syncthreads();
        int64_t len = P.T;
        if (P.lengths != nullptr) {
            const int64_t l = __ldg(&P.lengths[b]);
            len = l < 0 ? 0 : (l < len ? l : len);
        }
        const int64_t bytes = len * P.row;
        for (int64_t gh = blockIdx.z; gh < P.G * P.H; gh += gridDim.z) {
            const int64_t g = P.H == 1 ? gh : gh / P.H, h = gh - g * P.H;
            const char* s0 = P.src + g * P.sg + b * P.sb + h * P.sh;
            char* d0 = P.dst + g * P.dg + b * P.db + h * P.dh;
            for (int64_t k = static_cast<int64_t>(blockIdx.x) * NT + t; k * 16 < bytes; k += static_cast<int64_t>(gridDim.x) * NT) {
                for (int i0 = 0; i0 < P.W; i0 += kShiftRows) {
                    uint4 lo[kShiftRows], hi[kShiftRows];
                    int64_t off[kShiftRows];  // of the thread's 16 bytes in the run; -1: none
#pragma unroll
                    for (int j = 0; j < kShiftRows; ++j) {
                        const int i = i0 + j;
                        off[j] = -1;
                        if (i < P.W && parent[i] >= 0) {
                            const char* d = d0 + i * P.dw;
                            const int64_t head = -reinterpret_cast<intptr_t>(d) & 15;  // bytes before the first boundary
                            if (k * 16 + head + 16 <= bytes) {
                                off[j] = k * 16 + head;
                                const uintptr_t from = reinterpret_cast<uintptr_t>(s0 + parent[i] * P.sw + off[j]);
                                const uint4* q = reinterpret_cast<const uint4*>(from & ~static_cast<uintptr_t>(15));
                                lo[j] = __ldg(q);
                                hi[j] = (from & 15) != 0 ? __ldg(q + 1) : lo[j];
                            }
                        }
                    }
#pragma unroll
                    for (int j = 0; j < kShiftRows; ++j)
                        if (off[j] >= 0) {
                            const int i = i0 + j;
                            const int by = static_cast<int>(reinterpret_cast<uintptr_t>(s0 + parent[i] * P.sw + off[j]) & 15);
                            *reinterpret_cast<uint4*>(d0 + i * P.dw + off[j]) = shift_words(lo[j], hi[j], by);
                        }
                }
            }
            if (blockIdx.x == 0) {  // the bytes before the first and behind the last boundary of each row
                for (int x = t; x < P.W * 32; x += NT) {
                    const int i = x >> 5, e = x & 31;
                    if (parent[i] < 0) continue;
                    char* d = d0 + i * P.dw;
                    const int64_t head = min(static_cast<int64_t>(-reinterpret_cast<intptr_t>(d) & 15), bytes);
                    const int64_t tail = (bytes - head) & 15;
                    int64_t at = -1;
                    if (e < 16) at = e < head ? e : -1;
                    else at = e - 16 < tail ? bytes - tail + (e - 16) : -1;
                    if (at >= 0) d[at] = s0[parent[i] * P.sw + at];
                }
            }
        }
    }
}

struct CommitParams {
    const char* src;
    char* dst;
    const int32_t* accept_len;    // [B]
    const int32_t* accept_nodes;  // [B, depth]
    const int64_t* src_slots;     // [B, nodes] or null: src rows are [B, nodes]
    const int64_t* dst_slots;     // [B, >= depth + 1], row stride dst_slots_stride
    int64_t src_slots_stride, dst_slots_stride;
    int64_t G;
    int B, nodes, depth;
    int64_t src_rows, dst_rows;   // rows that slots may name (src_rows: with src_slots)
    int64_t row;                  // columns of a row (units of VT)
    int64_t sg, sb, sr, dg, dr;   // strides in bytes: group, request (without src_slots), row
};

constexpr int kCommitThreads = 128;
constexpr int kMaxPath = 33;  // the root and up to 32 nodes

// CTAs (x: column tiles, y: requests, z: groups).  The path's rows are looked
// up once per request, all at once (accepted length, nodes and slots are one
// round trip); a thread then copies its column of every row.
template <class VT>
__global__ void __launch_bounds__(kCommitThreads) commit_path_kernel(const CommitParams P) {
    constexpr int kBatch = 8;  // rows loaded before the first of them is stored
    __shared__ int64_t from[kMaxPath], to[kMaxPath];  // byte offsets, -1: not moved
    __shared__ int last;                              // accepted length, clamped to depth
    grid_dependency_wait();
    grid_launch_dependents();
    const int t = threadIdx.x;
    for (int b = blockIdx.y; b < P.B; b += gridDim.y) {
        __syncthreads();
        if (t <= P.depth) {
            const int h = __ldg(&P.accept_len[b]);
            const int node = t == 0 ? 0 : __ldg(&P.accept_nodes[static_cast<int64_t>(b) * P.depth + t - 1]);
            int64_t d = __ldg(&P.dst_slots[b * P.dst_slots_stride + t]);
            int64_t f = -1;
            if (t <= h && node >= 0 && node < P.nodes && d >= 0 && d < P.dst_rows) {
                d *= P.dr;
                if (P.src_slots != nullptr) {
                    f = __ldg(&P.src_slots[b * P.src_slots_stride + node]);
                    f = f >= 0 && f < P.src_rows ? f * P.sr : -1;
                } else {
                    f = b * P.sb + node * P.sr;
                }
            }
            from[t] = f;
            to[t] = d;
            if (t == 0) last = h < P.depth ? h : P.depth;
        }
        __syncthreads();
        for (int64_t g = blockIdx.z; g < P.G; g += gridDim.z)
            for (int64_t x = static_cast<int64_t>(blockIdx.x) * kCommitThreads + t; x < P.row;
                 x += static_cast<int64_t>(gridDim.x) * kCommitThreads) {
                const char* s = P.src + g * P.sg + x * static_cast<int64_t>(sizeof(VT));
                char* d = P.dst + g * P.dg + x * static_cast<int64_t>(sizeof(VT));
                for (int j0 = 0; j0 <= last; j0 += kBatch) {
                    VT v[kBatch];
#pragma unroll
                    for (int i = 0; i < kBatch; ++i)
                        if (j0 + i <= last && from[j0 + i] >= 0) v[i] = *reinterpret_cast<const VT*>(s + from[j0 + i]);
#pragma unroll
                    for (int i = 0; i < kBatch; ++i)
                        if (j0 + i <= last && from[j0 + i] >= 0) *reinterpret_cast<VT*>(d + to[j0 + i]) = v[i];
                }
            }
    }
}

}  // namespace specdec
