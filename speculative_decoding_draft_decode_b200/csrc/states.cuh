// states.cuh — moving cached states (keys, values, hidden states) after a
// selection or a verification: pure copies, bound by memory bandwidth.
//
// reorder_states_kernel: beams.  Row (b, i) of every group becomes row
// (b, parents[b, i]).  One thread owns one column (the same 4 to 16 bytes of
// every beam): it loads each parent that moves once and then stores to all of
// its children, so the move is safe in place and a parent is read once
// however many children it has.
//
// commit_path_kernel: draft trees (handbook page, "Medusa": the longest
// accepted candidate prefix is kept).  The states of the root and of the
// accepted nodes go to the slots of the request's next positions.  A node of
// depth j has an index >= j, so in place (source and destination rows of one
// cache, addressed by the same slots) row j is written only after every row
// with an index <= j has been read.
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
    int64_t tiles;                          // column tiles per (group, head, request)
    int flat;                               // positions follow one another without a gap on both sides
    int in_place;
};

// Work item: (group, head, request, tile of NT * C columns).
template <class VT, int WT, int C>
__global__ void __launch_bounds__(NT) reorder_states_kernel(const ReorderParams P) {
    const int lane = threadIdx.x & 31;
    grid_dependency_wait();
    grid_launch_dependents();
    const int64_t items = P.G * P.H * P.B * P.tiles;
    for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
        const int64_t tile = it % P.tiles;
        int64_t q = it / P.tiles;
        const int b = static_cast<int>(q % P.B);
        q /= P.B;
        const int64_t h = q % P.H, g = q / P.H;
        int64_t len = P.T;
        if (P.lengths != nullptr) {
            const int64_t l = __ldg(&P.lengths[b]);
            len = l < 0 ? 0 : (l < len ? l : len);
        }
        const int64_t cols = len * P.row;
        const int64_t c0 = tile * (NT * C);
        if (c0 >= cols) continue;
        int par = -1;
        if (lane < P.W) {
            par = __ldg(&P.parents[static_cast<int64_t>(b) * P.W + lane]);
            if (par >= P.W || par < 0 || (P.in_place && par == lane)) par = -1;  // row left as it is
        }
        unsigned child[WT];
#pragma unroll
        for (int p = 0; p < WT; ++p) child[p] = __ballot_sync(FULL_MASK, par == p);
        const char* s0 = P.src + g * P.sg + b * P.sb + h * P.sh;
        char* d0 = P.dst + g * P.dg + b * P.db + h * P.dh;
        VT v[C][WT];
        int64_t so[C], dof[C];
        bool ok[C];
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int64_t x = c0 + c * NT + threadIdx.x;
            ok[c] = x < cols;
            const int64_t t = P.flat ? 0 : x / P.row, e = x - t * P.row;
            so[c] = t * P.st + e * static_cast<int64_t>(sizeof(VT));
            dof[c] = t * P.dt + e * static_cast<int64_t>(sizeof(VT));
#pragma unroll
            for (int p = 0; p < WT; ++p)
                if (child[p] != 0u && ok[c]) v[c][p] = *reinterpret_cast<const VT*>(s0 + p * P.sw + so[c]);
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
    int64_t tiles;
};

template <class VT>
__global__ void __launch_bounds__(NT) commit_path_kernel(const CommitParams P) {
    constexpr int kBatch = 8;  // rows loaded before the first of them is stored
    __shared__ int64_t from[kBatch], to[kBatch];
    grid_dependency_wait();
    grid_launch_dependents();
    const int64_t items = P.G * P.B * P.tiles;
    for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
        const int64_t tile = it % P.tiles;
        const int64_t q = it / P.tiles;
        const int64_t b = q % P.B, g = q / P.B;
        int h = __ldg(&P.accept_len[b]);
        if (h > P.depth) h = P.depth;
        const int64_t x = tile * NT + threadIdx.x;
        for (int j0 = 0; j0 <= h; j0 += kBatch) {
            __syncthreads();
            if (threadIdx.x < kBatch) {
                const int j = j0 + threadIdx.x;
                int64_t f = -1, d = -1;
                if (j <= h) {
                    const int node = j == 0 ? 0 : __ldg(&P.accept_nodes[b * P.depth + j - 1]);
                    if (node >= 0 && node < P.nodes) {
                        d = __ldg(&P.dst_slots[b * P.dst_slots_stride + j]);
                        if (P.src_slots != nullptr) {
                            f = __ldg(&P.src_slots[b * P.src_slots_stride + node]);
                            f = f >= 0 && f < P.src_rows ? f * P.sr : -1;
                        } else {
                            f = b * P.sb + node * P.sr;
                        }
                        d = d >= 0 && d < P.dst_rows ? d * P.dr : -1;
                    }
                }
                if (d < 0) f = -1;
                from[threadIdx.x] = f;
                to[threadIdx.x] = d;
            }
            __syncthreads();
            if (x < P.row) {
                const char* s = P.src + g * P.sg + x * static_cast<int64_t>(sizeof(VT));
                char* d = P.dst + g * P.dg + x * static_cast<int64_t>(sizeof(VT));
                VT v[kBatch];
#pragma unroll
                for (int i = 0; i < kBatch; ++i)
                    if (from[i] >= 0) v[i] = *reinterpret_cast<const VT*>(s + from[i]);
#pragma unroll
                for (int i = 0; i < kBatch; ++i)
                    if (from[i] >= 0) *reinterpret_cast<VT*>(d + to[i]) = v[i];
            }
        }
    }
}

}  // namespace specdec
