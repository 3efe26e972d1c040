// decode_api.cuh — the part of the C-ABI (include/specdec.h) around the verify
// step: argument checks, workspace layout and launches of beam selection, state
// reordering, path commit and slot planning.  Compiled behind specdec_api.cu, whose
// checks and launch helpers it shares.
#pragma once

#include "beam_select.cuh"
#include "slots.cuh"
#include "states.cuh"

namespace specdec {
namespace {

// Memory of an argument; none if its address is null.
struct Span {
    const void* at;
    int64_t bytes;
};
bool meet(const Span& a, const Span& b) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.at), y = reinterpret_cast<uintptr_t>(b.at);
    return x != 0 && y != 0 && a.bytes > 0 && b.bytes > 0 && x < y + static_cast<uintptr_t>(b.bytes) &&
           y < x + static_cast<uintptr_t>(a.bytes);
}
// Whether an output meets another one or an input.  Output i may be input
// replaces[i] itself (-1: none).
template <int O, int I>
bool outputs_meet(const Span (&out)[O], const int (&replaces)[O], const Span (&in)[I]) {
    for (int i = 0; i < O; ++i) {
        for (int j = 0; j < i; ++j)
            if (meet(out[i], out[j])) return true;
        for (int j = 0; j < I; ++j)
            if (meet(out[i], in[j]) && !(replaces[i] == j && out[i].at == in[j].at && out[i].bytes == in[j].bytes))
                return true;
    }
    return false;
}

// Beam selection: the segments' sums and the tiles' largest logits, behind the
// fixed area (which it does not touch).
struct BeamLayout {
    int tiles = 0, seg_tiles = 0, segs = 0;
    size_t stats = 0, peaks = 0, total = 0;
};

BeamLayout make_beam_layout(int B, int W, int V, specdec_dtype dtype) {
    BeamLayout L;
    const int nv = V / vec_elems(dtype);
    L.tiles = nv > kTileVecs ? (nv + kTileVecs - 1) / kTileVecs : 1;
    const int64_t rows = static_cast<int64_t>(B) * W;
    // Tiles of a warp: enough warps to fill the GPU come first, then longer
    // segments (fewer partial sums and less start-up per byte).  Calls with
    // segments of 1, 2 and 4 tiles: 1008 tiles 8.7, 9.8, 10.9 us (bf16) and 9.6, 9.1,
    // 9.8 (fp32); 2376 tiles 10.4, 9.7, 9.6 (fp32); 4032 tiles 10.0, 10.4, 11.1
    // (bf16); 11880 tiles 14.4, 12.8, 12.4 (fp32); 64512 tiles 36.6, 33.7, 32.7
    // (bf16).  One rule for both types; bf16 alone would take one tile up to 4032.
    const int64_t all = rows * L.tiles;
    L.seg_tiles = W * L.tiles <= kSmallTiles || all < 1024 ? 1 : all < 4096 ? 2 : 4;
    L.segs = (L.tiles + L.seg_tiles - 1) / L.seg_tiles;
    // Sized for segments of one tile, so that a smaller call never needs more.
    L.stats = kPartialBase;
    L.peaks = align_up(L.stats + static_cast<size_t>(rows) * static_cast<size_t>(L.tiles) * sizeof(BeamStat), 256);
    L.total = align_up(L.peaks + static_cast<size_t>(rows) * static_cast<size_t>(L.tiles) * sizeof(float), 256);
    return L;
}

template <class Tag>
specdec_status launch_beam(const BeamParams& P, cudaStream_t stream) {
    if (P.W * P.tiles <= kSmallTiles) {
        if (launch_pdl(beam_small_kernel<Tag, Tag::VEC>, dim3(static_cast<unsigned>(P.B)), 0, stream, P) != cudaSuccess)
            return SPECDEC_ERR_CUDA;
        return cudaGetLastError() == cudaSuccess ? SPECDEC_OK : SPECDEC_ERR_CUDA;
    }
    const int64_t units = static_cast<int64_t>(P.B) * P.W * P.segs;
    if (units > 0x7fffffff) return SPECDEC_ERR_UNSUPPORTED;  // units are counted in 32 bits
    const unsigned ctas = static_cast<unsigned>((units + NWARPS - 1) / NWARPS);
    if (launch_pdl(beam_pass_kernel<Tag, Tag::VEC>, dim3(ctas), 0, stream, P) != cudaSuccess) return SPECDEC_ERR_CUDA;
    if (launch_pdl(beam_merge_kernel<Tag, Tag::VEC>, dim3(static_cast<unsigned>(P.B)), 0, stream, P) != cudaSuccess)
        return SPECDEC_ERR_CUDA;
    return cudaGetLastError() == cudaSuccess ? SPECDEC_OK : SPECDEC_ERR_CUDA;
}

// One cluster over the batch: a CTA per kPlanThreads requests, up to kPlanCtas.
cudaError_t launch_plan_tables(const PlanParams& P, cudaStream_t stream) {
    const int need = (P.B + kPlanThreads - 1) / kPlanThreads;
    const unsigned ctas = static_cast<unsigned>(need < kPlanCtas ? need : kPlanCtas);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kPlanThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = ctas;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, plan_tables_kernel<false, kPlanThreads>, P);
}

// Runs of a beam's positions from which unaligned ones are put together from
// aligned words.
constexpr int64_t kShiftBytes = 256;

// Grid of a copy kernel: requests and groups first, then column tiles, about
// `each` of them per CTA (a CTA looks its request up before it copies), but
// enough CTAs to fill the GPU and at most kCopyMost.  Measured: 42 x 5 groups
// and requests of 13 tiles 15.3 us with three tiles a CTA, 17.7 us with one;
// 16 x 8 of 128 tiles 168 us with 5461 CTAs, 172 us with 2368, 207 us with 296.
constexpr int64_t kSMs = 148, kCopyLeast = kSMs * 4, kCopyMost = kSMs * 64;
dim3 tile_grid(int64_t tiles, int B, int64_t groups, int each) {
    const unsigned z = static_cast<unsigned>(groups < 65535 ? groups : 65535);
    const unsigned y = static_cast<unsigned>(B < 65535 ? B : 65535);
    const int64_t rest = static_cast<int64_t>(y) * z;
    const double want = static_cast<double>(tiles) * static_cast<double>(rest) / each;
    const int64_t ctas = want < kCopyLeast ? kCopyLeast : want > kCopyMost ? kCopyMost : static_cast<int64_t>(want);
    const int64_t room = ctas / rest + 1;
    return dim3(static_cast<unsigned>(tiles < room ? tiles : room), y, z);
}

template <class VT, int WT, int C>
specdec_status launch_reorder_as(const ReorderParams& P, cudaStream_t stream) {
    const dim3 grid = tile_grid((P.T * P.row + NT * C - 1) / (NT * C), P.B, P.G * P.H, 3);
    if (launch_pdl(reorder_states_kernel<VT, WT, C>, grid, 0, stream, P) != cudaSuccess) return SPECDEC_ERR_CUDA;
    return cudaGetLastError() == cudaSuccess ? SPECDEC_OK : SPECDEC_ERR_CUDA;
}

specdec_status launch_reorder_shift(ReorderParams P, int64_t row_bytes, cudaStream_t stream) {
    P.row = row_bytes;
    const dim3 grid = tile_grid((P.T * row_bytes + NT * 16 - 1) / (NT * 16), P.B, P.G * P.H, 1);
    if (launch_pdl(reorder_shift_kernel, grid, 0, stream, P) != cudaSuccess) return SPECDEC_ERR_CUDA;
    return cudaGetLastError() == cudaSuccess ? SPECDEC_OK : SPECDEC_ERR_CUDA;
}

template <class VT>
specdec_status launch_reorder(ReorderParams P, int64_t row_bytes, cudaStream_t stream) {
    P.row = row_bytes / static_cast<int64_t>(sizeof(VT));
    P.narrow = static_cast<double>(P.T) * static_cast<double>(P.row) < 4e9 ? 1 : 0;
    // Columns of a thread: 32 registers of state bytes.  16-byte columns, beams of
    // 5: 14.8 us, 15.5 us with twice as many; 2-byte columns, beams of 6: 31.9 us
    // with two, 44.8 us with one.
    constexpr int kRegs = sizeof(VT) >= 4 ? sizeof(VT) / 4 : 1;
    constexpr auto cols = [](int beams) { return 32 / kRegs / beams > 8 ? 8 : 32 / kRegs / beams < 1 ? 1 : 32 / kRegs / beams; };
    if (P.W <= 2) return launch_reorder_as<VT, 2, cols(2)>(P, stream);
    if (P.W <= 4) return launch_reorder_as<VT, 4, cols(4)>(P, stream);
    if (P.W <= 8) return launch_reorder_as<VT, 8, cols(8)>(P, stream);
    if (P.W <= 16) return launch_reorder_as<VT, 16, cols(16)>(P, stream);
    return launch_reorder_as<VT, 32, cols(32)>(P, stream);
}

template <class VT>
specdec_status launch_commit(CommitParams P, int64_t row_bytes, cudaStream_t stream) {
    P.row = row_bytes / static_cast<int64_t>(sizeof(VT));
    const dim3 grid = tile_grid((P.row + kCommitThreads - 1) / kCommitThreads, P.B, P.G, 1);
    if (launch_pdl(commit_path_kernel<VT>, grid, 0, stream, P, kCommitThreads) != cudaSuccess) return SPECDEC_ERR_CUDA;
    return cudaGetLastError() == cudaSuccess ? SPECDEC_OK : SPECDEC_ERR_CUDA;
}

}  // namespace
}  // namespace specdec

using namespace specdec;

extern "C" {

size_t specdec_workspace_size_beam(int B, int W, int K, int V, specdec_dtype dtype) {
    if (!dtype_ok(dtype) || B < 0 || B > SPECDEC_MAX_B || W < 1 || W > SPECDEC_MAX_BEAMS || K < 1 ||
        K > SPECDEC_MAX_BEAMS || V < 1 || V > SPECDEC_MAX_V)
        return 0;
    return make_beam_layout(B, W, V, dtype).total;
}

specdec_status specdec_beam_select(const void* logits, specdec_dtype dtype, int64_t row_stride,
                                   const float* beam_scores, const int32_t* finished, int eos_token, int B, int W,
                                   int K, int V, float* out_scores, int32_t* out_parents, int32_t* out_tokens,
                                   void* ws, size_t ws_bytes, struct CUstream_st* stream) {
    if (!dtype_ok(dtype)) return SPECDEC_ERR_UNSUPPORTED;
    if (B < 0 || B > SPECDEC_MAX_B || W < 1 || W > SPECDEC_MAX_BEAMS || K < 1 || K > SPECDEC_MAX_BEAMS || V < 1 ||
        V > SPECDEC_MAX_V)
        return SPECDEC_ERR_INVALID_ARG;
    if (finished != nullptr && (eos_token < 0 || eos_token >= V)) return SPECDEC_ERR_INVALID_ARG;
    if (B == 0) return SPECDEC_OK;
    const int64_t rows = static_cast<int64_t>(B) * W;
    if (!rows_fit(rows, row_stride, V)) return SPECDEC_ERR_INVALID_ARG;
    if (logits == nullptr || beam_scores == nullptr || out_scores == nullptr || out_parents == nullptr ||
        out_tokens == nullptr)
        return SPECDEC_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(logits) % static_cast<uintptr_t>(elem_size(dtype)) != 0)
        return SPECDEC_ERR_INVALID_ARG;
    const BeamLayout L = make_beam_layout(B, W, V, dtype);
    specdec_status st = check_ws(ws, ws_bytes, L.total);
    if (st != SPECDEC_OK) return st;
    // A request's outputs are written while other requests' inputs may not have been read.
    const int64_t got = static_cast<int64_t>(B) * K * 4;
    const Span out[3] = {{out_scores, got}, {out_parents, got}, {out_tokens, got}};
    const Span in[4] = {{beam_scores, rows * 4},
                        {finished, rows * 4},
                        {logits, ((rows - 1) * row_stride + V) * static_cast<int64_t>(elem_size(dtype))},
                        {ws, static_cast<int64_t>(L.total)}};
    if (outputs_meet(out, {0, -1, -1}, in)) return SPECDEC_ERR_INVALID_ARG;
    BeamParams P;
    P.logits = logits;
    P.row_stride = row_stride;
    P.scores = beam_scores;
    P.finished = finished;
    P.B = B;
    P.W = W;
    P.K = K;
    P.V = V;
    P.eos = eos_token;
    P.tiles = L.tiles;
    P.seg_tiles = L.seg_tiles;
    P.segs = L.segs;
    P.stats = reinterpret_cast<BeamStat*>(static_cast<char*>(ws) + L.stats);
    P.peaks = reinterpret_cast<float*>(static_cast<char*>(ws) + L.peaks);
    P.out_scores = out_scores;
    P.out_parents = out_parents;
    P.out_tokens = out_tokens;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return dtype == SPECDEC_BF16 ? launch_beam<BF16Tag>(P, s) : launch_beam<F32Tag>(P, s);
}

specdec_status specdec_reorder_states(const void* src, void* dst, const int32_t* parents, const int32_t* lengths,
                                      int64_t G, int B, int W, int64_t H, int64_t T, int64_t row_bytes,
                                      const int64_t src_strides[5], const int64_t dst_strides[5],
                                      struct CUstream_st* stream) {
    if (B < 0 || B > SPECDEC_MAX_B || W < 1 || W > SPECDEC_MAX_BEAMS || G < 0 || H < 0 || T < 0 || row_bytes < 0)
        return SPECDEC_ERR_INVALID_ARG;
    constexpr int64_t kMost = int64_t(1) << 40;
    if (G > kMost || H > kMost || T > kMost || row_bytes > kMost) return SPECDEC_ERR_INVALID_ARG;
    if (src_strides == nullptr || dst_strides == nullptr) return SPECDEC_ERR_INVALID_ARG;
    if (B == 0 || G == 0 || H == 0 || T == 0 || row_bytes == 0) return SPECDEC_OK;
    // Bytes of one beam of everything: every index below stays in 63 bits.
    if (static_cast<double>(G) * static_cast<double>(H) * B *
            (static_cast<double>(T) * static_cast<double>(row_bytes) + 65536.0) > 0x1p60)
        return SPECDEC_ERR_INVALID_ARG;
    if (src == nullptr || dst == nullptr || parents == nullptr) return SPECDEC_ERR_INVALID_ARG;
    for (int i = 0; i < 5; ++i)
        if (src_strides[i] < 0 || dst_strides[i] < 0 || src_strides[i] > (int64_t(1) << 52) ||
            dst_strides[i] > (int64_t(1) << 52) || (src == dst && src_strides[i] != dst_strides[i]))
            return SPECDEC_ERR_INVALID_ARG;
    ReorderParams P;
    P.src = static_cast<const char*>(src);
    P.dst = static_cast<char*>(dst);
    P.parents = parents;
    P.lengths = lengths;
    P.G = G;
    P.H = H;
    P.B = B;
    P.W = W;
    P.T = T;
    P.sg = src_strides[0];
    P.sb = src_strides[1];
    P.sw = src_strides[2];
    P.sh = src_strides[3];
    P.st = src_strides[4];
    P.dg = dst_strides[0];
    P.db = dst_strides[1];
    P.dw = dst_strides[2];
    P.dh = dst_strides[3];
    P.dt = dst_strides[4];
    P.flat = (T == 1 || (P.st == row_bytes && P.dt == row_bytes)) ? 1 : 0;
    P.in_place = src == dst ? 1 : 0;
    // The widest access that every address allows.
    uint64_t bits = reinterpret_cast<uintptr_t>(src) | reinterpret_cast<uintptr_t>(dst) |
                    static_cast<uint64_t>(row_bytes);
    const int64_t dims[5] = {G, B, W, H, T};
    for (int i = 0; i < 5; ++i)
        if (dims[i] > 1) bits |= static_cast<uint64_t>(src_strides[i]) | static_cast<uint64_t>(dst_strides[i]);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (bits % 16 == 0) return launch_reorder<uint4>(P, row_bytes, s);
    if (bits % 8 == 0) return launch_reorder<uint2>(P, row_bytes, s);
    if (bits % 4 == 0) return launch_reorder<uint32_t>(P, row_bytes, s);
    // 9 beams of 472 x 249 bf16 in 28 groups: 21.9 us put together from aligned
    // words, 33.9 us in 2-byte accesses (4-byte accesses beat both).
    if (!P.in_place && P.flat && T * row_bytes >= kShiftBytes) return launch_reorder_shift(P, row_bytes, s);
    if (bits % 2 == 0) return launch_reorder<uint16_t>(P, row_bytes, s);
    return launch_reorder<uint8_t>(P, row_bytes, s);
}

specdec_status specdec_commit_path(const void* src, int64_t src_group_stride, int64_t src_request_stride,
                                   int64_t src_row_stride, const int64_t* src_slots, int64_t src_slots_stride,
                                   int64_t src_rows, void* dst, int64_t dst_group_stride, int64_t dst_row_stride,
                                   const int64_t* dst_slots, int64_t dst_slots_stride, int64_t dst_rows,
                                   const int32_t* accept_len, const int32_t* accept_nodes, int64_t G, int B, int N,
                                   int max_depth, int64_t row_bytes, struct CUstream_st* stream) {
    if (B < 0 || B > SPECDEC_MAX_B || N < 0 || N + 1 > SPECDEC_MAX_TREE_NODES || max_depth < 1 ||
        max_depth > SPECDEC_MAX_DEPTH || G < 0 || row_bytes < 0)
        return SPECDEC_ERR_INVALID_ARG;
    constexpr int64_t kMost = int64_t(1) << 40;
    if (G > kMost || row_bytes > kMost || src_rows < 0 || dst_rows < 0 || src_rows > kMost || dst_rows > kMost)
        return SPECDEC_ERR_INVALID_ARG;
    const int64_t strides[5] = {src_group_stride, src_request_stride, src_row_stride, dst_group_stride,
                                dst_row_stride};
    for (int i = 0; i < 5; ++i)
        if (strides[i] < 0 || strides[i] > kMost) return SPECDEC_ERR_INVALID_ARG;
    if (B == 0 || G == 0 || row_bytes == 0) return SPECDEC_OK;
    if (static_cast<double>(G) * B * (static_cast<double>(row_bytes) + 65536.0) > 0x1p60)
        return SPECDEC_ERR_INVALID_ARG;
    if (src == nullptr || dst == nullptr || dst_slots == nullptr || accept_len == nullptr || accept_nodes == nullptr)
        return SPECDEC_ERR_INVALID_ARG;
    if (dst_slots_stride < max_depth + 1 || (src_slots != nullptr && src_slots_stride < N + 1))
        return SPECDEC_ERR_INVALID_ARG;
    if (src_row_stride < row_bytes || dst_row_stride < row_bytes) return SPECDEC_ERR_INVALID_ARG;
    CommitParams P;
    P.src = static_cast<const char*>(src);
    P.dst = static_cast<char*>(dst);
    P.accept_len = accept_len;
    P.accept_nodes = accept_nodes;
    P.src_slots = src_slots;
    P.dst_slots = dst_slots;
    P.src_slots_stride = src_slots_stride;
    P.dst_slots_stride = dst_slots_stride;
    P.G = G;
    P.B = B;
    P.nodes = N + 1;
    P.depth = max_depth;
    P.src_rows = src_rows;
    P.dst_rows = dst_rows;
    P.sg = src_group_stride;
    P.sb = src_slots != nullptr ? 0 : src_request_stride;
    P.sr = src_row_stride;
    P.dg = dst_group_stride;
    P.dr = dst_row_stride;
    const uint64_t bits = reinterpret_cast<uintptr_t>(src) | reinterpret_cast<uintptr_t>(dst) |
                          static_cast<uint64_t>(row_bytes | P.sg | P.sb | P.sr | P.dg | P.dr);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (bits % 16 == 0) return launch_commit<uint4>(P, row_bytes, s);
    if (bits % 8 == 0) return launch_commit<uint2>(P, row_bytes, s);
    if (bits % 4 == 0) return launch_commit<uint32_t>(P, row_bytes, s);
    if (bits % 2 == 0) return launch_commit<uint16_t>(P, row_bytes, s);
    return launch_commit<uint8_t>(P, row_bytes, s);
}

specdec_status specdec_plan_slots(const int32_t* seq_lens, const int32_t* accept_len, const int32_t* release,
                                  const int32_t* draft_offsets, int B, int k, int64_t total_drafts, int block_size,
                                  int32_t* block_tables, int64_t table_stride, int max_blocks,
                                  const int32_t* held_blocks, int32_t* free_ring, int ring_capacity,
                                  const int32_t* ring_state, int32_t* seq_lens_out, int32_t* held_out,
                                  int32_t* ring_state_out, int64_t* positions, int64_t* slots,
                                  struct CUstream_st* stream) {
    if (B < 0 || B > SPECDEC_MAX_B || k < 0 || k > SPECDEC_MAX_PLAN_ROWS - 1 || block_size < 1 ||
        block_size > SPECDEC_MAX_PLAN_ROWS || max_blocks < 1 || table_stride < max_blocks ||
        table_stride > (int64_t(1) << 40) || ring_capacity < 1)
        return SPECDEC_ERR_INVALID_ARG;
    if (draft_offsets != nullptr && (total_drafts < 0 || total_drafts > static_cast<int64_t>(B) * k))
        return SPECDEC_ERR_INVALID_ARG;
    if (B == 0) {  // nobody takes or returns a page: the ring stays as it is
        if (ring_state == nullptr || ring_state_out == nullptr || ring_state == ring_state_out) return SPECDEC_OK;
        if (meet({ring_state, 8}, {ring_state_out, 8})) return SPECDEC_ERR_INVALID_ARG;
        return cudaMemcpyAsync(ring_state_out, ring_state, 8, cudaMemcpyDeviceToDevice,
                               reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
                   ? SPECDEC_OK
                   : SPECDEC_ERR_CUDA;
    }
    if (seq_lens == nullptr || block_tables == nullptr || held_blocks == nullptr || free_ring == nullptr ||
        ring_state == nullptr || seq_lens_out == nullptr || held_out == nullptr || ring_state_out == nullptr ||
        positions == nullptr || slots == nullptr)
        return SPECDEC_ERR_INVALID_ARG;
    const int64_t rows = draft_offsets != nullptr ? B + total_drafts : static_cast<int64_t>(B) * (k + 1);
    const int64_t each = static_cast<int64_t>(B) * 4;
    const Span out[7] = {{seq_lens_out, each},
                         {held_out, each},
                         {ring_state_out, 8},
                         {positions, rows * 8},
                         {slots, rows * 8},
                         {block_tables, ((B - 1) * table_stride + max_blocks) * 4},
                         {free_ring, static_cast<int64_t>(ring_capacity) * 4}};
    const Span in[6] = {{seq_lens, each}, {held_blocks, each}, {ring_state, 8}, {accept_len, each}, {release, each},
                        {draft_offsets, each + 4}};
    if (outputs_meet(out, {0, 1, 2, -1, -1, -1, -1}, in)) return SPECDEC_ERR_INVALID_ARG;
    PlanParams P;
    P.seq_lens = seq_lens;
    P.accept_len = accept_len;
    P.release = release;
    P.offsets = draft_offsets;
    P.B = B;
    P.k = k;
    P.total = draft_offsets != nullptr ? total_drafts : static_cast<int64_t>(B) * k;
    P.block_size = block_size;
    P.tables = block_tables;
    P.table_stride = table_stride;
    P.max_blocks = max_blocks;
    P.held = held_blocks;
    P.ring = free_ring;
    P.capacity = ring_capacity;
    P.ring_state = ring_state;
    P.seq_out = seq_lens_out;
    P.held_out = held_out;
    P.ring_out = ring_state_out;
    P.positions = positions;
    P.slots = slots;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (B <= kPlanThreads && rows <= kPlanFusedRows) {
        // 64 requests of 6 rows: 4.7 us with 256 threads, 5.2 us with 1024; 141 of 20
        // rows: 8.7 and 6.4 us.
        const cudaError_t e = B <= kPlanFew && rows <= 4 * kPlanFew ? launch_pdl(plan_tables_kernel<true, kPlanFew>, dim3(1), 0, s, P, kPlanFew)
                                                                    : launch_pdl(plan_tables_kernel<true, kPlanThreads>, dim3(1), 0, s, P, kPlanThreads);
        if (e != cudaSuccess) return SPECDEC_ERR_CUDA;
        return cudaGetLastError() == cudaSuccess ? SPECDEC_OK : SPECDEC_ERR_CUDA;
    }
    if (launch_plan_tables(P, s) != cudaSuccess) return SPECDEC_ERR_CUDA;
    const dim3 grid(static_cast<unsigned>((B + NWARPS - 1) / NWARPS),
                    static_cast<unsigned>(static_cast<int64_t>(k) / kSlotTile + 1));
    if (launch_pdl(plan_slots_kernel, grid, 0, s, P) != cudaSuccess) return SPECDEC_ERR_CUDA;
    return cudaGetLastError() == cudaSuccess ? SPECDEC_OK : SPECDEC_ERR_CUDA;
}

}  // extern "C"
