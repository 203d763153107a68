// chunk_merge.cu -- the merge of row tiles that a chunk attention's plan cut, and the
// layout of its workspace.
#include <math.h>

#include <cuda_bf16.h>

#include "chunk.h"
#include "common.cuh"
#include "kernels.h"

namespace splash {
namespace {

// One row of a split row tile and Q quarters of its value dims from `quarter` on, by a warp:
// out = sum_s w_s part_s / sum_s w_s over the pieces, as in the split combine of the decode.  Grouped: piece s
// is the s-th of the row's own pieces, then of those over the group's prefix, `pre` rows of slots further on.
template <bool F32, int Q, bool GROUPS>
__device__ __forceinline__ void merge_row(const ChunkArgs& a, const ChunkSplit& sp, const ChunkRow& at, int row,
                                          int quarter, int lane, int pre_pieces, int64_t pre) {
    const float* lse = reinterpret_cast<const float*>(a.ws + a.plse_off) + int64_t(sp.slot) * (2 * kChunkRows) + row;
    const float4* part = reinterpret_cast<const float4*>(a.ws + a.pout_off) +
                         (int64_t(sp.slot) * (2 * kChunkRows) + row) * (kDv / 4) + quarter * 32 + lane;
    const int pieces = GROUPS ? sp.pieces + pre_pieces : sp.pieces;
    // rows of slots from the first piece's row on
    auto piece = [&](int s) -> int64_t {
        return int64_t(s) * (2 * kChunkRows) + (GROUPS && s >= sp.pieces ? pre : int64_t(0));
    };
    // lane s reads piece s; a NaN stays
    float m = -INFINITY;
    bool nan = false;
#pragma unroll 1
    for (int s0 = 0; s0 < pieces; s0 += 32) {
        const float x = s0 + lane < pieces ? lse[piece(s0 + lane)] : -INFINITY;
        nan |= __any_sync(0xffffffffu, x != x);
        m = fmaxf(m, x);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (nan) m = __int_as_float(0x7fc00000);
    float acc[Q][4] = {};
    float l = 0.f;
    if (m != -INFINITY)
#pragma unroll 1
        for (int s0 = 0; s0 < pieces; s0 += 32) {
            const int n = min(32, pieces - s0);
            const float x = lane < n ? lse[piece(s0 + lane)] : -INFINITY;
            const float mine = x == -INFINITY ? 0.f : expf(x - m);
            float t = mine;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
            l += t;
#pragma unroll(8 / Q)
            for (int s = 0; s < n; ++s) {
                const float wt = __shfl_sync(0xffffffffu, mine, s);
#pragma unroll
                for (int q = 0; q < Q; ++q) {
                    const float4 v = __ldcs(part + piece(s0 + s) * (kDv / 4) + q * 32);
                    acc[q][0] += wt * v.x;        // (an empty piece holds zeros)
                    acc[q][1] += wt * v.y;
                    acc[q][2] += wt * v.z;
                    acc[q][3] += wt * v.w;
                }
            }
        }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const int64_t o = int64_t(sp.tok + at.token) * a.H + a.head_lo + at.head;
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        const float4 v = make_float4(acc[q][0] * inv, acc[q][1] * inv, acc[q][2] * inv, acc[q][3] * inv);
        const int64_t to = o * (kDv / 4) + (quarter + q) * 32 + lane;
        if (F32) {
            reinterpret_cast<float4*>(a.out)[to] = v;
        } else {
            const __nv_bfloat162 x = __floats2bfloat162_rn(v.x, v.y), y = __floats2bfloat162_rn(v.z, v.w);
            reinterpret_cast<uint2*>(a.out)[to] =
                make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
        }
    }
    if (quarter == 0 && lane == 0) a.lse[o] = l == 0.f ? -INFINITY : m + logf(l);
}

// A warp per row, or per row and quarter of its dims when the rows alone would leave three quarters of the
// warps idle (one token over a long context: one row tile of up to a piece per pair).  Its time is
// a chain of loads (count and split, weights, partials), so one pass of the resident warps over the rows
// is what counts: with quarters always, the 64 splits of drafted tokens take 10.6 us instead of 6.
template <bool F32, bool GROUPS>
__global__ void __launch_bounds__(256) chunk_combine_kernel(const __grid_constant__ ChunkArgs a) {
    pdl_wait();
    const ChunkHeader* head = reinterpret_cast<const ChunkHeader*>(a.ws);
    const ChunkSplit* splits = reinterpret_cast<const ChunkSplit*>(a.ws + a.splits_off);
    const int lane = threadIdx.x & 31;
    const int64_t warps = int64_t(gridDim.x) * 8, first = int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5);
    // Grouped: a request's row tile may have few rows (16 of 128 for a single token and 16 heads), and the rows
    // that it cannot have are not visited
    const int per_split = GROUPS ? head->split_rows : 2 * kChunkRows;
    const int64_t rows = int64_t(head->num_splits) * per_split;
    const int parts = rows * 4 <= warps ? 4 : 1;
#pragma unroll 1
    for (int64_t w = first; w < rows * parts; w += warps) {
        const int64_t r = parts == 4 ? w >> 2 : w;
        int split, row;
        if (GROUPS) {                             // (splits times rows: the workspace has a slot of 262 KB for each split)
            split = int(uint32_t(r) / uint32_t(per_split));
            row = int(r) - split * per_split;
            if (!a.tile.flat) {                   // the row's token and head, to its place in the pair's rows
                const int token = a.tile.by_heads(row), second = token >= a.tile.tokens;
                row += second * (kChunkRows - a.tile.tokens * a.tile.heads);
            }
        } else {
            split = int(r / (2 * kChunkRows));
            row = int(r % (2 * kChunkRows));
        }
        const ChunkSplit sp = splits[split];
        const ChunkRow at = chunk_row(a.tile, a.Hs, sp.row0, sp.ntok, sp.pair_group, row / kChunkRows, row % kChunkRows);
        if (!at.live) continue;
        int pre_pieces = 0;
        int64_t pre = 0;
        if (GROUPS && sp.pre != 0) {
            if (sp.pre < 0) continue;
            // the row among the group's, and the group's row tile that holds it
            const int rel = sp.tok + at.token - sp.c0;
            int tile, in;
            if (a.tile.flat) {
                const int x = rel * a.Hs + at.head;   // (the call's rows are fewer than 2^31)
                tile = x / (2 * kChunkRows);
                in = x % (2 * kChunkRows);
            } else {                                  // one head group: more would leave one token to a pair
                tile = a.tile.by_per(rel);
                const int tok = rel - tile * a.tile.per, second = tok >= a.tile.tokens;
                in = second * kChunkRows + (tok - second * a.tile.tokens) * a.tile.heads + at.head;
            }
            const ChunkSplit& g = splits[sp.pre - 1 + tile];
            pre_pieces = g.pieces;
            pre = int64_t(g.slot - sp.slot - sp.pieces) * (2 * kChunkRows) + in - row;
        }
        if (parts == 4) merge_row<F32, 1, GROUPS>(a, sp, at, row, int(w) & 3, lane, pre_pieces, pre);
        else merge_row<F32, 4, GROUPS>(a, sp, at, row, 0, lane, pre_pieces, pre);
    }
}

}  // namespace

size_t chunk_layout(ChunkArgs& a) {
    const int64_t tiles = (int64_t(a.max_ctx) + kChunkKeys - 1) / kChunkKeys;
    const int64_t u = a.tile.row_tiles(a.total_q) + int64_t(a.B) * a.tile.pair_groups();   // each request rounds up
    const int64_t most = int64_t(kChunkSlotsPerPair) * a.pairs;
    int64_t slots = tiles <= 1 ? 0 : (tiles >= most || u * tiles > most ? most : u * tiles), more = 0;
    // Grouped: the groups' row tiles, and a partial result of every row tile, two of 262 KB for 128 rows.  Only the row tiles of
    // groups that are worth it use theirs, but which those are is in arrays on the device, and the size may not wait for it.
    if (a.mode == kChunkGroups) {
        more = a.tile.row_tiles(a.total_q) + a.groups;
        slots += u + more;
    }
    a.cap_slots = int(slots);
    a.cap_items = u + more + slots + a.pairs;   // a dealt plan pads the pairs to equal counts
    a.words_off = kChunkWordsOff;
    a.items_off = align256(a.words_off + sizeof(uint32_t) * 2 * size_t(a.pairs));
    a.splits_off = align256(a.items_off + sizeof(ChunkItem) * size_t(a.cap_items));
    a.plse_off = align256(a.splits_off + sizeof(ChunkSplit) * size_t(slots));
    a.pout_off = align256(a.plse_off + size_t(slots) * 2 * kChunkRows * sizeof(float));
    return align256(a.pout_off + size_t(slots) * 2 * kChunkRows * kDv * sizeof(float));
}

cudaError_t launch_chunk_combine(const ChunkArgs& a, int sms, cudaStream_t stream) {
    if (a.cap_slots == 0) return cudaSuccess;
    // enough blocks for every split of a small call (two slots each at least), eight a SM at most
    const int64_t want = int64_t(a.cap_slots + 1) / 2 * (2 * kChunkRows * 4 / 8);
    const int blocks = int(want < int64_t(sms) * 8 ? want : int64_t(sms) * 8);
    const dim3 g(blocks), b(256);
    if (a.mode == kChunkGroups)
        return a.out_f32 ? launch_pdl(chunk_combine_kernel<true, true>, g, b, 0, stream, a)
                         : launch_pdl(chunk_combine_kernel<false, true>, g, b, 0, stream, a);
    return a.out_f32 ? launch_pdl(chunk_combine_kernel<true, false>, g, b, 0, stream, a)
                     : launch_pdl(chunk_combine_kernel<false, false>, g, b, 0, stream, a);
}

}  // namespace splash
