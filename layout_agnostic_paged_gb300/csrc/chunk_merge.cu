// chunk_merge.cu -- the merge of row tiles that a chunk attention's plan cut, and the
// layout of its workspace.
#include <math.h>

#include <cuda_bf16.h>

#include "chunk.h"
#include "common.cuh"
#include "kernels.h"

namespace splash {
namespace {

// One warp per row of a split row tile: out = sum_s w_s part_s / sum_s w_s, as in the
// split combine of the decode.
template <bool F32>
__global__ void __launch_bounds__(256) chunk_combine_kernel(const __grid_constant__ ChunkArgs a) {
    pdl_wait();
    const ChunkHeader* head = reinterpret_cast<const ChunkHeader*>(a.ws);
    const ChunkSplit* splits = reinterpret_cast<const ChunkSplit*>(a.ws + a.splits_off);
    const float* plse = reinterpret_cast<const float*>(a.ws + a.plse_off);
    const float* pout = reinterpret_cast<const float*>(a.ws + a.pout_off);
    const int lane = threadIdx.x & 31;
    const int64_t warps = int64_t(gridDim.x) * 8;
    int64_t w = int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5);
    // (the first split is read with the count: their round trips overlap; the array has room for it)
    ChunkSplit sp = splits[w / (2 * kChunkRows) < a.cap_slots ? w / (2 * kChunkRows) : 0];
    const int64_t rows = int64_t(head->num_splits) * (2 * kChunkRows);
    for (bool first = true; w < rows; w += warps, first = false) {
        if (!first) sp = splits[w / (2 * kChunkRows)];
        const int row = int(w % (2 * kChunkRows)), c = row / kChunkRows, i = row % kChunkRows;
        const ChunkRow at = chunk_row(a.tile, a.Hs, sp.row0, sp.ntok, sp.pair_group, c, i);
        if (!at.live) continue;
        const float* lse = plse + int64_t(sp.slot) * (2 * kChunkRows) + row;
        // lane s reads piece s; a NaN stays
        float m = -INFINITY;
        bool nan = false;
        for (int s0 = 0; s0 < sp.pieces; s0 += 32) {
            const float x = s0 + lane < sp.pieces ? lse[int64_t(s0 + lane) * (2 * kChunkRows)] : -INFINITY;
            nan |= __any_sync(0xffffffffu, x != x);
            m = fmaxf(m, x);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        if (nan) m = __int_as_float(0x7fc00000);
        float acc[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[e] = 0.f;
        float l = 0.f;
        if (m != -INFINITY)
            for (int s0 = 0; s0 < sp.pieces; s0 += 32) {
                const int n = min(32, sp.pieces - s0);
                const float x = lane < n ? lse[int64_t(s0 + lane) * (2 * kChunkRows)] : -INFINITY;
                const float mine = x == -INFINITY ? 0.f : expf(x - m);
                float t = mine;
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
                l += t;
#pragma unroll 2
                for (int s = 0; s < n; ++s) {
                    const float wt = __shfl_sync(0xffffffffu, mine, s);
                    if (wt == 0.f) continue;      // an empty piece
                    const float4* src = reinterpret_cast<const float4*>(
                                            pout + ((int64_t(sp.slot) + s0 + s) * (2 * kChunkRows) + row) * kDv) + lane * 2;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float4 v = __ldcs(src + (j >> 1) * 64 + (j & 1));
                        acc[4 * j] += wt * v.x;
                        acc[4 * j + 1] += wt * v.y;
                        acc[4 * j + 2] += wt * v.z;
                        acc[4 * j + 3] += wt * v.w;
                    }
                }
            }
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const int64_t o = int64_t(sp.tok + at.token) * a.H + a.head_lo + at.head;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            if (F32) {
                float4* d = reinterpret_cast<float4*>(static_cast<float*>(a.out) + o * kDv) + j * 64 + lane * 2;
#pragma unroll
                for (int k = 0; k < 2; ++k)
                    d[k] = make_float4(acc[8 * j + 4 * k] * inv, acc[8 * j + 4 * k + 1] * inv,
                                       acc[8 * j + 4 * k + 2] * inv, acc[8 * j + 4 * k + 3] * inv);
            } else {
                uint32_t v[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const __nv_bfloat162 b = __floats2bfloat162_rn(acc[8 * j + 2 * k] * inv, acc[8 * j + 2 * k + 1] * inv);
                    v[k] = *reinterpret_cast<const uint32_t*>(&b);
                }
                reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + o * kDv)[j * 32 + lane] =
                    make_uint4(v[0], v[1], v[2], v[3]);
            }
        }
        if (lane == 0) a.lse[o] = l == 0.f ? -INFINITY : m + logf(l);
    }
}

}  // namespace

size_t chunk_layout(ChunkArgs& a) {
    const int64_t tiles = (int64_t(a.max_ctx) + kChunkKeys - 1) / kChunkKeys;
    const int64_t u = a.tile.row_tiles(a.total_q) + int64_t(a.B) * a.tile.pair_groups();   // each request rounds up
    const int64_t most = int64_t(kChunkSlotsPerPair) * a.pairs;
    const int64_t slots = tiles <= 1 ? 0 : (tiles >= most || u * tiles > most ? most : u * tiles);
    a.cap_slots = int(slots);
    a.cap_items = u + slots + a.pairs;   // a dealt plan pads the pairs to equal counts
    a.words_off = kChunkWordsOff;
    a.items_off = align256(a.words_off + sizeof(uint32_t) * 2 * size_t(a.pairs));
    a.splits_off = align256(a.items_off + sizeof(ChunkItem) * size_t(a.cap_items));
    a.plse_off = align256(a.splits_off + sizeof(ChunkSplit) * size_t(slots));
    a.pout_off = align256(a.plse_off + size_t(slots) * 2 * kChunkRows * sizeof(float));
    return align256(a.pout_off + size_t(slots) * 2 * kChunkRows * kDv * sizeof(float));
}

cudaError_t launch_chunk_combine(const ChunkArgs& a, int sms, cudaStream_t stream) {
    if (a.cap_slots == 0) return cudaSuccess;
    // a warp per row: enough blocks for every split of a small call, eight a SM at most
    const int64_t rows = int64_t(a.cap_slots) * (2 * kChunkRows) / 16;
    const int blocks = int(rows < int64_t(sms) * 8 ? (rows > 0 ? rows : 1) : int64_t(sms) * 8);
    if (a.out_f32) return launch_pdl(chunk_combine_kernel<true>, dim3(blocks), dim3(256), 0, stream, a);
    return launch_pdl(chunk_combine_kernel<false>, dim3(blocks), dim3(256), 0, stream, a);
}

}  // namespace splash
