// chunk_merge.cu -- the merge of row tiles that a chunk attention's plan cut, and the
// layout of its workspace.
#include <math.h>

#include <cuda_bf16.h>

#include "chunk.h"
#include "common.cuh"
#include "kernels.h"

namespace splash {
namespace {

// out = sum_s w_s part_s / sum_s w_s over the pieces of a split row tile, as in the split combine of the
// decode.  A warp has one row and a quarter of its value dims: one token over a long context is one row
// tile of up to one piece per CTA pair, whose merge is then spread over 512 warps.
template <bool F32>
__global__ void __launch_bounds__(256) chunk_combine_kernel(const __grid_constant__ ChunkArgs a) {
    pdl_wait();
    const ChunkHeader* head = reinterpret_cast<const ChunkHeader*>(a.ws);
    const ChunkSplit* splits = reinterpret_cast<const ChunkSplit*>(a.ws + a.splits_off);
    const float* plse = reinterpret_cast<const float*>(a.ws + a.plse_off);
    const float* pout = reinterpret_cast<const float*>(a.ws + a.pout_off);
    const int lane = threadIdx.x & 31;
    constexpr int kWarps = 2 * kChunkRows * 4;   // of a split
    const int64_t warps = int64_t(gridDim.x) * 8;
    int64_t w = int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5);
    // (the first split is read with the count: their round trips overlap; the array has room for it)
    ChunkSplit sp = splits[w / kWarps < a.cap_slots ? w / kWarps : 0];
    const int64_t all = int64_t(head->num_splits) * kWarps;
    for (bool first = true; w < all; w += warps, first = false) {
        if (!first) sp = splits[w / kWarps];
        const int row = int(w % kWarps) >> 2, quarter = int(w) & 3, c = row / kChunkRows, i = row % kChunkRows;
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
        float acc[4] = {0.f, 0.f, 0.f, 0.f};
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
                const float4* src = reinterpret_cast<const float4*>(
                                        pout + ((int64_t(sp.slot) + s0) * (2 * kChunkRows) + row) * kDv) + quarter * 32 + lane;
#pragma unroll 8
                for (int s = 0; s < n; ++s) {
                    const float wt = __shfl_sync(0xffffffffu, mine, s);
                    const float4 v = __ldcs(src + int64_t(s) * (2 * kChunkRows * kDv / 4));
                    acc[0] += wt * v.x;           // (an empty piece holds zeros)
                    acc[1] += wt * v.y;
                    acc[2] += wt * v.z;
                    acc[3] += wt * v.w;
                }
            }
        const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[e] *= inv;
        const int64_t o = int64_t(sp.tok + at.token) * a.H + a.head_lo + at.head;
        if (F32) {
            reinterpret_cast<float4*>(static_cast<float*>(a.out) + o * kDv)[quarter * 32 + lane] =
                make_float4(acc[0], acc[1], acc[2], acc[3]);
        } else {
            const __nv_bfloat162 x = __floats2bfloat162_rn(acc[0], acc[1]), y = __floats2bfloat162_rn(acc[2], acc[3]);
            reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + o * kDv)[quarter * 32 + lane] =
                make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
        }
        if (quarter == 0 && lane == 0) a.lse[o] = l == 0.f ? -INFINITY : m + logf(l);
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
    // enough blocks for every split of a small call (two slots each at least), eight a SM at most
    const int64_t want = int64_t(a.cap_slots + 1) / 2 * (2 * kChunkRows * 4 / 8);
    const int blocks = int(want < int64_t(sms) * 8 ? want : int64_t(sms) * 8);
    if (a.out_f32) return launch_pdl(chunk_combine_kernel<true>, dim3(blocks), dim3(256), 0, stream, a);
    return launch_pdl(chunk_combine_kernel<false>, dim3(blocks), dim3(256), 0, stream, a);
}

}  // namespace splash
