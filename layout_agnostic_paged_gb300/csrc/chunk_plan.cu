// chunk_plan.cu -- the plan of a chunk attention call (which CTA pair works on which rows
// and keys) and the merge of row tiles that the plan cut.
//
// A row tile (128 query rows of one request, see chunk.h) is the natural unit of work, but
// there may be fewer of them than CTA pairs, with contexts of any length.  The plan cuts a
// request's row tiles along the keys into equal pieces when that shortens the call: it
// estimates the call's length in key tiles for five piece lengths, from the requests' lengths,
// and takes the best.  One block; a few microseconds.
#include <limits.h>
#include <math.h>

#include <cuda_bf16.h>

#include "chunk.h"
#include "common.cuh"
#include "kernels.h"

namespace splash {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kCuts = 4;                  // piece lengths tried: an even share of 1..4 rounds of the pairs
// Costs in key tiles, measured against the 1.5 us of a key tile: what an item costs beside its tiles
// (first loads, epilogue), what a partial costs to write and merge, and the merge's own latency.
constexpr float kItemCost = 2.0f;
constexpr float kSlotCost = 0.06f;
constexpr float kMergeCost = 1.5f;

struct Span {
    int c0, n;        // first row and number of new tokens
    int ctx;
    int u;            // row tiles
    int m;            // key tiles of the last token, the request's most
    bool bad;
};

__device__ __forceinline__ int key_tiles(const ChunkArgs& a, int seen) {
    const int e = min(seen, a.tok_hi);
    return e > a.tok_lo ? (e + kChunkKeys - 1) / kChunkKeys - a.tok_lo / kChunkKeys : 0;
}

__device__ __forceinline__ Span span_of(const ChunkArgs& a, int r) {
    Span s;
    const int c0 = a.cu_q[r], c1 = a.cu_q[r + 1], ctx = a.ctx_lens[r];
    s.c0 = min(max(c0, 0), a.total_q);
    s.n = min(max(c1, s.c0), a.total_q) - s.c0;
    s.ctx = min(max(ctx, 0), a.max_ctx);
    s.bad = s.c0 != c0 || c1 != s.c0 + s.n || s.ctx != ctx;
    const int pt = a.tile.pair_tokens();
    s.u = (s.n + pt - 1) / pt * a.tile.pair_groups();
    s.m = key_tiles(a, s.ctx);
    return s;
}

__device__ __forceinline__ int64_t block_sum(int64_t v, int64_t* scratch) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
    __syncthreads();
    int64_t s = scratch[threadIdx.x & 31];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    __syncthreads();
    return s;
}

// Exclusive prefix sum over the block; *total gets the sum.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* scratch, int64_t* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t s = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += x;
    }
    if (lane == 31) scratch[warp] = s;
    __syncthreads();
    int64_t w = scratch[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w += x;
    }
    const int64_t before = warp > 0 ? __shfl_sync(0xffffffffu, w, warp - 1) : 0;
    *total = __shfl_sync(0xffffffffu, w, 31);
    __syncthreads();
    return before + s - v;
}

__global__ void __launch_bounds__(kPlanThreads) chunk_plan_kernel(const __grid_constant__ ChunkArgs a) {
    __shared__ int64_t scratch[32];
    __shared__ int64_t item0[kPlanThreads + 1], slot0[kPlanThreads], split0[kPlanThreads];
    __shared__ int pieces[kPlanThreads], piece_tiles[kPlanThreads];
    pdl_wait();
    const int tid = threadIdx.x;
    ChunkHeader* head = reinterpret_cast<ChunkHeader*>(a.ws);
    ChunkItem* items = reinterpret_cast<ChunkItem*>(a.ws + a.items_off);
    ChunkSplit* splits = reinterpret_cast<ChunkSplit*>(a.ws + a.splits_off);

    // all the row tiles, all their key tiles (a row tile's are about the mean of its request's
    // first and last), the longest
    int64_t U = 0, C2 = 0, longest = 0;
    bool bad = false;
    for (int r = tid; r < a.B; r += kPlanThreads) {
        const Span s = span_of(a, r);
        U += s.u;
        C2 += int64_t(s.u) * (s.m + (s.n > 0 ? key_tiles(a, s.ctx - s.n + min(s.n, a.tile.pair_tokens())) : 0));
        if (s.u > 0 && s.m > longest) longest = s.m;
        bad |= s.bad;
    }
    U = block_sum(U, scratch);
    const float C = 0.5f * float(block_sum(C2, scratch));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const int64_t x = __shfl_xor_sync(0xffffffffu, longest, o);
        longest = x > longest ? x : longest;
    }
    if ((tid & 31) == 0) scratch[tid >> 5] = longest;
    bad = __syncthreads_or(bad);
    for (int i = 0; i < 32; ++i) longest = scratch[i] > longest ? scratch[i] : longest;
    __syncthreads();

    const float G = float(a.pairs);
    int best_len = INT_MAX;
    float best = U > 0 ? fmaxf(float(longest) + kItemCost, ceilf(float(U) / G) * (C / float(U) + kItemCost)) : 0.f;
    for (int w = 1; w <= kCuts && U > 0; ++w) {
        const int len = max(1, int(ceilf(C / (G * float(w)))));
        if (len >= longest) continue;
        int64_t n = 0, slots = 0;
        for (int r = tid; r < a.B; r += kPlanThreads) {
            const Span s = span_of(a, r);
            const int np = max(1, (s.m + len - 1) / len);
            n += int64_t(s.u) * np;
            if (np > 1) slots += int64_t(s.u) * np;
        }
        n = block_sum(n, scratch);
        slots = block_sum(slots, scratch);
        const float cost = fmaxf(float(len) + kItemCost, ceilf(float(n) / G) * (C / float(n) + kItemCost)) +
                           float(slots) * kSlotCost + kMergeCost;
        if (slots <= a.cap_slots && cost < best) {
            best = cost;
            best_len = len;
        }
    }

    int64_t item_base = 0, slot_base = 0, split_base = 0;
    const int per_block = a.tile.pair_tokens(), pg = a.tile.pair_groups();
    for (int r0 = 0; r0 < a.B; r0 += kPlanThreads) {
        const int r = r0 + tid;
        Span s = {};
        int np = 1;
        if (r < a.B) {
            s = span_of(a, r);
            np = best_len == INT_MAX ? 1 : max(1, (s.m + best_len - 1) / best_len);
        }
        const int64_t n = int64_t(s.u) * np;
        int64_t all, all_slots, all_splits;
        const int64_t i0 = block_scan(n, scratch, &all);
        const int64_t sl0 = block_scan(np > 1 ? n : 0, scratch, &all_slots);
        const int64_t sp0 = block_scan(np > 1 ? s.u : 0, scratch, &all_splits);
        item0[tid] = i0;
        slot0[tid] = slot_base + sl0;
        split0[tid] = split_base + sp0;
        pieces[tid] = np;
        piece_tiles[tid] = (s.m + np - 1) / np;
        if (tid == kPlanThreads - 1) item0[kPlanThreads] = all;
        __syncthreads();
        for (int64_t i = tid; i < all; i += kPlanThreads) {
            int lo = 0, hi = kPlanThreads;          // the last request with item0 <= i
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (item0[mid] <= i) lo = mid;
                else hi = mid;
            }
            const Span q = span_of(a, r0 + lo);
            const int k = pieces[lo];
            const int64_t local = i - item0[lo];
            const int tile = int(local / k), piece = int(local % k);
            ChunkItem it = {};
            it.r = r0 + lo;
            it.tok = q.c0 + tile / pg * per_block;
            it.ntok = q.c0 + q.n - it.tok;
            it.pair_group = tile % pg;
            it.seen = q.ctx - q.n + (it.tok - q.c0) + 1;
            it.ctx = q.ctx;
            const int t0 = a.tok_lo / kChunkKeys;
            const int nt = key_tiles(a, it.seen + min(it.ntok, per_block) - 1);
            it.t_lo = t0 + min(nt, piece * piece_tiles[lo]);
            it.t_hi = t0 + min(nt, (piece + 1) * piece_tiles[lo]);
            it.slot = k > 1 ? int(slot0[lo] + local) : -1;
            if (item_base + i < a.cap_items) items[item_base + i] = it;
            if (k > 1 && piece == 0) {
                ChunkSplit sp = {};
                sp.tok = it.tok;
                sp.ntok = it.ntok;
                sp.pair_group = it.pair_group;
                sp.slot = it.slot;
                sp.pieces = k;
                splits[split0[lo] + tile] = sp;
            }
        }
        item_base += all;
        slot_base += all_slots;
        split_base += all_splits;
        __syncthreads();
    }
    if (tid == 0) {
        // the capacities bound both counts; an item past them would be a fault of theirs
        head->status = bad ? uint32_t(SPLASH_DEVICE_BAD_INPUT) : 0u;
        head->num_items = int(item_base < a.cap_items ? item_base : a.cap_items);
        head->num_splits = int(split_base);
    }
}

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
    const int64_t rows = int64_t(head->num_splits) * (2 * kChunkRows);
    const int64_t warps = int64_t(gridDim.x) * 8;
    for (int64_t w = int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5); w < rows; w += warps) {
        const ChunkSplit sp = splits[w / (2 * kChunkRows)];
        const int row = int(w % (2 * kChunkRows)), c = row / kChunkRows, i = row % kChunkRows;
        const int qi = i / a.tile.heads + (a.tile.groups == 1 ? c * a.tile.tokens : 0);
        const int hs = (a.tile.groups == 1 ? 0 : (2 * sp.pair_group + c) * a.tile.heads) + i % a.tile.heads;
        if (i >= a.tile.heads * a.tile.tokens || qi >= sp.ntok || hs >= a.Hs) continue;
        float m = -INFINITY;
        for (int s = 0; s < sp.pieces; ++s) {
            const float x = plse[(int64_t(sp.slot) + s) * (2 * kChunkRows) + row];
            m = x != x ? x : fmaxf(m, x);          // a NaN stays
            if (m != m) break;
        }
        float acc[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[e] = 0.f;
        float l = 0.f;
        if (m != -INFINITY)
            for (int s = 0; s < sp.pieces; ++s) {
                const int64_t p = (int64_t(sp.slot) + s) * (2 * kChunkRows) + row;
                const float x = plse[p];
                if (x == -INFINITY) continue;
                const float wt = expf(x - m);
                l += wt;
                const float4* src = reinterpret_cast<const float4*>(pout + p * kDv) + lane * 2;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float4 v = __ldcs(src + (j >> 1) * 64 + (j & 1));
                    acc[4 * j] += wt * v.x;
                    acc[4 * j + 1] += wt * v.y;
                    acc[4 * j + 2] += wt * v.z;
                    acc[4 * j + 3] += wt * v.w;
                }
            }
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const int64_t o = int64_t(sp.tok + qi) * a.H + a.head_lo + hs;
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
    const int64_t u = (int64_t(a.total_q) / a.tile.pair_tokens() + a.B) * a.tile.pair_groups();
    const int64_t most = int64_t(kChunkSlotsPerPair) * a.pairs;
    const int64_t slots = tiles <= 1 ? 0 : (tiles >= most || u * tiles > most ? most : u * tiles);
    a.cap_slots = int(slots);
    a.cap_items = u + slots;
    a.items_off = 256;
    a.splits_off = align256(a.items_off + sizeof(ChunkItem) * size_t(a.cap_items));
    a.plse_off = align256(a.splits_off + sizeof(ChunkSplit) * size_t(slots));
    a.pout_off = align256(a.plse_off + size_t(slots) * 2 * kChunkRows * sizeof(float));
    return align256(a.pout_off + size_t(slots) * 2 * kChunkRows * kDv * sizeof(float));
}

cudaError_t launch_chunk_plan(const ChunkArgs& a, cudaStream_t stream) {
    return launch_pdl(chunk_plan_kernel, dim3(1), dim3(kPlanThreads), 0, stream, a);
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
