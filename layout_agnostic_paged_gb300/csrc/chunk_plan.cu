// chunk_plan.cu -- the plan of a chunk attention call (which CTA pair works on which rows
// and keys) and the merge of row tiles that the plan cut.
//
// A row tile (128 query rows of one request, see chunk.h) is the natural unit of work, but
// there may be fewer of them than CTA pairs, with contexts of any length.  The plan has two ways to
// lay the row tiles over the pairs, and takes the one that it expects to be shorter:
//   - even: the row tiles' key tiles, in order, cut into one equal run per pair.  A run's ends may
//     fall inside a row tile, whose pieces are then merged.  For up to 1,024 row tiles, unless
//     the row tiles of one request would sweep a context larger than L2 out of step;
//   - dealt: row tile i goes to pair i mod pairs, so that the pairs sweep the same context together
//     and share it in L2.  Requests with long contexts are cut into equal pieces if that helps.
// One block; its time is latency, so the block is small for few requests.
#include <limits.h>
#include <math.h>

#include <cuda_bf16.h>

#include "chunk.h"
#include "common.cuh"
#include "kernels.h"

namespace splash {
namespace {

constexpr int kPlanThreads = 1024;        // most threads of the plan's block, and row tiles of an even cut
constexpr int kCuts = 4;                  // piece lengths tried: an even share of 1..4 rounds of the pairs
// Costs in key tiles (1.15 us each): what an item costs beside its tiles (first loads, epilogue), what a
// partial costs to write and merge, and the merge's own latency.
constexpr float kItemCost = 3.0f;
constexpr float kSlotCost = 0.04f;
constexpr float kMergeCost = 1.5f;
constexpr int kLeastPiece = 2;            // an even cut leaves no piece of fewer tiles
constexpr int kAlone = 4;                 // row tiles of a request whose keys come from HBM, not from L2
// Contexts (bytes) whose row tiles may be swept out of step: what stays in the 129 MB L2.
constexpr int64_t kSharedBytes = 96ll << 20;

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

// Over the whole block: sums of N ints and a float, and a maximum.
template <int N>
struct Totals {
    int v[N];
    float f;
    int most;
};
template <int N>
__device__ __forceinline__ void block_totals(Totals<N>& x, Totals<N>* scratch) {
    const int lane = threadIdx.x & 31;
    auto warp = [&]() {
#pragma unroll
        for (int k = 0; k < N; ++k) x.v[k] = __reduce_add_sync(0xffffffffu, x.v[k]);
        x.most = __reduce_max_sync(0xffffffffu, x.most);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) x.f += __shfl_xor_sync(0xffffffffu, x.f, o);
    };
    warp();
    if (lane == 0) scratch[threadIdx.x >> 5] = x;
    __syncthreads();
    x = lane < int(blockDim.x >> 5) ? scratch[lane] : Totals<N>{};
    warp();
    __syncthreads();
}

// Exclusive prefix sums of N values over the block; totals[] get the sums.
template <int N>
__device__ __forceinline__ void block_scan(int (&v)[N], int (&totals)[N], int (*scratch)[N]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int s[N];
#pragma unroll
    for (int k = 0; k < N; ++k) {
        s[k] = v[k];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, s[k], o);
            if (lane >= o) s[k] += x;
        }
        if (lane == 31) scratch[warp][k] = s[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < N; ++k) {
        int w = lane < int(blockDim.x >> 5) ? scratch[lane][k] : 0;
        const int own = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, w, o);
            if (lane >= o) w += x;
        }
        totals[k] = __shfl_sync(0xffffffffu, w, 31);
        v[k] = __shfl_sync(0xffffffffu, w - own, warp) + s[k] - v[k];
    }
    __syncthreads();
}

// The row tile `tile` of request r.
__device__ __forceinline__ ChunkItem row_tile(const ChunkArgs& a, const Span& s, int r, int tile, int* tiles) {
    const int pg = a.tile.pair_groups(), per_block = a.tile.pair_tokens();
    ChunkItem it = {};
    it.r = r;
    it.tok = s.c0 + (pg == 1 ? tile : tile / pg) * per_block;
    it.ntok = s.c0 + s.n - it.tok;
    it.pair_group = pg == 1 ? 0 : tile % pg;
    it.seen = s.ctx - s.n + (it.tok - s.c0) + 1;
    it.ctx = s.ctx;
    it.alone = s.u <= kAlone;
    it.slot = -1;
    *tiles = key_tiles(a, it.seen + min(it.ntok, per_block) - 1);
    return it;
}

// The last index in [0, n) with from[i] <= x (from[0] <= x, ascending).
__device__ __forceinline__ int last_at_most(const int* from, int n, int x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (from[mid] <= x) lo = mid;
        else hi = mid;
    }
    return lo;
}

__global__ void __launch_bounds__(kPlanThreads) chunk_plan_kernel(const __grid_constant__ ChunkArgs a) {
    __shared__ Totals<3> scratch_a[32];
    __shared__ Totals<2 * kCuts> scratch_b[32];
    __shared__ int scratch1[32][1], scratch3[32][3];
    __shared__ int from[kPlanThreads], slot0[kPlanThreads], split0[kPlanThreads];
    __shared__ int pieces[kPlanThreads], piece_tiles[kPlanThreads];
    __shared__ Span spans[kPlanThreads];
    pdl_wait();
    pdl_trigger();                                // the attention's blocks set themselves up while the plan runs
    const int tid = threadIdx.x, NT = blockDim.x;
    ChunkHeader* head = reinterpret_cast<ChunkHeader*>(a.ws);
    int2* ranges = reinterpret_cast<int2*>(a.ws + a.ranges_off);
    ChunkItem* items = reinterpret_cast<ChunkItem*>(a.ws + a.items_off);
    ChunkSplit* splits = reinterpret_cast<ChunkSplit*>(a.ws + a.splits_off);

    // all the row tiles, all their key tiles (a row tile's are about the mean of its request's first and
    // last), the longest, whether an even cut is allowed
    Span mine = {};
    Totals<3> sum = {};
    for (int r = tid; r < a.B; r += NT) {
        const Span s = span_of(a, r);
        if (r == tid) mine = s;
        sum.v[0] += s.u;
        if (s.n > 0) sum.f += 0.5f * float(s.u) * float(s.m + key_tiles(a, s.ctx - s.n + min(s.n, a.tile.pair_tokens())));
        sum.v[1] |= s.bad;
        sum.v[2] |= s.u > 1 && int64_t(s.ctx) * (kDqk * 2) > kSharedBytes;
        if (s.u > 0) sum.most = max(sum.most, s.m);
    }
    block_totals(sum, scratch_a);
    const int U = sum.v[0], longest = sum.most;
    const float C = sum.f;

    const float G = float(a.pairs);
    const float ideal = (C + kItemCost * float(U)) / G;
    int best_len = INT_MAX, dealt = U;            // the items of a dealt plan
    float best = U > 0 ? fmaxf(float(longest) + kItemCost, ceilf(float(U) / G) * (C / float(U) + kItemCost)) : 0.f;
    const bool may_cut = a.cap_slots > 0 && U > 0 && best > 1.02f * ideal + kMergeCost;
    // an even cut: a run of every pair is (C + item costs) / G, and up to pairs - 1 cuts make two partials each
    const float even = ideal + kItemCost + 2.f * G * kSlotCost + kMergeCost;
    // (cuts make at most pairs - 1 more items, two partials each, and no more than there are tiles;
    // positions times pairs stay below 2^31)
    const int64_t tiles_most = int64_t(U) * longest;
    const bool room = U + (tiles_most < a.pairs ? tiles_most : a.pairs) <= a.cap_items &&
                      (tiles_most < 2 * a.pairs ? tiles_most : 2 * a.pairs) <= a.cap_slots &&
                      tiles_most + 4 * int64_t(U) < (int64_t(1) << 31) / (a.pairs + 1);
    const bool is_even = may_cut && room && U <= NT && a.pairs <= 256 && a.pairs <= NT && sum.v[2] == 0 && even < best;
    if (!is_even && may_cut) {
        Totals<2 * kCuts> n = {};
        for (int r = tid; r < a.B; r += NT) {
            const Span s = r == tid ? mine : span_of(a, r);
#pragma unroll
            for (int w = 0; w < kCuts; ++w) {
                const int len = max(1, int(ceilf(C / (G * float(w + 1)))));
                const int np = max(1, (s.m + len - 1) / len);
                n.v[w] += s.u * np;
                if (np > 1) n.v[kCuts + w] += s.u * np;
            }
        }
        block_totals(n, scratch_b);
#pragma unroll
        for (int w = 0; w < kCuts; ++w) {
            const int len = max(1, int(ceilf(C / (G * float(w + 1)))));
            const float cost = fmaxf(float(len) + kItemCost, ceilf(float(n.v[w]) / G) * (C / float(n.v[w]) + kItemCost)) +
                               float(n.v[kCuts + w]) * kSlotCost + kMergeCost;
            if (len < longest && n.v[kCuts + w] <= a.cap_slots && cost < best) {
                best = cost;
                best_len = len;
                dealt = n.v[w];
            }
        }
    }

    int num_items = 0, num_splits = 0;
    if (is_even) {
        // one thread per row tile; from[] holds the requests' first row tiles
        ChunkItem it = {};
        int tiles = 0, base = 0;
        for (int r0 = 0; r0 < a.B; r0 += NT) {
            const Span s = r0 + tid >= a.B ? Span{} : (r0 == 0 ? mine : span_of(a, r0 + tid));
            int v[1] = {s.u}, tot[1];
            block_scan<1>(v, tot, scratch1);
            from[tid] = base + v[0];
            spans[tid] = s;
            __syncthreads();
            if (tid >= base && tid < base + tot[0]) {
                const int k = last_at_most(from, min(NT, a.B - r0), tid);
                it = row_tile(a, spans[k], r0 + k, tid - from[k], &tiles);
            }
            base += tot[0];
            __syncthreads();
        }
        const bool has = tid < U;
        // positions along the sequence in tiles, an item's own cost included: pair j's run is
        // [j T / P, (j + 1) T / P), and this row tile's tiles lie at [A + own, A + own + tiles)
        const int own = int(kItemCost);
        int v[1] = {has ? tiles + own : 0}, W[1];
        block_scan<1>(v, W, scratch1);
        const int A = v[0];
        const uint32_t T = uint32_t(W[0]), P = uint32_t(a.pairs);
        int j0 = 0, j1 = -1;
        if (has) {
            j0 = int((uint32_t(A + 1) * P - 1) / T);
            j1 = int((uint32_t(A + own + tiles) * P - 1) / T);
        }
        auto cut = [&](int j) -> int {            // first tile of pair j's piece
            if (j <= j0) return 0;
            if (j > j1) return tiles;
            const int x = int(uint32_t(j) * T / P) - A - own;
            return x < kLeastPiece ? 0 : (tiles - x < kLeastPiece ? tiles : x);
        };
        int np = 0;
        for (int j = j0; j <= j1; ++j) np += cut(j + 1) > cut(j);
        if (has && np == 0) np = 1;               // no key in sight: its rows become zeros
        // items, partials and split row tiles before this one's: at most 1,024 + pairs, 2 pairs, pairs
        int packed[1] = {np | (np > 1 ? np : 0) << 12 | (np > 1 ? 1 : 0) << 22}, packed_tot[1];
        block_scan<1>(packed, packed_tot, scratch1);
        const int c[3] = {packed[0] & 0xfff, packed[0] >> 12 & 0x3ff, packed[0] >> 22};
        const int tot[3] = {packed_tot[0] & 0xfff, 0, packed_tot[0] >> 22};
        // the items are in the order of their pairs, so a pair's are a range: first in from[], end in slot0[]
        for (int j = tid; j < a.pairs; j += NT) {
            from[j] = INT_MAX;
            slot0[j] = 0;
        }
        __syncthreads();
        if (has) {
            const int t0 = a.tok_lo / kChunkKeys;
            int k = 0;
            for (int j = j0; k < np; ++j) {
                const int lo = cut(j), hi = cut(j + 1);
                if (hi <= lo && tiles > 0) continue;
                it.t_lo = t0 + lo;
                it.t_hi = t0 + hi;
                it.slot = np > 1 ? c[1] + k : -1;
                items[c[0] + k] = it;
                atomicMin(&from[j], c[0] + k);
                atomicMax(&slot0[j], c[0] + k + 1);
                ++k;
            }
            if (np > 1) {
                ChunkSplit sp = {};
                sp.tok = it.tok;
                sp.ntok = it.ntok;
                sp.pair_group = it.pair_group;
                sp.slot = c[1];
                sp.pieces = np;
                splits[c[2]] = sp;
            }
        }
        __syncthreads();
        for (int j = tid; j < a.pairs; j += NT) ranges[j] = make_int2(from[j], slot0[j]);
        num_items = tot[0];
        num_splits = tot[2];
    } else {
        // item i is the (i / pairs)-th of pair i mod pairs, whose items lie next to each other
        const int per_pair = (dealt + a.pairs - 1) / a.pairs;
        int slot_base = 0;
        for (int r0 = 0; r0 < a.B; r0 += NT) {
            const int r = r0 + tid;
            Span s = {};
            int np = 1;
            if (r < a.B) {
                s = r0 == 0 ? mine : span_of(a, r);
                spans[tid] = s;
                np = best_len == INT_MAX ? 1 : max(1, (s.m + best_len - 1) / best_len);
            }
            const int n = s.u * np;
            int c[3] = {n, np > 1 ? n : 0, np > 1 ? s.u : 0}, tot[3];
            block_scan<3>(c, tot, scratch3);
            from[tid] = c[0];
            slot0[tid] = slot_base + c[1];
            split0[tid] = num_splits + c[2];
            pieces[tid] = np;
            piece_tiles[tid] = (s.m + np - 1) / np;
            __syncthreads();
            for (int i = tid; i < tot[0]; i += NT) {
                const int q = last_at_most(from, NT, i);
                const int k = pieces[q], local = i - from[q];
                const int tile = k == 1 ? local : local / k, piece = k == 1 ? 0 : local % k;
                int tiles;
                ChunkItem it = row_tile(a, spans[q], r0 + q, tile, &tiles);
                const int t0 = a.tok_lo / kChunkKeys;
                it.t_lo = t0 + min(tiles, piece * piece_tiles[q]);
                it.t_hi = t0 + min(tiles, (piece + 1) * piece_tiles[q]);
                if (k > 1) it.slot = slot0[q] + local;
                const uint32_t x = uint32_t(num_items + i), y = x / uint32_t(a.pairs);
                const int64_t at = int64_t(x - y * a.pairs) * per_pair + y;
                if (at < a.cap_items) items[at] = it;
                if (k > 1 && piece == 0) {
                    ChunkSplit sp = {};
                    sp.tok = it.tok;
                    sp.ntok = it.ntok;
                    sp.pair_group = it.pair_group;
                    sp.slot = it.slot;
                    sp.pieces = k;
                    splits[split0[q] + tile] = sp;
                }
            }
            num_items += tot[0];
            slot_base += tot[1];
            num_splits += tot[2];
            __syncthreads();
        }
        // (offsets that overlap, in a bad cu_q, could ask for more than the capacity)
        for (int j = tid; j < a.pairs; j += NT) {
            const int64_t x = int64_t(j) * per_pair, y = x + (num_items - j + a.pairs - 1) / a.pairs;
            ranges[j] = make_int2(int(x < a.cap_items ? x : a.cap_items), int(y < a.cap_items ? y : a.cap_items));
        }
    }
    if (tid == 0) {
        head->status = sum.v[1] ? uint32_t(SPLASH_DEVICE_BAD_INPUT) : 0u;
        head->num_items = num_items;
        head->num_splits = num_splits;
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
    const int64_t warps = int64_t(gridDim.x) * 8;
    int64_t w = int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5);
    // (the first split is read with the count: their round trips overlap; the array has room for it)
    ChunkSplit sp = splits[w / (2 * kChunkRows) < a.cap_slots ? w / (2 * kChunkRows) : 0];
    const int64_t rows = int64_t(head->num_splits) * (2 * kChunkRows);
    for (bool first = true; w < rows; w += warps, first = false) {
        if (!first) sp = splits[w / (2 * kChunkRows)];
        const int row = int(w % (2 * kChunkRows)), c = row / kChunkRows, i = row % kChunkRows;
        const int qi = i / a.tile.heads + (a.tile.groups == 1 ? c * a.tile.tokens : 0);
        const int hs = (a.tile.groups == 1 ? 0 : (2 * sp.pair_group + c) * a.tile.heads) + i % a.tile.heads;
        if (i >= a.tile.heads * a.tile.tokens || qi >= sp.ntok || hs >= a.Hs) continue;
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
    a.cap_items = u + slots + a.pairs;   // a dealt plan pads the pairs to equal counts
    a.ranges_off = 256;
    a.items_off = align256(a.ranges_off + sizeof(int2) * size_t(a.pairs));
    a.splits_off = align256(a.items_off + sizeof(ChunkItem) * size_t(a.cap_items));
    a.plse_off = align256(a.splits_off + sizeof(ChunkSplit) * size_t(slots));
    a.pout_off = align256(a.plse_off + size_t(slots) * 2 * kChunkRows * sizeof(float));
    return align256(a.pout_off + size_t(slots) * 2 * kChunkRows * kDv * sizeof(float));
}

cudaError_t launch_chunk_plan(const ChunkArgs& a, cudaStream_t stream) {
    // few requests and row tiles: a block whose barriers cost less
    const bool few = a.B <= 256 && a.cap_items - a.cap_slots - a.pairs <= 256;
    return launch_pdl(chunk_plan_kernel, dim3(1), dim3(few ? 256 : kPlanThreads), 0, stream, a);
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
