// chunk_plan.cuh -- the plan of a chunk attention call: which CTA pair works on which rows
// and keys.  Every CTA computes it in its prologue, for its own pair's items.
//
// A row tile (128 query rows of one request, see chunk.h) is the natural unit of work, but
// there may be fewer of them than CTA pairs, with contexts of any length.  The plan has two ways to
// lay the row tiles over the pairs, and takes the one that it expects to be shorter:
//   - even: the row tiles' key tiles, in order, cut into one equal run per pair.  A run's ends may
//     fall inside a row tile, whose pieces are then merged.  For up to 1,024 row tiles, unless
//     the row tiles of one request would sweep a context larger than L2 out of step;
//   - dealt: row tile i goes to pair i mod pairs, so that the pairs sweep the same context together
//     and share it in L2.  Requests with long contexts are cut into equal pieces if that helps.
// As a kernel of its own the plan took 5 us for the smallest call and 11 us for 2,561 row tiles, and
// each call one more launch.
#pragma once

#include <limits.h>
#include <math.h>

#include "chunk.h"
#include "common.cuh"

namespace splash {

constexpr int kPlanThreads = 512;         // threads of the block
constexpr int kEvenTiles = 2;             // row tiles of an even cut per thread
constexpr int kCuts = 4;                  // piece lengths tried: an even share of 1..4 rounds of the pairs
// Costs in key tiles (1.15 us each): what an item costs beside its tiles (first loads, epilogue), what a
// partial costs to write and merge, and the merge's own latency.
constexpr float kItemCost = 3.0f;
constexpr float kSlotCost = 0.04f;
constexpr float kMergeCost = 1.5f;
constexpr int kLeastPiece = 1;            // an even cut leaves no piece of fewer tiles (2: drafted tokens take 55 us instead of 53.7)
constexpr int kAlone = 4;                 // row tiles of a request whose keys come from HBM, not from L2
// Contexts (bytes) whose row tiles may be swept out of step: what stays in the 129 MB L2.
constexpr int64_t kSharedBytes = 96ll << 20;

struct Span {
    int c0, n;        // first row and number of new tokens
    int ctx;
    int u;            // row tiles
    int m;            // key tiles of the last token, the request's most
    bool bad;         // the length or the offsets
    bool bad_order;   // the offsets
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
    s.bad_order = s.c0 != c0 || c1 != s.c0 + s.n;
    s.bad = s.bad_order || s.ctx != ctx;
    s.u = int(a.tile.row_tiles(s.n));
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
    ChunkItem it = {};
    it.r = r;
    it.ctx = s.ctx;
    it.alone = s.u <= kAlone;
    it.slot = -1;
    int last;                                     // the tile's last token, from `tok` on
    if (a.tile.flat) {
        it.row0 = tile * (2 * kChunkRows);
        it.tok = s.c0;
        last = min(s.n - 1, (it.row0 + 2 * kChunkRows - 1) / a.Hs);
    } else {
        const int pg = a.tile.pair_groups(), per_block = a.tile.pair_tokens();
        it.tok = s.c0 + (pg == 1 ? tile : tile / pg) * per_block;
        it.pair_group = pg == 1 ? 0 : tile % pg;
        last = min(s.c0 + s.n - it.tok, per_block) - 1;
    }
    it.ntok = s.c0 + s.n - it.tok;
    it.seen = s.ctx - s.n + (it.tok - s.c0) + 1;
    *tiles = key_tiles(a, it.seen + last);
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

// Shared memory of the plan (its buffers are not in use yet).
struct PlanScratch {
    Totals<4> totals[32];
    Totals<2 * kCuts> cuts[32];
    int scan1[32][1], scan3[32][3];
    int from[kPlanThreads], slot0[kPlanThreads], split0[kPlanThreads];
    int pieces[kPlanThreads], piece_tiles[kPlanThreads];
    Span spans[kPlanThreads];
    int first, last;
};

// The items [x, y) of `pair`, written to the workspace's item array (by both of its CTAs, the same
// values).  `writer`: also write the header and the split row tiles.  Called by the whole block.
__device__ __forceinline__ int2 plan_items(const ChunkArgs& a, int pair, bool writer, PlanScratch& sh) {
    const int tid = threadIdx.x;
    constexpr int NT = kPlanThreads;
    ChunkItem* items = reinterpret_cast<ChunkItem*>(a.ws + a.items_off);
    ChunkSplit* splits = reinterpret_cast<ChunkSplit*>(a.ws + a.splits_off);

    // all the row tiles, all their key tiles (a row tile's are about the mean of its request's first and
    // last), the longest, whether an even cut is allowed; requests with bad values, and with bad offsets
    Span mine = {};
    Totals<4> sum = {};
    for (int r = tid; r < a.B; r += NT) {
        const Span s = span_of(a, r);
        if (r == tid) mine = s;
        sum.v[0] += s.u;
        if (s.n > 0) sum.f += 0.5f * float(s.u) * float(s.m + key_tiles(a, s.ctx - s.n + min(s.n, a.tile.pair_tokens())));
        sum.v[1] |= s.bad;
        sum.v[2] |= s.u > 1 && int64_t(s.ctx) * (kDqk * 2) > kSharedBytes;
        sum.v[3] |= s.bad_order;
        if (s.u > 0) sum.most = max(sum.most, s.m);
    }
    block_totals(sum, sh.totals);
    // Requests whose rows overlap could ask for more items than there is room for, so offsets out of order
    // leave the whole call without work.
    if (sum.v[3]) {
        if (writer && tid == 0)
            *reinterpret_cast<ChunkHeader*>(a.ws) = ChunkHeader{SPLASH_DEVICE_BAD_INPUT, kChunkMagic, 0, 2 * a.pairs};
        return make_int2(0, 0);
    }
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
    const bool is_even = may_cut && room && U <= kEvenTiles * NT && a.pairs <= 256 && sum.v[2] == 0 && even < best;
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
        block_totals(n, sh.cuts);
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

    const int t0 = a.tok_lo / kChunkKeys;
    int num_splits = 0;
    int2 range;
    if (is_even) {
        // kEvenTiles consecutive row tiles per thread; from[] holds the requests' first row tiles
        ChunkItem it[kEvenTiles] = {};
        int tiles[kEvenTiles] = {}, base = 0;
        for (int r0 = 0; r0 < a.B; r0 += NT) {
            const Span s = r0 + tid >= a.B ? Span{} : (r0 == 0 ? mine : span_of(a, r0 + tid));
            int v[1] = {s.u}, tot[1];
            block_scan<1>(v, tot, sh.scan1);
            sh.from[tid] = base + v[0];
            sh.spans[tid] = s;
            __syncthreads();
#pragma unroll
            for (int e = 0; e < kEvenTiles; ++e) {
                const int x = tid * kEvenTiles + e;
                if (x >= base && x < base + tot[0]) {
                    const int k = last_at_most(sh.from, min(NT, a.B - r0), x);
                    it[e] = row_tile(a, sh.spans[k], r0 + k, x - sh.from[k], &tiles[e]);
                }
            }
            base += tot[0];
            __syncthreads();
        }
        // positions along the sequence in tiles, an item's own cost included: pair j's run is
        // [j T / P, (j + 1) T / P), and a row tile's tiles lie at [A + own, A + own + tiles)
        const int own = int(kItemCost);
        int v[1] = {0}, W[1];
#pragma unroll
        for (int e = 0; e < kEvenTiles; ++e) v[0] += tid * kEvenTiles + e < U ? tiles[e] + own : 0;
        block_scan<1>(v, W, sh.scan1);
        // Runs are own + kLeastPiece long at least, so that only one boundary can fall on a row tile's own
        // cost and first tiles, and one on its last: only its first and last piece can come out too
        // short, and then go to their neighbours.
        const uint32_t T = uint32_t(W[0]);
        const uint32_t P = max(1u, min(uint32_t(a.pairs), T / uint32_t(own + kLeastPiece)));
        int np[kEvenTiles] = {}, j0[kEvenTiles] = {}, j1[kEvenTiles] = {}, A[kEvenTiles] = {};
        bool no_first[kEvenTiles] = {};
        auto cut = [&](int e, int j) -> int {     // first tile of pair j's piece
            if (j <= j0[e]) return 0;
            if (j > j1[e]) return tiles[e];
            const int x = int(uint32_t(j) * T / P) - A[e] - own;
            return x < kLeastPiece ? 0 : (tiles[e] - x < kLeastPiece ? tiles[e] : x);
        };
        int packed[1] = {0}, packed_tot[1];
        int at = v[0];
#pragma unroll
        for (int e = 0; e < kEvenTiles; ++e) {
            A[e] = at;
            if (tid * kEvenTiles + e >= U) continue;
            j0[e] = int((uint32_t(at + 1) * P - 1) / T);
            j1[e] = int((uint32_t(at + own + tiles[e]) * P - 1) / T);
            np[e] = j1[e] - j0[e] + 1;
            if (np[e] > 1 && tiles[e] > 0) {
                no_first[e] = cut(e, j0[e] + 1) == 0;
                np[e] -= no_first[e] + (cut(e, j1[e]) == tiles[e]);
            } else {
                np[e] = 1;                        // (no key in sight: its rows become zeros)
            }
            // items, partials and split row tiles: at most 1,024 + pairs, 2 pairs, pairs
            packed[0] += np[e] | (np[e] > 1 ? np[e] : 0) << 12 | (np[e] > 1 ? 1 : 0) << 22;
            at += tiles[e] + own;
        }
        block_scan<1>(packed, packed_tot, sh.scan1);
        if (tid == 0) {
            sh.first = INT_MAX;
            sh.last = 0;
        }
        __syncthreads();
        // the items are in the order of their pairs, so a pair's are a range
        int item = packed[0] & 0xfff, slot = packed[0] >> 12 & 0x3ff, split = packed[0] >> 22;
#pragma unroll
        for (int e = 0; e < kEvenTiles; ++e) {
            if (np[e] > 0 && pair >= j0[e] && pair <= j1[e]) {
                const int lo = cut(e, pair), hi = cut(e, pair + 1);
                const bool empty = tiles[e] == 0;
                if (empty ? pair == j0[e] : hi > lo) {
                    const int k = empty ? 0 : pair - j0[e] - no_first[e];
                    ChunkItem o = it[e];
                    o.t_lo = t0 + (empty ? 0 : lo);
                    o.t_hi = t0 + (empty ? 0 : hi);
                    o.slot = np[e] > 1 ? slot + k : -1;
                    items[item + k] = o;
                    atomicMin(&sh.first, item + k);
                    atomicMax(&sh.last, item + k + 1);
                }
            }
            if (np[e] > 1) {
                if (writer) {
                    ChunkSplit sp = {};
                    sp.tok = it[e].tok;
                    sp.ntok = it[e].ntok;
                    sp.row0 = it[e].row0;
                    sp.pair_group = it[e].pair_group;
                    sp.slot = slot;
                    sp.pieces = np[e];
                    splits[split] = sp;
                }
                slot += np[e];
                ++split;
            }
            item += np[e];
        }
        __syncthreads();
        range = make_int2(sh.first < sh.last ? sh.first : 0, sh.first < sh.last ? sh.last : 0);
        num_splits = packed_tot[0] >> 22;
    } else {
        // item i is the (i / pairs)-th of pair i mod pairs, whose items lie next to each other
        const int per_pair = (dealt + a.pairs - 1) / a.pairs;
        const int64_t x0 = int64_t(pair) * per_pair;
        int slot_base = 0, base = 0;
        for (int r0 = 0; r0 < a.B; r0 += NT) {
            const int r = r0 + tid;
            Span s = {};
            int np = 1;
            if (r < a.B) {
                s = r0 == 0 ? mine : span_of(a, r);
                np = best_len == INT_MAX ? 1 : max(1, (s.m + best_len - 1) / best_len);
            }
            sh.spans[tid] = s;
            const int n = s.u * np;
            int c[3] = {n, np > 1 ? n : 0, np > 1 ? s.u : 0}, tot[3];
            block_scan<3>(c, tot, sh.scan3);
            sh.from[tid] = c[0];
            sh.slot0[tid] = slot_base + c[1];
            sh.split0[tid] = c[2];
            sh.pieces[tid] = np;
            sh.piece_tiles[tid] = (s.m + np - 1) / np;
            __syncthreads();
            // this pair's items among the batch's [base, base + tot[0])
            const int k0 = (base - pair + a.pairs - 1) / a.pairs;
            for (int k = (k0 > 0 ? k0 : 0) + tid;; k += NT) {
                const int64_t i = int64_t(k) * a.pairs + pair - base;
                if (i >= tot[0]) break;
                const int q = last_at_most(sh.from, NT, int(i));
                const int pc = sh.pieces[q], local = int(i) - sh.from[q];
                const int tile = pc == 1 ? local : local / pc, piece = pc == 1 ? 0 : local % pc;
                int tiles;
                ChunkItem it = row_tile(a, sh.spans[q], r0 + q, tile, &tiles);
                it.t_lo = t0 + min(tiles, piece * sh.piece_tiles[q]);
                it.t_hi = t0 + min(tiles, (piece + 1) * sh.piece_tiles[q]);
                if (pc > 1) it.slot = sh.slot0[q] + local;
                items[x0 + k] = it;
            }
            if (writer)
                for (int i = tid; i < tot[2]; i += NT) {
                    const int q = last_at_most(sh.split0, NT, i);   // (others share a start with the next split request)
                    int tiles;
                    const ChunkItem it = row_tile(a, sh.spans[q], r0 + q, i - sh.split0[q], &tiles);
                    ChunkSplit sp = {};
                    sp.tok = it.tok;
                    sp.ntok = it.ntok;
                    sp.row0 = it.row0;
                    sp.pair_group = it.pair_group;
                    sp.slot = sh.slot0[q] + (i - sh.split0[q]) * sh.pieces[q];
                    sp.pieces = sh.pieces[q];
                    splits[num_splits + i] = sp;
                }
            base += tot[0];
            slot_base += tot[1];
            num_splits += tot[2];
            __syncthreads();
        }
        const int64_t y0 = x0 + (base - pair + a.pairs - 1) / a.pairs;
        range = make_int2(int(x0), int(y0));
    }
    if (writer && tid == 0) {
        ChunkHeader* head = reinterpret_cast<ChunkHeader*>(a.ws);
        head->status = sum.v[1] ? uint32_t(SPLASH_DEVICE_BAD_INPUT) : 0u;
        head->magic = kChunkMagic;
        head->num_splits = num_splits;
        head->words = 2 * a.pairs;
    }
    return range;
}

}  // namespace splash
