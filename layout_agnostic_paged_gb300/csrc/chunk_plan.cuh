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
//
// Its time is a chain of instructions that each run once, some 8 clocks apiece: warps without requests sit out,
// one warp alone weighs the ways, and divisions are products where the host knows the divisor.  A call of 64 requests has its
// plan after 7,500 clocks, 4 us (9,800 before that).
#pragma once

#include <limits.h>
#include <math.h>

#include <type_traits>

#include "chunk.h"
#include "common.cuh"

namespace splash {

constexpr int kPlanThreads = 512;         // threads of the block
// Row tiles of an even cut per thread (one makes shorter code, and grouped calls take the even cut more often).
template <int MODE>
constexpr int even_tiles = MODE == kChunkGroups ? 1 : 2;
constexpr int kMostPairs = 256;           // an even cut is for so many pairs
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
    // grouped: the request whose pages these are, the first key, and what becomes of the results
    int r, lo;
    int group;        // kOwn: a request's own keys are all it sees; kPrefix: a group's prefix; else the group
};
constexpr int kOwn = -1, kPrefix = -2;

// The groups of a call, in shared memory.
struct GroupScratch {
    int cu[kChunkMaxGroups + 1];
    int prefix[kChunkMaxGroups];   // shared keys; ~keys for a group that is not worth it
    int split0[kChunkMaxGroups];   // first split row tile
};

// The last index in [0, n) with from[i] <= x (from[0] <= x, ascending).
__device__ __forceinline__ int last_at_most(const int* from, int n, int x) {
    int lo = 0, hi = n;
#pragma unroll 1
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (from[mid] <= x) lo = mid;
        else hi = mid;
    }
    return lo;
}

// The rows of request r.
template <int MODE>
__device__ __forceinline__ Span request_span(const ChunkArgs& a, int r) {
    Span s;
    const int c0 = a.cu_q[r], c1 = a.cu_q[r + 1], ctx = a.ctx_lens[r];
    s.c0 = min(max(c0, 0), a.total_q);
    s.n = min(max(c1, s.c0), a.total_q) - s.c0;
    s.ctx = min(max(ctx, 0), a.max_ctx);
    s.bad_order = s.c0 != c0 || c1 != s.c0 + s.n;
    s.bad = s.bad_order || s.ctx != ctx;
    s.u = a.tile.row_tiles(s.n);
    s.r = r;
    s.lo = a.tok_lo;
    s.group = kOwn;
    s.m = key_tiles<kChunkPlain>(a, s.lo, s.ctx, s.ctx);
    if constexpr (MODE == kChunkWindow) s.m = min(s.m, most_window_tiles(a));
    return s;
}

// The i-th of the call's runs of rows.  Grouped: the groups' prefixes come first, then the requests, whose
// keys begin behind the prefix that they share.
template <int MODE>
__device__ __forceinline__ Span span_of(const ChunkArgs& a, int i, const GroupScratch& gs) {
    if constexpr (MODE == kChunkGroups) {
        if (i < a.groups) {
            Span s = {};
            s.r = gs.cu[i];
            s.lo = a.tok_lo;
            s.group = kPrefix;
            if (gs.prefix[i] > 0) {
                s.c0 = min(max(a.cu_q[s.r], 0), a.total_q);
                s.n = min(max(a.cu_q[gs.cu[i + 1]], s.c0), a.total_q) - s.c0;
                s.ctx = gs.prefix[i];
                s.u = a.tile.row_tiles(s.n);
                s.m = key_tiles<MODE>(a, s.lo, s.ctx, s.ctx);
            }
            return s;
        }
        const int r = i - a.groups;
        Span s = request_span<MODE>(a, r);
        if (s.n > 0 && r >= gs.cu[0] && r < gs.cu[a.groups]) {
            const int g = last_at_most(gs.cu, a.groups, r), p = gs.prefix[g];
            s.bad |= s.ctx - s.n < (p < 0 ? ~p : p);
            if (p > 0) {
                s.group = g;
                s.lo = max(a.tok_lo, p);
                s.m = key_tiles<MODE>(a, s.lo, s.ctx, s.ctx);
            }
        }
        return s;
    }
    return request_span<MODE>(a, i);
}

// The key tiles of all row tiles of a request, about: in a row as long as windows grow, then all the same.
template <int MODE>
__device__ __forceinline__ float tiles_about(const ChunkArgs& a, const Span& s) {
    if (MODE == kChunkGroups && s.group == kPrefix) return float(s.u) * float(s.m);
    const int past = s.ctx - s.n, seen = past + min(s.n, a.tile.pair_tokens());
    const float mean = 0.5f * float(s.m + key_tiles<MODE>(a, s.lo, past + 1, seen));
    if constexpr (MODE == kChunkWindow) {
        const float grow = float(min(max(a.window - past, 0), s.n)) / float(s.n);
        return float(s.u) * (grow * mean + (1.f - grow) * float(s.m));
    }
    return float(s.u) * mean;
}

// What the choice of a plan goes by: row tiles, key tiles (about), the most of a row tile, and flags.
constexpr uint32_t kBadLength = 1, kBadOrder = 2;
constexpr uint32_t kFarApart = 4;         // a request's row tiles sweep more than L2 holds
constexpr uint32_t kShared = 8;           // a group's rows are worked on together
struct Totals {
    int u, most, rows;
    float f;
    uint32_t flags;
};
template <bool GROUPS>
__device__ __forceinline__ void warp_totals(Totals& x) {
    x.u = __reduce_add_sync(0xffffffffu, x.u);
    x.most = __reduce_max_sync(0xffffffffu, x.most);
    if (GROUPS) x.rows = __reduce_max_sync(0xffffffffu, x.rows);
    x.flags = __reduce_or_sync(0xffffffffu, x.flags);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x.f += __shfl_xor_sync(0xffffffffu, x.f, o);
}

// Exclusive prefix sums of N values over the block's first `active` warps, which alone have any and get theirs;
// totals[] get the sums everywhere.
template <int N>
__device__ __forceinline__ void block_scan(int (&v)[N], int (&totals)[N], int (*scratch)[N], int active) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int s[N];
    if (warp < active) {
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
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < N; ++k) {
        int w = lane < active ? scratch[lane][k] : 0;
        if (warp < active) {
            const int own = w;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int x = __shfl_up_sync(0xffffffffu, w, o);
                if (lane >= o) w += x;
            }
            totals[k] = __shfl_sync(0xffffffffu, w, 31);
            v[k] = __shfl_sync(0xffffffffu, w - own, warp) + s[k] - v[k];
        } else {
            totals[k] = __reduce_add_sync(0xffffffffu, w);
        }
    }
    __syncthreads();
}

// Warps that hold n values, one a thread.
__device__ __forceinline__ int warps_of(int n) { return min(kPlanThreads, n + 31) >> 5; }

// The row tile `tile` of a run of rows.
template <int MODE>
__device__ __forceinline__ ChunkItem row_tile(const ChunkArgs& a, const Span& s, int tile, int* tiles) {
    ChunkItem it = {};
    it.r = s.r;
    it.ctx = s.ctx;
    it.flags = s.u <= kAlone ? kItemAlone : 0;
    it.slot = -1;
    int last;                                     // the tile's last token, from `tok` on
    if (a.tile.flat) {
        it.row0 = tile * (2 * kChunkRows);
        it.tok = s.c0;
        last = min(s.n - 1, a.tile.by_heads(it.row0 + 2 * kChunkRows - 1));
    } else {
        const int pg = a.tile.pair_groups(), per_block = a.tile.pair_tokens();
        it.tok = s.c0 + (pg == 1 ? tile : tile / pg) * per_block;
        it.pair_group = pg == 1 ? 0 : tile % pg;
        last = min(s.c0 + s.n - it.tok, per_block) - 1;
    }
    it.ntok = s.c0 + s.n - it.tok;
    if (MODE == kChunkGroups && s.group == kPrefix) {
        it.seen = s.ctx;
        it.flags |= kItemPrefix;
        *tiles = key_tiles<MODE>(a, s.lo, s.ctx, s.ctx, &it.base);
        return it;
    }
    it.seen = s.ctx - s.n + (it.tok - s.c0) + 1;
    *tiles = key_tiles<MODE>(a, s.lo, it.seen + a.tile.by_heads(it.row0), it.seen + last, &it.base);
    return it;
}

// Shared memory of the plan (its buffers are not in use yet).
struct PlanScratch {
    Totals totals[32];
    int cuts[32][2 * kCuts];
    struct {
        int U, longest, best_len, dealt;   // row tiles; key tiles of the longest; the plan
        int split_rows;                    // grouped: rows of a request's row tile, at most
        int len[kCuts];                    // piece lengths to try
        float C, best;
        bool bad, bad_order, is_even, cuts;
    } choice;
    int scan1[32][1], scan3[32][3];
    int from[kPlanThreads], slot0[kPlanThreads], split0[kPlanThreads];
    int pieces[kPlanThreads], piece_tiles[kPlanThreads];
    Span spans[kPlanThreads];
    int first, last;
    int bound[kMostPairs];             // an even cut's first position of every pair
    GroupScratch groups;
};

// What it gains, in key tiles of all pairs, to work on the m requests of a group, n new tokens, at once over their `keys`
// shared keys: the tiles that their own row tiles would take beyond the group's, less the group's items and a partial
// result of every row tile.  (The merge's latency comes once a call.)  Measured, 16 heads and single tokens: 128 requests over
// 512 keys take 31.4 us together and 31.3 apart, over 1,024 keys 33 and 42, over 8,192 keys 52 and 167.
__device__ __forceinline__ float gain_of_sharing(const ChunkArgs& a, int m, int n, int keys) {
    if (m < 2 || n < 2) return 0.f;
    const float own = float(m) * float(a.tile.row_tiles((n + m - 1) / m)), together = float(a.tile.row_tiles(n));
    const float tiles = float(key_tiles<kChunkGroups>(a, a.tok_lo, keys, keys));
    return (own - together) * tiles - kItemCost * together - kSlotCost * float(a.pairs) * (own + together);
}

// Reads the groups into shared memory; returns {a length is bad, the groups are out of order} for the thread's.
__device__ __forceinline__ int2 read_groups(const ChunkArgs& a, PlanScratch& sh) {
    GroupScratch& gs = sh.groups;
    int2 bad = {0, 0};
#pragma unroll 1
    for (int g = threadIdx.x; g <= a.groups; g += kPlanThreads) {
        const int r = a.cu_groups[g];
        gs.cu[g] = min(max(r, 0), a.B);
        bad.y |= r != gs.cu[g];
    }
    __syncthreads();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, active = warps_of(a.groups);
    if (warp < active) {
        float gain = 0.f;
#pragma unroll 1
        for (int g = threadIdx.x; g < a.groups; g += kPlanThreads) {
            const int r0 = gs.cu[g], r1 = gs.cu[g + 1], given = a.prefix_lens[g];
            const int p = min(max(given, 0), a.max_ctx);
            bad.x |= p != given;
            bad.y |= r1 < r0;
            const int c0 = min(max(a.cu_q[r0], 0), a.total_q), n = min(max(a.cu_q[max(r0, r1)], c0), a.total_q) - c0;
            const float x = gain_of_sharing(a, r1 - r0, n, p);
            gs.prefix[g] = x > 0.f ? p : ~p;
            gain += fmaxf(x, 0.f);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) gain += __shfl_xor_sync(0xffffffffu, gain, o);
        if (lane == 0) sh.totals[warp].f = gain;
    }
    __syncthreads();
    if (warp < active) {
        float all = 0.f;
#pragma unroll 1
        for (int w = 0; w < active; ++w) all += sh.totals[w].f;
        if (all <= kMergeCost * float(a.pairs))
#pragma unroll 1
            for (int g = threadIdx.x; g < a.groups; g += kPlanThreads)
                if (gs.prefix[g] >= 0) gs.prefix[g] = ~gs.prefix[g];
    }
    __syncthreads();
    return bad;
}

// The split row tile of an item whose first slot and number of pieces are given.
template <int MODE>
__device__ __forceinline__ ChunkSplit split_of(const ChunkArgs& a, const ChunkItem& it, int slot, int pieces, int group,
                                               const GroupScratch& gs) {
    ChunkSplit sp = {};
    sp.tok = it.tok;
    sp.ntok = it.ntok;
    sp.row0 = it.row0;
    sp.pair_group = it.pair_group;
    sp.slot = slot;
    sp.pieces = pieces;
    if constexpr (MODE == kChunkGroups) {
        if (group == kPrefix) sp.pre = -1;
        if (group >= 0) {
            sp.pre = gs.split0[group] + 1;
            sp.c0 = a.cu_q[gs.cu[group]];
        }
    }
    return sp;
}

// The items [x, y) of `pair`, written to the workspace's item array (by both of its CTAs, the same
// values).  `writer`: also write the header and the split row tiles.  Called by the whole block, whose last warp does
// `meanwhile` while the first one weighs the ways.
template <int MODE, typename F>
__device__ __forceinline__ int2 plan_items(const ChunkArgs& a, int pair, bool writer, PlanScratch& sh, F meanwhile) {
    const int tid = threadIdx.x;
    constexpr int NT = kPlanThreads;
    ChunkItem* items = reinterpret_cast<ChunkItem*>(a.ws + a.items_off);
    ChunkSplit* splits = reinterpret_cast<ChunkSplit*>(a.ws + a.splits_off);

    // all the row tiles, all their key tiles (a row tile's are about the mean of its request's first and
    // last), the longest, whether an even cut is allowed; requests with bad values, and with bad offsets
    Span mine = {};
    const int B = MODE == kChunkGroups ? a.groups + a.B : a.B;     // runs of rows
    const int lane = tid & 31, warp = tid >> 5, active = warps_of(B);
    int2 bad = {0, 0};
    if constexpr (MODE == kChunkGroups) bad = read_groups(a, sh);
    if (warp < active) {
        Totals sum = {};
        sum.flags = (bad.x ? kBadLength : 0) | (bad.y ? kBadOrder : 0);
#pragma unroll 1
        for (int r = tid; r < B; r += NT) {
            const Span s = span_of<MODE>(a, r, sh.groups);
            if (r == tid) mine = s;
            sum.u += s.u;
            if (s.n > 0) sum.f += tiles_about<MODE>(a, s);
            sum.flags |= (s.bad ? kBadLength : 0) | (s.bad_order ? kBadOrder : 0);
            const int64_t swept = MODE == kChunkWindow ? min(int64_t(s.ctx), int64_t(a.window) + s.n)
                                                       : (MODE == kChunkGroups ? int64_t(s.ctx) - s.lo : int64_t(s.ctx));
            if (s.u > 1 && swept * (kDqk * 2) > kSharedBytes) sum.flags |= kFarApart;
            if (s.u > 0) sum.most = max(sum.most, s.m);
            if (MODE == kChunkGroups && s.group == kPrefix && s.u > 0) sum.flags |= kShared;
            if (MODE == kChunkGroups && s.group != kPrefix) sum.rows = max(sum.rows, min(s.n, a.tile.per) * a.tile.heads);
        }
        warp_totals<MODE == kChunkGroups>(sum);
        if (lane == 0) sh.totals[warp] = sum;
    }
    __syncthreads();
    if (warp == NT / 32 - 1) meanwhile();
    if (warp == 0) {
        Totals sum = lane < active ? sh.totals[lane] : Totals{};
        warp_totals<MODE == kChunkGroups>(sum);
        const int U = sum.u, longest = sum.most;
        const float C = sum.f, G = float(a.pairs);
        float best = 0.f;
        bool may_cut = true, is_even = false;
        // (cuts make at most pairs - 1 more items, two partials each, and no more than there are tiles;
        // positions times pairs stay below 2^31)
        const int64_t tiles_most = int64_t(U) * longest;
        const bool room = U + (tiles_most < a.pairs ? tiles_most : a.pairs) <= a.cap_items &&
                          (MODE == kChunkGroups ? int64_t(U) + 2 * a.pairs : (tiles_most < 2 * a.pairs ? tiles_most : 2 * a.pairs)) <= a.cap_slots &&
                          tiles_most + 4 * int64_t(U) < (int64_t(1) << 31) / (a.pairs + 1);
        const bool even_fits = room && U <= even_tiles<MODE> * NT && a.pairs <= kMostPairs && !(sum.flags & kFarApart);
        if (MODE == kChunkGroups && even_fits && (sum.flags & kShared)) {
            is_even = true;                        // (the results of most row tiles are merged anyhow)
        } else {
            const float ideal = (C + kItemCost * float(U)) / G;
            best = U > 0 ? fmaxf(float(longest) + kItemCost, ceilf(float(U) / G) * (C / float(U) + kItemCost)) : 0.f;
            may_cut = a.cap_slots > 0 && U > 0 && best > 1.02f * ideal + kMergeCost;
            // an even cut: a run of every pair is (C + item costs) / G, and up to pairs - 1 cuts make two partials each
            const float even = ideal + kItemCost + 2.f * G * kSlotCost + kMergeCost;
            is_even = may_cut && even_fits && even < best;
        }
        if (lane < kCuts) sh.choice.len[lane] = max(1, int(ceilf(C / (G * float(lane + 1)))));
        if (lane == 0) {
            sh.choice.U = U;
            sh.choice.longest = longest;
            sh.choice.split_rows = min(sum.rows, 2 * kChunkRows);
            sh.choice.best_len = INT_MAX;
            sh.choice.dealt = U;                   // the items of a dealt plan
            sh.choice.C = C;
            sh.choice.best = best;
            sh.choice.bad = (sum.flags & kBadLength) != 0;
            sh.choice.bad_order = (sum.flags & kBadOrder) != 0;
            sh.choice.is_even = is_even;
            sh.choice.cuts = may_cut && !is_even;
        }
    }
    __syncthreads();
    // Requests whose rows overlap could ask for more items than there is room for, so offsets out of order
    // leave the whole call without work.
    if (sh.choice.bad_order) {
        if (writer && tid == 0)
            *reinterpret_cast<ChunkHeader*>(a.ws) = ChunkHeader{SPLASH_DEVICE_BAD_INPUT, kChunkMagic, 0, 2 * a.pairs};
        return make_int2(0, 0);
    }
    if (sh.choice.cuts) {
        if (warp < active) {
            int n[2 * kCuts] = {};
#pragma unroll 1
            for (int r = tid; r < B; r += NT) {
                const Span s = r == tid ? mine : span_of<MODE>(a, r, sh.groups);
#pragma unroll
                for (int w = 0; w < kCuts; ++w) {
                    const int len = sh.choice.len[w];
                    const int np = max(1, (s.m + len - 1) / len);
                    n[w] += s.u * np;
                    if (np > 1 || (MODE == kChunkGroups && s.group != kOwn)) n[kCuts + w] += s.u * np;
                }
            }
#pragma unroll
            for (int w = 0; w < 2 * kCuts; ++w) {
                n[w] = __reduce_add_sync(0xffffffffu, n[w]);
                if (lane == w) sh.cuts[warp][w] = n[w];
            }
        }
        __syncthreads();
        if (warp == 0) {
            // lane w: the w-th piece length
            const float C = sh.choice.C, G = float(a.pairs);
            int items_n = 0, slots_n = 0;
            if (lane < kCuts)
#pragma unroll 1
                for (int w = 0; w < active; ++w) {
                    items_n += sh.cuts[w][lane];
                    slots_n += sh.cuts[w][kCuts + lane];
                }
            const int len = sh.choice.len[lane & (kCuts - 1)];
            const float cost = fmaxf(float(len) + kItemCost, ceilf(float(items_n) / G) * (C / float(items_n) + kItemCost)) +
                               float(slots_n) * kSlotCost + kMergeCost;
            const bool fits = lane < kCuts && len < sh.choice.longest && slots_n <= a.cap_slots;
            float best = sh.choice.best;
            int at = -1;
#pragma unroll
            for (int w = 0; w < kCuts; ++w) {
                const float c = __shfl_sync(0xffffffffu, cost, w);
                if (__shfl_sync(0xffffffffu, int(fits), w) && c < best) {
                    best = c;
                    at = w;
                }
            }
            if (lane == at) {
                sh.choice.best_len = len;
                sh.choice.dealt = items_n;
            }
        }
        __syncthreads();
    }
    const int U = sh.choice.U, best_len = sh.choice.best_len, dealt = sh.choice.dealt;
    const bool is_even = sh.choice.is_even, bad_input = sh.choice.bad;

    const int t0 = MODE == kChunkPlain ? a.tok_lo / kChunkKeys : 0;
    int num_splits = 0;
    int2 range;
    // An even cut with E consecutive row tiles per thread; from[] holds the requests' first row tiles.
    auto cut_even = [&](auto row_tiles_a_thread) {
        constexpr int E = decltype(row_tiles_a_thread)::value;
        ChunkItem it[E] = {};
        int tiles[E] = {}, group[E], base = 0;
#pragma unroll 1
        for (int r0 = 0; r0 < B; r0 += NT) {
            const Span s = r0 + tid >= B ? Span{} : (r0 == 0 ? mine : span_of<MODE>(a, r0 + tid, sh.groups));
            int v[1] = {s.u}, tot[1];
            block_scan<1>(v, tot, sh.scan1, warps_of(B - r0));
            sh.from[tid] = base + v[0];
            sh.spans[tid] = s;
            if (MODE == kChunkGroups && r0 + tid < a.groups) sh.groups.split0[r0 + tid] = base + v[0];   // (each is split)
            __syncthreads();
#pragma unroll
            for (int e = 0; e < E; ++e) {
                const int x = tid * E + e;
                if (x >= base && x < base + tot[0]) {
                    const int k = last_at_most(sh.from, min(NT, B - r0), x);
                    it[e] = row_tile<MODE>(a, sh.spans[k], x - sh.from[k], &tiles[e]);
                    group[e] = sh.spans[k].group;
                }
            }
            base += tot[0];
            __syncthreads();
        }
        // positions along the sequence in tiles, an item's own cost included: pair j's run is
        // [j T / P, (j + 1) T / P), and a row tile's tiles lie at [A + own, A + own + tiles)
        const int own = int(kItemCost);
        const int holders = warps_of((U + E - 1) / E);
        int v[1] = {0}, W[1];
#pragma unroll
        for (int e = 0; e < E; ++e) v[0] += tid * E + e < U ? tiles[e] + own : 0;
        block_scan<1>(v, W, sh.scan1, holders);
        // Runs are own + kLeastPiece long at least, so that only one boundary can fall on a row tile's own
        // cost and first tiles, and one on its last: only its first and last piece can come out too
        // short, and then go to their neighbours.
        const uint32_t T = uint32_t(W[0]);
        const uint32_t P = max(1u, min(uint32_t(a.pairs), T / uint32_t(own + kLeastPiece)));
        if (tid < int(P)) sh.bound[tid] = int(uint32_t(tid) * T / P);
        __syncthreads();
        int np[E] = {}, j0[E] = {}, j1[E] = {}, A[E] = {};
        bool no_first[E] = {};
        auto cut = [&](int e, int j) -> int {     // first tile of pair j's piece
            if (j <= j0[e]) return 0;
            if (j > j1[e]) return tiles[e];
            const int x = sh.bound[j] - A[e] - own;
            return x < kLeastPiece ? 0 : (tiles[e] - x < kLeastPiece ? tiles[e] : x);
        };
        // items, partials and split row tiles
        int sums[3] = {}, totals[3];
        bool split_up[E] = {};
        int at = v[0];
#pragma unroll
        for (int e = 0; e < E; ++e) {
            A[e] = at;
            if (tid * E + e >= U) continue;
            j0[e] = int((uint32_t(at + 1) * P - 1) / T);
            j1[e] = int((uint32_t(at + own + tiles[e]) * P - 1) / T);
            np[e] = j1[e] - j0[e] + 1;
            if (np[e] > 1 && tiles[e] > 0) {
                no_first[e] = cut(e, j0[e] + 1) == 0;
                np[e] -= no_first[e] + (cut(e, j1[e]) == tiles[e]);
            } else {
                np[e] = 1;                        // (no key in sight: its rows become zeros)
            }
            split_up[e] = np[e] > 1 || (MODE == kChunkGroups && group[e] != kOwn);
            sums[0] += np[e];
            sums[1] += split_up[e] ? np[e] : 0;
            sums[2] += split_up[e];
            at += tiles[e] + own;
        }
        if constexpr (MODE == kChunkGroups) {
            block_scan<3>(sums, totals, sh.scan3, holders);
        } else {
            // in one word: at most 1,024 + pairs, 2 pairs, pairs
            int packed[1] = {sums[0] | sums[1] << 12 | sums[2] << 22}, tot[1];
            block_scan<1>(packed, tot, sh.scan1, holders);
            sums[0] = packed[0] & 0xfff;
            sums[1] = packed[0] >> 12 & 0x3ff;
            sums[2] = packed[0] >> 22;
            totals[2] = tot[0] >> 22;
        }
        if (tid == 0) {
            sh.first = INT_MAX;
            sh.last = 0;
        }
        __syncthreads();
        // the items are in the order of their pairs, so a pair's are a range
        int item = sums[0], slot = sums[1], split = sums[2];
#pragma unroll
        for (int e = 0; e < E; ++e) {
            if (np[e] > 0 && pair >= j0[e] && pair <= j1[e]) {
                const int lo = cut(e, pair), hi = cut(e, pair + 1);
                const bool empty = tiles[e] == 0;
                if (empty ? pair == j0[e] : hi > lo) {
                    const int k = empty ? 0 : pair - j0[e] - no_first[e];
                    ChunkItem o = it[e];
                    o.t_lo = t0 + (empty ? 0 : lo);
                    o.t_hi = t0 + (empty ? 0 : hi);
                    o.slot = split_up[e] ? slot + k : -1;
                    items[item + k] = o;
                    atomicMin(&sh.first, item + k);
                    atomicMax(&sh.last, item + k + 1);
                }
            }
            if (split_up[e]) {
                if (writer) splits[split] = split_of<MODE>(a, it[e], slot, np[e], group[e], sh.groups);
                slot += np[e];
                ++split;
            }
            item += np[e];
        }
        __syncthreads();
        range = make_int2(sh.first < sh.last ? sh.first : 0, sh.first < sh.last ? sh.last : 0);
        num_splits = totals[2];
    };
    if (is_even) {
        cut_even(std::integral_constant<int, even_tiles<MODE>>{});
    } else {
        // item i is the (i / pairs)-th of pair i mod pairs, whose items lie next to each other
        const int per_pair = a.by_pairs(dealt + a.pairs - 1);
        const int64_t x0 = int64_t(pair) * per_pair;
        int slot_base = 0, base = 0;
#pragma unroll 1
        for (int r0 = 0; r0 < B; r0 += NT) {
            const int r = r0 + tid;
            Span s = {};
            int np = 1;
            if (r < B) {
                s = r0 == 0 ? mine : span_of<MODE>(a, r, sh.groups);
                np = best_len == INT_MAX ? 1 : max(1, (s.m + best_len - 1) / best_len);
            }
            sh.spans[tid] = s;
            const int n = s.u * np;
            const bool split_up = np > 1 || (MODE == kChunkGroups && r < B && s.group != kOwn);
            int c[3] = {n, split_up ? n : 0, split_up ? s.u : 0}, tot[3] = {};
            if (MODE != kChunkGroups && best_len == INT_MAX) {
                int one[1] = {n}, sum[1];                        // nothing is split
                block_scan<1>(one, sum, sh.scan1, warps_of(B - r0));
                c[0] = one[0];
                tot[0] = sum[0];
            } else {
                block_scan<3>(c, tot, sh.scan3, warps_of(B - r0));
            }
            sh.from[tid] = c[0];
            sh.slot0[tid] = slot_base + c[1];
            sh.split0[tid] = c[2];
            sh.pieces[tid] = np;
            sh.piece_tiles[tid] = np == 1 ? s.m : (s.m + np - 1) / np;
            if (MODE == kChunkGroups && r < a.groups) sh.groups.split0[r] = num_splits + c[2];
            __syncthreads();
            // this pair's items among the batch's [base, base + tot[0])
            const int k0 = a.by_pairs(base - pair + a.pairs - 1);
#pragma unroll 1
            for (int k = (k0 > 0 ? k0 : 0) + tid;; k += NT) {
                const int64_t i = int64_t(k) * a.pairs + pair - base;
                if (i >= tot[0]) break;
                const int q = last_at_most(sh.from, min(NT, B - r0), int(i));
                const int pc = sh.pieces[q], local = int(i) - sh.from[q];
                const int tile = pc == 1 ? local : local / pc, piece = pc == 1 ? 0 : local % pc;
                int tiles;
                ChunkItem it = row_tile<MODE>(a, sh.spans[q], tile, &tiles);
                it.t_lo = t0 + min(tiles, piece * sh.piece_tiles[q]);
                it.t_hi = t0 + (piece + 1 == pc ? tiles : min(tiles, (piece + 1) * sh.piece_tiles[q]));
                if (pc > 1 || (MODE == kChunkGroups && sh.spans[q].group != kOwn)) it.slot = sh.slot0[q] + local;
                items[x0 + k] = it;
            }
            if (writer)
#pragma unroll 1
                for (int i = tid; i < tot[2]; i += NT) {
                    const int q = last_at_most(sh.split0, min(NT, B - r0), i);   // (others share a start with the next split request)
                    int tiles;
                    const ChunkItem it = row_tile<MODE>(a, sh.spans[q], i - sh.split0[q], &tiles);
                    splits[num_splits + i] = split_of<MODE>(a, it, sh.slot0[q] + (i - sh.split0[q]) * sh.pieces[q],
                                                            sh.pieces[q], sh.spans[q].group, sh.groups);
                }
            base += tot[0];
            slot_base += tot[1];
            num_splits += tot[2];
            __syncthreads();
        }
        const int64_t y0 = x0 + a.by_pairs(base - pair + a.pairs - 1);
        range = make_int2(int(x0), int(y0));
    }
    if (writer && tid == 0) {
        ChunkHeader* head = reinterpret_cast<ChunkHeader*>(a.ws);
        head->status = bad_input ? uint32_t(SPLASH_DEVICE_BAD_INPUT) : 0u;
        head->magic = kChunkMagic;
        head->num_splits = num_splits;
        head->words = 2 * a.pairs;
        if (MODE == kChunkGroups) head->split_rows = sh.choice.split_rows;
    }
    return range;
}

}  // namespace splash
