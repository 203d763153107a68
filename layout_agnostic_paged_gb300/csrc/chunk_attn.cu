// chunk_attn.cu -- causal attention of new tokens over the paged latent cache, on pairs of
// CTAs (cta_group::2 tensor cores, TMEM, TMA).
//
// With H heads reading one latent KV head, a new token is H query rows over the same keys,
// so a chunk is a matrix product with many rows: 2 * (576 + 512) operations per row and key.
// It is bound by the tensor cores; a single token per request is bound by HBM as in the decode.
//
// Per 128 query rows and 128 keys:
//   S [128 x 128] = Q [128 x 576] . K^T          36 MMAs of M 128, N 128, K 16
//   online softmax per row (fp32, exp2 domain, lazily rescaled running maximum)
//   O [128 x 512] += P [128 x 128] . V           16 MMAs of M 128, N 256, K 16
// The value is the latent prefix of the key.
//
// P is rounded to bf16, because an MMA takes both operands in one type and V is bf16: half a step, 2^-8 of a
// weight at most, and independent from weight to weight.  Measured, out is off by 0.0021 of its norm instead
// of the 0.0017 that its own rounding to bf16 gives; an fp32 out has the 0.0012 in between, as the decode's does.
// Everything else is fp32: scores, maxima, sums, O and lse.
//
// Why a pair.  O of 128 rows fills the whole TMEM of one SM (512 fp32 columns), and Q of 128
// rows plus one key tile is more than its shared memory.  A pair of CTAs splits the rows: each has
// 64 (Q 72 KB, O in 256 columns because an M = 128 pair MMA puts its two column halves on
// lanes 0-63 and 64-127), so a thread's lane is one row and one half of the columns, and the
// softmax needs no exchange beyond its own CTA.  The hardware splits B between the CTAs: for
// S each holds 64 of the 128 keys, for O each holds its 256 of the 512 value dims of all
// 128 keys.  These are different cuts of the cache, so K and V are loaded separately (the V
// bytes come from L2).  Issued in uniform control flow a tile's 52 MMAs take 2,178 clocks, the full
// rate (2,988 from a branch that one lane takes).
//
// Shared memory of each CTA: Q 72 KB, K 72 KB, V 64 KB, P 16 KB.  K and V have one buffer
// each: a piece of it is loaded again as soon as the MMAs that read it are done, and needed a
// whole tile later, because S of the next tile is computed before O of this one.
//
// Roles (512 threads): warp 0 loads Q and K (and warp 3 every other copy of K for pages below 64),
// warp 2 loads V, the leader's warp 1 issues every MMA, warps 4-11 run the softmax, warps 12-15
// store the results beside the next item's first tiles.
//
// Measured.  The last 1,024 tokens of a 16K-token prompt, 128 heads (4.53 TFLOP): 2.52 ms, 1,795 TF/s,
// 93% of the library's burst rate for matrix products and more than its sustained one: the SMs run at
// 1.6 GHz there, held by power.  16 requests of 1-256 tokens over up to 3,840: 0.975 to 1.07 ms (81 to
// 89%).  Four whole prompts of 257-1,024 tokens: 0.24 ms (55%), an item being three tiles long on average
// and the causal edge half of one; what is left is the chain from an item's last scores over
// their softmax and O to the next item's first (6,400 clocks for an item of one tile).  64 requests of 4
// drafted tokens, 16 heads, over 512-4,096 (173 MB): 50 us, 3.4 TB/s: 15 tiles a pair, each held
// by the latency of its keys, between the start (5 us) and the merge (6 us).
//
// Windows.  A token sees its last keys and some first ones, two ranges that move from row tile to row tile.  They are
// laid end to end in blocks of 64 keys, two to a tile, so that four first tokens cost half a tile and a window
// begins within 64 keys of its first.  1,024 tokens over a window of 4,096 and 64 first tokens, 128 heads: 0.67 to 0.73 ms,
// 83 to 90% of the library's rate; three prompts of 700-2,600 tokens over a window of 512: 0.47 to 0.52 ms, 54 to 60%: an
// item is five tiles for 516 keys, and its Q (72 KB a CTA) comes in at the same 62 bytes a clock as its keys.
//
// Groups.  Requests with a common prefix have its keys multiplied with all their rows at once: the group's rows make
// row tiles of their own, every row tile's result is a partial one, and the merge joins a request's with its group's.
// 256 single tokens of 16 heads behind 32,768 shared keys: 0.22 to 0.23 ms (68% of the library's rate) where each by itself
// takes 1.28 ms; 64 behind 8,192: 37 us instead of 103, of which the tiles take 14.
//
// Code length counts: the roles' loops share an instruction cache, and a launch fetches the code of its first tiles
// anew.  Loops of the loading warps that are not unrolled took whole prompts from 254 to 242 us, the plan's decisions in one
// copy each drafted tokens from 52.4 to 51.5 us.
//
// The tensor cores' fp32 additions truncate, so O comes out small where one item sums very many keys: by
// 0.05% over 131,072 keys and 0.44% over a million, measured with values of one sign, which is the worst case
// (0.07% over a million normal ones); l, summed in registers with rounding, does not share it.
#include <math.h>

#include "chunk.h"
#include "chunk_plan.cuh"
#include "common.cuh"
#include "kernels.h"
#include "pair.cuh"
#include "vec32.cuh"

namespace splash {
namespace {

constexpr int kBlk = kChunkRows * 128;           // 64 rows of one 64-dim block: 8 KB
constexpr int kKBlks = kChunkKBlocks;
constexpr int kKGroups = 9 / kKBlks;             // K is loaded and released in groups of its 9 blocks
constexpr int kQOff = 0;
constexpr int kKOff = 9 * kBlk;
constexpr int kVOff = kKOff + 9 * kBlk;          // [2 halves of the keys][pages][4 blocks][rows][128 B]
constexpr int kVHalf = 4 * kBlk;
constexpr int kPOff = kVOff + 2 * kVHalf;        // [2 halves of the keys][64 rows][128 B]
constexpr int kBarOff = kPOff + 2 * kBlk;
// barriers: K full / empty, V full / empty, Q full / empty, S full, P full, O full / free,
// row statistics full / empty, drain
constexpr int kNumBars = 4 * kKGroups + 4 + 2 + 2 + 4 + 2 + 1;
constexpr int kMiscOff = kBarOff + kNumBars * 8;
constexpr int kMaxOff = kMiscOff + 32;           // row maxima [2 tiles][4 shares of the keys][64]; row sums reuse them
constexpr int kFinOff = kMaxOff + 8 * kChunkRows * 4;   // an item's final (maximum, sum) of every row
constexpr int kSmem = kFinOff + kChunkRows * 8;
static_assert(kSmem <= 232448, "shared memory budget");
constexpr int kThreads = kPlanThreads;
constexpr int kSoftThreads = 256;
constexpr int kSCol = 384;                       // TMEM: halves of O in columns 0, 128 and 256, S in 2 x 64
constexpr int kTmemCols = 512;

// O takes 256 columns, and 384 are left beside S: three buffers of half an O (value dims 0-127 and
// 128-255 of each CTA).  An item's halves are in the buffers `o` and the one after it, the next
// item's begin two on, so that the next item waits for the results of the first half only.
__device__ __forceinline__ uint32_t o_second(uint32_t o) { return o == 2 ? 0 : o + 1; }
__device__ __forceinline__ uint32_t o_next(uint32_t o) { return o == 0 ? 2 : o - 1; }

// What a key tile adds to the limit of a wait that lasts as long as an item: a tile takes 1.15 to 1.7 us.
constexpr uint64_t kTileLimitNs = 20000;

constexpr float kTau = 8.0f;                     // rescale O when a score beats the maximum by 2^8

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&v);
}

// The low n bits, for any n.
__device__ __forceinline__ uint32_t low_bits(int n) { return n <= 0 ? 0u : 0xffffffffu >> (32 - min(n, 32)); }

// The page id behind a key, or -1 where there is none (past the context, or a bad id).
__device__ __forceinline__ int page_of(const ChunkArgs& a, const int32_t* table, int key, int ctx) {
    if (key >= ctx) return -1;
    const int id = table[key >> a.P_log];
    return id >= 0 && id < a.num_pages ? id : -1;
}

// First key of a half of tile t.
template <int MODE>
__device__ __forceinline__ int tile_key(const ChunkArgs& a, const ChunkItem& it, int t, int half) {
    if constexpr (MODE == kChunkWindow) {
        const int b = 2 * t + half;
        return (b + (b < a.sink_blocks ? a.tok_lo / kChunkRows : it.base)) * kChunkRows;
    }
    const int from = MODE == kChunkGroups ? it.base & ~(kChunkRows - 1) : 0;
    return from + t * kChunkKeys + half * kChunkRows;
}

// No row of the item sees keys before it.
template <int MODE>
__device__ __forceinline__ int first_key(const ChunkArgs& a, const ChunkItem& it) {
    return MODE == kChunkGroups ? it.base : a.tok_lo;
}

// Where the keys of an item begin, the first tokens aside.  Keys [key, key + n) that lie before it are seen by none of
// its rows: their page may be gone, and nothing of it is read.
template <int MODE>
__device__ __forceinline__ int item_start(const ChunkArgs& a, const ChunkItem& it) {
    return MODE == kChunkWindow ? max(it.seen + a.tile.by_heads(it.row0), 1) - a.window : (MODE == kChunkGroups ? it.base : 0);
}
template <int MODE>
__device__ __forceinline__ bool left_behind(const ChunkArgs& a, int start, int key, int n) {
    return MODE != kChunkPlain && key + n <= start && (MODE != kChunkWindow || key >= a.sinks);
}

// Asks for the first keys of every request (grouped: of every prefix) into L2 while the plan is made, during which HBM has
// nothing else to do: block b's share of the units of 64 keys, `early` to a request.  A window over 64 single tokens 30.5 to
// 29.0 us, drafted tokens 51.1 to 50.1, 64 single tokens behind a prefix 38.6 to 37.4.  Twice the units change nothing;
// the smallest call (2 requests of 100 keys), whose code it lengthens, takes 10.7 us where it took 10.6.
template <int MODE>
__device__ __forceinline__ void ask_early(const ChunkArgs& a, int lane) {
    const int R = min(a.P, kChunkRows), loads = kChunkRows / R;
    const int u = int(blockIdx.x + gridDim.x * (lane / loads)), i = a.by_early(u);
    if (lane >= kEarlyUnits * loads || i >= (MODE == kChunkGroups ? a.groups : a.B)) return;
    const int r = MODE == kChunkGroups ? min(max(a.cu_groups[i], 0), a.B - 1) : i;
    const int end = min(min(MODE == kChunkGroups ? a.prefix_lens[i] : a.ctx_lens[i], a.max_ctx), a.tok_hi);
    int start = a.tok_lo;
    if (MODE == kChunkWindow) start = max(start, end - min(max(a.cu_q[r + 1] - a.cu_q[r], 0), a.total_q) + 1 - a.window);
    const uint32_t key = (uint32_t(start) / kChunkRows + uint32_t(u - i * a.early)) * kChunkRows + lane % loads * R;
    if (end <= 0 || key >= uint32_t(end)) return;
    const int id = page_of(a, a.block_table + int64_t(r) * a.max_pages, int(key), end);
    if (id >= 0) prefetch_l2(a.kv + ((int64_t(id) << a.P_log) + (key & (a.P - 1))) * (kDqk * 2), R * kDqk * 2);
}

template <int MODE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    chunk_attn_kernel(const __grid_constant__ ChunkMaps maps, const __grid_constant__ ChunkArgs a) {
    extern __shared__ __align__(1024) uint8_t smem[];
    if (smem_u32(smem) & 1023) {                 // no room is left to align it here
        if (threadIdx.x == 0) {
            ChunkHeader* h = reinterpret_cast<ChunkHeader*>(a.ws);
            reinterpret_cast<uint32_t*>(a.ws + a.words_off)[blockIdx.x] = SPLASH_DEVICE_TIMEOUT;
            if (blockIdx.x == 0) *h = ChunkHeader{SPLASH_DEVICE_TIMEOUT, kChunkMagic, 0, 2 * a.pairs};
        }
        return;
    }
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kBarOff);
    uint64_t* k_full = bars;                     // leader's: both CTAs' loads
    uint64_t* k_empty = k_full + kKGroups;       // each CTA's own, as every *_empty
    uint64_t* v_full = k_empty + kKGroups;       // leader's
    uint64_t* v_empty = v_full + 2;
    uint64_t* q_full = v_empty + 2;              // leader's
    uint64_t* q_empty = q_full + kKGroups;       // Q in the groups of K
    uint64_t* s_full = q_empty + kKGroups;       // each CTA's
    uint64_t* p_full = s_full + 2;               // leader's, of each half of the keys: the softmax warps of both CTAs
    uint64_t* o_full = p_full + 2;               // each CTA's: the item's last PV is done
    uint64_t* o_free = o_full + 1;               // leader's, of each buffer: the storing warps of both CTAs
    uint64_t* fin_full = o_free + 3;             // each CTA's own softmax and storing warps
    uint64_t* fin_empty = fin_full + 1;
    uint64_t* drain = fin_empty + 1;             // each CTA's
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kMiscOff);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kMiscOff + 8);
    uint32_t* status = reinterpret_cast<uint32_t*>(smem + kMiscOff + 16);
    float* sm_max = reinterpret_cast<float*>(smem + kMaxOff);
    float2* sm_fin = reinterpret_cast<float2*>(smem + kFinOff);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const int pair = blockIdx.x >> 1;

    if (threadIdx.x == 0) {
        // a warp's arrival counts once: 8 softmax and 4 storing warps a CTA, both CTAs' on P full and O free
        for (int i = 0; i < kNumBars; ++i)
            mbar_init(&bars[i], &bars[i] >= p_full && &bars[i] < p_full + 2 ? 16
                                : &bars[i] >= o_free && &bars[i] < o_free + 3 ? 8
                                : &bars[i] == fin_full                        ? 2
                                : &bars[i] == fin_empty                       ? 4
                                                                              : 1);
        *abort_flag = 0;
        *status = 0;
        fence_barrier_init();
    }
    if (warp == 1) tmem_alloc_pair(tmem_slot, kTmemCols);
    tc_fence_before();
    __syncthreads();
    cluster_sync();                              // both CTAs' barriers exist
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    pdl_wait();
    // the plan: this pair's items (its scratch lies in buffers that the copies below fill)
    static_assert(sizeof(PlanScratch) <= 9 * kBlk, "the plan's scratch fits in K's buffer");
    int2* planned = reinterpret_cast<int2*>(smem + kMiscOff + 24);
    {
        const int2 r = plan_items<MODE>(a, pair, blockIdx.x == 0, *reinterpret_cast<PlanScratch*>(smem + kKOff),
                                         [&]() { ask_early<MODE>(a, lane); });
        if (threadIdx.x == 0) *planned = r;
    }
    fence_proxy_async_smem();
    __syncthreads();
    // Read back from one address, so that the compiler knows it to be the same in all threads: the MMA
    // issue is only fast in control flow that it can prove uniform (see mma_pair_bf16).
    const int2 range = *planned;
    const ChunkItem* items = reinterpret_cast<const ChunkItem*>(a.ws + a.items_off);
    const int R = min(a.P, kChunkRows);          // rows of one load: pages of 128 come in halves
    const int loads = kChunkRows / R;            // loads for 64 keys
    const int rlog = R == 64 ? 6 : (R == 32 ? 5 : 4);

    if (warp == 0 || warp == 3) {
        // -------------------------------------------------------- Q and K loads
        // One warp issues a copy in some 90 clocks.  Pages of 16 tokens take 36 of 2 KB for a tile's keys, more
        // than the tile's time, so for pages below 64 a second warp issues every other one.  That warp also loads the
        // first item's Q: one warp's copies come from HBM one after the other (24 KB in 1,000 clocks), and the first scores
        // wait for Q and K (tiny 11.2 to 10.5 us).  Later items' Q lies in L2, and asking for it before K is faster.
        const bool second = warp == 3;
        const uint32_t sq = smem_u32(smem + kQOff), sk = smem_u32(smem + kKOff);
        int ph = 0, qph = 0;
        bool ok = true, fresh = true;
        // q's box of this CTA: head and token, or the flat row
        auto q_at = [&](const ChunkItem& x) -> int2 {
            if (a.tile.flat) return make_int2(x.tok * a.H + x.row0 + int(rank) * kChunkRows, 0);
            const bool one = a.tile.groups == 1;
            return make_int2(a.head_lo + (one ? 0 : (2 * x.pair_group + int(rank)) * a.tile.heads),
                             x.tok + (one ? int(rank) * a.tile.tokens : 0));
        };
        ChunkItem it = {}, next = {};
        if (range.x < range.y) next = items[range.x];
        for (int i = range.x; ok && i < range.y; ++i) {
            it = next;
            if (i + 1 < range.y) next = items[i + 1];
            if (it.t_lo >= it.t_hi) continue;
            const int2 at = q_at(it);
#pragma unroll 1
            for (int g = 0; g < kKGroups && ok && second == fresh; ++g) {
                if (!__all_sync(0xffffffffu, mbar_wait(&q_empty[g], qph ^ 1, abort_flag, status))) { ok = false; break; }
                const uint32_t bar = map_to_rank(smem_u32(&q_full[g]), 0);
                if (rank == 0 && lane == 0)
                    mbar_arrive_expect_tx(&q_full[g], 2 * kKBlks * a.tile.box_rows() * 128);
                __syncwarp();
                const int b = g * kKBlks + lane;
                if (lane < kKBlks) tma_pair_4d(sq + b * kBlk, &maps.q, bar, 0, at.x, at.y, b);
            }
            if (!ok) break;
            fresh = false;
            qph ^= 1;
            // Q of the next item comes from HBM while this one is worked on: its buffer is free only
            // when the last scores are done, and the next item's first scores wait for it
            if (i + 1 < range.y && next.t_lo < next.t_hi && lane < 9 && !second) {
                const int2 to = q_at(next);
                tma_prefetch_4d(&maps.q, 0, to.x, to.y, lane);
            }
            if (second && R == kChunkRows) break;
            const int32_t* table = a.block_table + int64_t(it.r) * a.max_pages;
            const int start = item_start<MODE>(a, it);
            for (int t = it.t_lo; t < it.t_hi && ok; ++t) {
                // lane k < loads looks up the page behind keys [64 c + k R, + R) of the tile
                const int key = tile_key<MODE>(a, it, t, int(rank)) + lane * R;
                int row = a.past_row;            // past the pool: the copy fills zeros
                if (lane < loads && !left_behind<MODE>(a, start, key, R)) {
                    const int id = page_of(a, table, key, it.ctx);
                    if (id >= 0) row = (id << a.P_log) + (key & (a.P - 1));
                    else if (key + R > first_key<MODE>(a, it) && key < min(it.ctx, a.tok_hi) && !second)   // a page of the share
                        atomicOr(status, uint32_t(SPLASH_DEVICE_BAD_INPUT));
                }
#pragma unroll 1
                for (int g = 0; g < kKGroups; ++g) {
                    if (!__all_sync(0xffffffffu, mbar_wait(&k_empty[g], ph ^ 1, abort_flag, status))) {
                        ok = false;
                        break;
                    }
                    const uint32_t bar = map_to_rank(smem_u32(&k_full[g]), 0);
                    if (rank == 0 && lane == 0 && !second) mbar_arrive_expect_tx(&k_full[g], 2 * kKBlks * kBlk);
                    __syncwarp();
                    if (R == kChunkRows) {
                        if (lane == 0) tma_pair_3d(sk + g * kKBlks * kBlk, &maps.k, bar, 0, row, g * kKBlks);
                    } else {
                        static_assert(kKBlks * 4 <= 32, "a lane per copy");
                        {
                            const int b = lane >> (6 - rlog), p = lane & (loads - 1);
                            const int y = __shfl_sync(0xffffffffu, row, p);
                            if (b < kKBlks && (lane & 1) == int(second))
                                tma_pair_3d(sk + (g * kKBlks + b) * kBlk + p * R * 128, &maps.k, bar, 0, y, g * kKBlks + b);
                        }
                    }
                }
                // Keys that no other pair has brought into L2 come from HBM, in more than a tile's time: the
                // next tile's into L2, each page's rows as one run (35 requests of 3-9 tokens and 16 heads
                // over some 10,000 keys: 117 -> 106 us; further ahead is slower, and where pairs share
                // the keys it costs 2%).
                const int ahead = MODE != kChunkPlain ? tile_key<MODE>(a, it, t + 1, int(rank)) + lane * R : key + kChunkKeys;
                if ((it.flags & kItemAlone) && t + 1 < it.t_hi && lane < loads && !second && !left_behind<MODE>(a, start, ahead, R)) {
                    const int id = page_of(a, table, ahead, it.ctx);
                    if (id >= 0)
                        prefetch_l2(a.kv + ((int64_t(id) << a.P_log) + (ahead & (a.P - 1))) * (kDqk * 2),
                                    min(R, it.ctx - ahead) * (kDqk * 2));
                }
                ph ^= 1;
            }
        }
    } else if (warp == 2) {
        // -------------------------------------------------------- V loads
        // this CTA's 256 value dims (blocks 4 c .. 4 c + 3) of all 128 keys, in two halves.  Rows
        // past the context must be zero, whatever their slots hold (0 * NaN is NaN): whole absent pages
        // are loaded from past the pool, and the page in which the context ends is loaded in
        // runs of 4^i rows, the valid ones from the pool and the others from past it.
        const uint32_t sv = smem_u32(smem + kVOff);
        const int past = a.past_row;
        int ph = 0;
        bool ok = true;
        for (int i = range.x; ok && i < range.y; ++i) {
            const ChunkItem it = items[i];
            const int32_t* table = a.block_table + int64_t(it.r) * a.max_pages;
            const int start = item_start<MODE>(a, it);
            for (int t = it.t_lo; t < it.t_hi && ok; ++t) {
                int key = t * kChunkKeys + lane * R;            // lane k < 2 * loads: load k of the tile
                if (MODE != kChunkPlain) key = lane < loads ? tile_key<MODE>(a, it, t, 0) + lane * R : tile_key<MODE>(a, it, t, 1) + (lane - loads) * R;
                int row = past;
                if (lane < 2 * loads && !left_behind<MODE>(a, start, key, R)) {
                    const int id = page_of(a, table, key, it.ctx);
                    if (id >= 0) row = (id << a.P_log) + (key & (a.P - 1));
                }
#pragma unroll 1
                for (int hh = 0; hh < 2; ++hh) {
                    if (!__all_sync(0xffffffffu, mbar_wait(&v_empty[hh], ph ^ 1, abort_flag, status))) {
                        ok = false;
                        break;
                    }
                    const uint32_t bar = map_to_rank(smem_u32(&v_full[hh]), 0);
                    if (rank == 0 && lane == 0) mbar_arrive_expect_tx(&v_full[hh], 2 * kVHalf);
                    __syncwarp();
                    const int first = hh * loads;
                    const bool mine = lane >= first && lane < first + loads;
                    const bool cut = mine && row != past && key + R > it.ctx;
                    if (mine && !cut)
                        tma_pair_3d(sv + lane * R * 512, &maps.v, bar, 0, row, 4 * int(rank));
                    const uint32_t cuts = __ballot_sync(0xffffffffu, cut);
                    if (cuts) {                                  // one page at most
                        const int src = __ffs(cuts) - 1;
                        const int y = __shfl_sync(0xffffffffu, row, src);
                        const int n = it.ctx - __shfl_sync(0xffffffffu, key, src);   // valid rows, 0 < n < R
                        if (lane < 4) {
                            const uint32_t d0 = sv + src * R * 512 + lane * R * 128;
#pragma unroll 1
                            for (int o = 0, b = 2; o < R;) {        // runs of 16, 4 and 1 rows
                                const int end = o < n ? n : R;
#pragma unroll 1
                                while (o + (1 << 2 * b) > end) --b;
                                tma_pair_3d(d0 + o * 128, &maps.rows[b], bar, 0, o < n ? y + o : past, 4 * int(rank) + lane);
                                o += 1 << 2 * b;
                                if (o == n) b = 2;
                            }
                        }
                        __syncwarp();
                    }
                }
                ph ^= 1;
            }
        }
    } else if (warp == 1) {
        // -------------------------------------------------------- MMA issue (leader)
        // The whole warp walks the schedule in uniform control flow and one elected lane
        // issues (see mma_pair_bf16).
        if (rank == 0) {
            constexpr uint32_t idesc_qk = idesc_bf16_f32(128, kChunkKeys, false, false);
            constexpr uint32_t idesc_pv = idesc_bf16_f32(128, 256, false, true);
            const uint32_t on = elect_one();
            const uint64_t dq = smem_desc(smem_u32(smem + kQOff), 16, 1024, 2);
            const uint64_t dk = smem_desc(smem_u32(smem + kKOff), 16, 1024, 2);
            const uint64_t dp = smem_desc(smem_u32(smem + kPOff), 16, 1024, 2);
            const uint64_t dv = smem_desc(smem_u32(smem + kVOff), uint32_t(R) * 128, 1024, 2);
            uint32_t vo[4];                      // 16-key steps of a V half
            for (int s = 0; s < 4; ++s) vo[s] = uint32_t((s * 16 >> rlog) * (R * 512) + (s * 16 & (R - 1)) * 128) >> 4;
            const uint32_t vh = uint32_t(R) * 256 >> 4;              // two 64-dim blocks on
            int kph = 0, vph = 0, qph = 0;
            uint32_t ob = 0, used = 0;           // first buffer of the item's O; parity of the buffers' uses
            uint32_t g = 0;                      // tiles so far: S of tile g is in buffer g & 1
            bool ok = true;
            auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
                const bool w = __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, status));
                tc_fence_after();
                return w;
            };
            int2 next = range.x < range.y ? make_int2(items[range.x].t_lo, items[range.x].t_hi) : make_int2(0, 0);
            for (int i = range.x; ok && i < range.y; ++i) {
                const int nt = next.y - next.x;
                // S of tile t, then O of tile t - 1: the softmax of one tile has the other product's
                // time.  One copy of each product's code: a second one for an item's first tile, run
                // once an item, took 5,500 clocks to fetch and issue instead of 1,200.
                for (int t = 0; ok && t <= nt; ++t) {
                    if (t < nt) {
                        const uint32_t s_col = kSCol + (g & 1) * 64;
#pragma unroll 1
                        for (int j = 0; j < kKGroups; ++j) {
                            if (t == 0 && !wait(&q_full[j], qph)) { ok = false; break; }
                            if (!wait(&k_full[j], kph)) { ok = false; break; }
                            const uint32_t jo = uint32_t(j * kKBlks * kBlk) >> 4;
#pragma unroll
                            for (int b = 0; b < kKBlks; ++b)
#pragma unroll
                                for (int k4 = 0; k4 < 4; ++k4) {
                                    const uint32_t o = jo + (uint32_t(b * kBlk + k4 * 32) >> 4);
                                    mma_pair_bf16(tmem + s_col, dq + o, dk + o, idesc_qk, (j | b | k4) != 0 ? 1u : 0u, on);
                                }
                            commit_pair(&k_empty[j], on);
                            if (t + 1 == nt) commit_pair(&q_empty[j], on);
                        }
                        if (!ok) break;
                        kph ^= 1;
                        commit_pair(&s_full[g & 1], on);
                        ++g;
                    }
                    if (t == 0) {                // (loaded while the tensor cores have work)
                        if (i + 1 < range.y) next = make_int2(items[i + 1].t_lo, items[i + 1].t_hi);
                        continue;
                    }
                    if (t == 1) {
                        const uint32_t o2 = o_second(ob);
                        if (!wait(&o_free[ob], (used >> ob & 1) ^ 1)) { ok = false; break; }
                        if (!wait(&o_free[o2], (used >> o2 & 1) ^ 1)) { ok = false; break; }
                        used ^= 1u << ob | 1u << o2;
                    }
#pragma unroll 1
                    for (int hh = 0; hh < 2; ++hh) {
                        if (!wait(&v_full[hh], vph)) { ok = false; break; }
                        if (!wait(&p_full[hh], vph)) { ok = false; break; }
                        const uint32_t ho = uint32_t(hh * kVHalf) >> 4, po = uint32_t(hh * kBlk) >> 4;
#pragma unroll
                        for (int s4 = 0; s4 < 4; ++s4)
#pragma unroll
                            for (int h = 0; h < 2; ++h)
                                mma_pair_bf16(tmem + (h ? o_second(ob) : ob) * 128, dp + (po + uint32_t(s4 * 2)), dv + (ho + vo[s4] + h * vh),
                                              idesc_pv, ((t - 1) | hh | s4) != 0 ? 1u : 0u, on);
                        commit_pair(&v_empty[hh], on);
                    }
                    if (!ok) break;
                    vph ^= 1;
                    if (t == nt) commit_pair(o_full, on);
                }
                if (nt > 0) {
                    qph ^= 1;
                    ob = o_next(ob);
                }
            }
            commit_pair(drain, on);
        }
    } else if (warp >= 4 && warp < 12) {
        // -------------------------------------------------------- softmax
        // Two warps per TMEM lane quadrant, each with 32 of a lane's 64 score columns: a lane
        // is a row (tl & 63) and one half of the tile's keys, so four threads share a row.
        const int quad = warp & 3, part = (warp - 4) >> 2;
        const int tl = quad * 32 + lane;
        const int row = tl & 63, half = tl >> 6;
        const int share = half * 2 + part;       // keys [32 share, 32 share + 32) of the tile
        const uint32_t t_lane = tmem + (uint32_t(quad * 32) << 16);
        const uint32_t bp = map_to_rank(smem_u32(p_full), 0);
        // scores in the exp2 domain are c * x, c > 0: the maximum is taken over x, so a negative
        // scale moves its sign to x, and a zero one (0 * -inf is NaN) becomes part of x
        const bool odd_scale = a.scale <= 0.f;
        const float sign = a.scale < 0.f ? -1.f : 0.f;
        const float cl = a.scale == 0.f ? 1.f : fabsf(a.scale) * 1.4426950408889634f;
        uint8_t* prow = smem + kPOff + half * kBlk + row * 128;
        uint32_t g = 0, ob = 0;
        int fph = 0;
        bool ok = true;
        for (int i = range.x; ok && i < range.y; ++i) {
            const ChunkItem it = items[i];
            const ChunkRow at = chunk_row(a.tile, a.Hs, it.row0, it.ntok, it.pair_group, int(rank), row);
            // keys [lo, lim)
            const int lo = first_key<MODE>(a, it);
            const bool whole = MODE == kChunkGroups && (it.flags & kItemPrefix);
            const int lim = at.live ? min(whole ? it.ctx : it.seen + at.token, a.tok_hi) : 0;
            const int from = it.seen + at.token - a.window;                       // windowed: the row's first key behind the sinks
            const int32_t* table = a.block_table + int64_t(it.r) * a.max_pages;
            float m = -INFINITY, l = 0.f;        // maximum and sum (this thread's keys) of c * x
            for (int t = it.t_lo; t < it.t_hi; ++t, ++g) {
                const int key0 = MODE != kChunkPlain ? tile_key<MODE>(a, it, t, half) + part * 32 : t * kChunkKeys + share * 32;
                uint32_t gone = 0;               // bit k: this thread's keys k R .. have no page
#pragma unroll 1
                for (int k = 0; k * R < 32; ++k)
                    if (key0 + k * R < it.ctx && page_of(a, table, key0 + k * R, it.ctx) < 0) gone |= 1u << k;
                if (!__all_sync(0xffffffffu, mbar_wait(&s_full[g & 1], (g >> 1) & 1, abort_flag, status)))
                    ok = false;
                tc_fence_after();
                float x[32];
                tmem_ld32(t_lane + kSCol + (g & 1) * 64 + part * 32, x);
                tmem_wait_ld();
                if (odd_scale) {
#pragma unroll
                    for (int e = 0; e < 32; ++e) x[e] *= sign;
                }
                // the keys that this row does not see, a bit each: in code this short, because a tile that needs it may be
                // the only one of a launch, and its instructions come from memory then
                uint32_t hidden = low_bits(lo - key0) | ~low_bits(lim - key0);
                if (MODE == kChunkWindow) hidden |= low_bits(from - key0) & ~low_bits(a.sinks - key0);
                if (gone) hidden |= rlog == 4 ? (gone & 1 ? 0xffffu : 0u) | (gone & 2 ? 0xffff0000u : 0u) : 0xffffffffu;
                if (hidden) {
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (hidden >> e & 1) x[e] = -INFINITY;
                }
                float mx[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) mx[e] = x[e];
#pragma unroll
                for (int e = 4; e < 32; ++e) mx[e & 3] = fmaxf(mx[e & 3], x[e]);
                float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                float* ex = sm_max + (g & 1) * (4 * kChunkRows) + row;
                ex[share * kChunkRows] = top;
                if (named_barrier_or(1, kSoftThreads, !ok)) { ok = false; break; }
                top = fmaxf(fmaxf(ex[0], ex[kChunkRows]), fmaxf(ex[2 * kChunkRows], ex[3 * kChunkRows]));
                // the four threads of a row see the same maxima, so they take the same branch; a row
                // whose keys are all masked so far has top = -inf and stays at m = -inf
                top = top == -INFINITY ? top : top * cl;
                float alpha = 1.f;
                const bool up = top > m + kTau;
                if (up) {
                    alpha = m == -INFINITY ? 0.f : ex2(m - top);
                    m = top;
                    l *= alpha;
                }
                // O is at rest once the previous tile's MMAs are done
                if (t > it.t_lo && __any_sync(0xffffffffu, up)) {
                    if (!__all_sync(0xffffffffu, mbar_wait(&v_empty[1], (g - 1) & 1, abort_flag, status)))
                        ok = false;
                    tc_fence_after();
#pragma unroll 1
                    for (int c = 0; c < 128; c += 16) {
                        float o[16];
                        const uint32_t at_o = t_lane + (part ? o_second(ob) : ob) * 128 + c;
                        tmem_ld16(at_o, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 16; ++e) o[e] *= alpha;
                        tmem_st16(at_o, o);
                    }
                    tmem_wait_st();
                }
                const float base = m == -INFINITY ? 0.f : m;
                uint32_t pk[16];
                float ls[2] = {0.f, 0.f};
#pragma unroll
                for (int e = 0; e < 32; e += 2) {
                    const float p0 = ex2(fmaf(x[e], cl, -base)), p1 = ex2(fmaf(x[e + 1], cl, -base));
                    ls[0] += p0;                 // the sum takes P before its rounding to bf16
                    ls[1] += p1;
                    pk[e >> 1] = pack2(p0, p1);
                }
                l += ls[0] + ls[1];
                // Each half of the keys has its product, which needs its half of P and every warp's O at rest:
                // a half of P's buffer is free, and its barrier's phase over, when the previous tile's
                // product of that half is done.
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if (g > 0) {
                        if (!__all_sync(0xffffffffu, mbar_wait(&v_empty[h], (g - 1) & 1, abort_flag, status)))
                            ok = false;
                    }
                    if (half == h) {
#pragma unroll
                        for (int ch = 0; ch < 4; ++ch)
                            *reinterpret_cast<uint4*>(prow + (((part * 4 + ch) ^ (row & 7)) << 4)) =
                                make_uint4(pk[4 * ch], pk[4 * ch + 1], pk[4 * ch + 2], pk[4 * ch + 3]);
                        fence_proxy_async_smem();
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_pair(bp + h * 8);
                }
            }
            if (it.t_hi <= it.t_lo) continue;
            // the rows' sums over the four shares of the keys, and their maxima, to the storing warps
            float* sums = sm_max + (g & 1) * (4 * kChunkRows) + row;   // not the last tile's buffer
            sums[share * kChunkRows] = l;
            // (a wait can give up in one warp alone: all of them leave here, or none)
            if (named_barrier_or(1, kSoftThreads, !ok)) break;
            if (share == 0) {                    // the part 0 warps of lanes 0-63: two whole warps
                if (!__all_sync(0xffffffffu, mbar_wait(fin_empty, fph ^ 1, abort_flag, status))) ok = false;
                l = (sums[0] + sums[kChunkRows]) + (sums[2 * kChunkRows] + sums[3 * kChunkRows]);
                sm_fin[row] = make_float2(m, l);
                __syncwarp();
                if (lane == 0) mbar_arrive(fin_full);
            }
            fph ^= 1;
            ob = o_next(ob);
            // the sums are read before the next tile's maxima take their place
            if (named_barrier_or(1, kSoftThreads, !ok)) break;
        }
    } else if (warp >= 12) {
        // -------------------------------------------------------- results
        const int tl = (warp & 3) * 32 + lane;   // TMEM lane: row tl & 63, value dims [256 (tl >> 6), + 256)
        const int row = tl & 63, half = tl >> 6;
        const uint32_t t_o = tmem + (uint32_t((warp & 3) * 32) << 16);
        const uint32_t bo = map_to_rank(smem_u32(o_free), 0);
        float* plse = reinterpret_cast<float*>(a.ws + a.plse_off);
        float* pout = reinterpret_cast<float*>(a.ws + a.pout_off);
        int ph = 0;
        uint32_t ob = 0;
        for (int i = range.x; i < range.y; ++i) {
            const ChunkItem it = items[i];
            const ChunkRow at = chunk_row(a.tile, a.Hs, it.row0, it.ntok, it.pair_group, int(rank), row);
            const bool live = at.live;
            const bool worked = it.t_hi > it.t_lo;   // no key tile: zeros
            float m = 0.f, l = 0.f;
            if (worked) {
                // a wait for all of the item (a role that gives up sooner raises the abort flag, which ends it)
                const uint64_t limit = kWaitLimitNs + uint64_t(it.t_hi - it.t_lo) * kTileLimitNs;
                if (!__all_sync(0xffffffffu, mbar_wait(fin_full, ph, abort_flag, status, limit))) break;
                const float2 f = sm_fin[row];
                m = f.x;
                l = f.y;
                __syncwarp();
                if (lane == 0) mbar_arrive(fin_empty);
                if (!__all_sync(0xffffffffu, mbar_wait(o_full, ph, abort_flag, status))) break;
                ph ^= 1;
                tc_fence_after();
            }
            const bool none = l == 0.f;
            const float inv = none ? 0.f : 1.f / l;
            const bool whole = it.slot < 0;
            const int64_t to = whole ? int64_t(it.tok + at.token) * a.H + a.head_lo + at.head
                                     : int64_t(it.slot) * (2 * kChunkRows) + int(rank) * kChunkRows + row;
            if (live && half == 0)
                *((whole ? a.lse : plse) + to) = none ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
            // 16 rows x 64 columns a round, four threads to a row, which trade their columns so that each
            // stores 32 bytes of a 128-byte line.  (A thread storing its own row, a line per 32
            // bytes, held O for 5,000 clocks.)
            const bool f32 = a.out_f32 || !whole;
            const int mine = live ? int(to) : -1;
            char* base = reinterpret_cast<char*>(whole ? a.out : static_cast<void*>(pout));
            const bool no_rows = __any_sync(0xffffffffu, none);
            const uint32_t alive = __ballot_sync(0xffffffffu, live);
            auto release = [&](uint32_t buf) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_pair(bo + buf * 8);
            };
#pragma unroll 1
            for (int k = 0; k < 4; ++k) {            // 128 columns of rows [16 rr, + 16) of the warp's 32
                const int oh = k >> 1, rr = k & 1;
                const uint32_t buf = oh ? o_second(ob) : ob;
                if ((alive >> (16 * rr) & 0xffff) == 0) {
                    if (worked && rr == 1) release(buf);
                    continue;
                }
                const int from = rr * 16 + (lane >> 2);
                const int to0 = __shfl_sync(0xffffffffu, mine, from), to1 = __shfl_sync(0xffffffffu, mine, from + 8);
                const float inv0 = __shfl_sync(0xffffffffu, inv, from), inv1 = __shfl_sync(0xffffffffu, inv, from + 8);
#pragma unroll 1
                for (int c = 0; c < 128; c += 64) {
                    float o[32];
                    if (worked) {
                        __syncwarp();            // (a row that is not stored leaves its threads ahead of the others)
                        tmem_ld_rows16(t_o + (uint32_t(rr * 16) << 16) + buf * 128 + c, o);
                        tmem_wait_ld();
                        if (rr == 1 && c == 64) release(buf);
                    }
                    if (no_rows) {                   // zeros, whatever O holds
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = (e & 2 ? inv1 : inv0) == 0.f ? 0.f : o[e];
                    }
                    const int col = half * 256 + oh * 128 + c;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {    // rows lane / 4 + 8 h
                        const int dst = h ? to1 : to0;
                        const float s = h ? inv1 : inv0;
                        float x[16];                 // 2 columns of each run of 8
#pragma unroll
                        for (int e = 0; e < 16; ++e) x[e] = o[4 * (e >> 1) + 2 * h + (e & 1)] * s;
                        if (f32) {
#pragma unroll
                            for (int g = 0; g < 2; ++g) {        // 32 columns each
                                uint32_t w[4][2];
#pragma unroll
                                for (int e = 0; e < 8; ++e) w[e >> 1][e & 1] = __float_as_uint(x[8 * g + e]);
                                quad_trade(w, lane);
                                if (dst >= 0) store32(base + (int64_t(dst) * kDv + col + g * 32 + 8 * (lane & 3)) * 4, &w[0][0]);
                            }
                        } else {
                            uint32_t w[4][2], v[8];
#pragma unroll
                            for (int e = 0; e < 8; ++e) w[e >> 1][e & 1] = pack2(x[2 * e], x[2 * e + 1]);
                            quad_trade(w, lane);
#pragma unroll
                            for (int e = 0; e < 8; ++e) v[e] = w[e & 3][e >> 2];
                            if (dst >= 0) store32(base + (int64_t(dst) * kDv + col + 16 * (lane & 3)) * 2, v);
                        }
                    }
                }
            }
            if (worked) ob = o_next(ob);
        }
        if (warp == 12) {
            // Every MMA has completed before TMEM and shared memory go (bounded like every wait).  Here the wait begins
            // when the work is done: begun by the second CTA's idle warp 1, it ran into its limit in calls of
            // more than 2 s.
            volatile int never = 0;
            mbar_wait(drain, 0, &never, status);
            __syncwarp();
        }
    }

    // the merge may launch: at the start its waiting blocks would hold SMs that another stream needs
    pdl_trigger();
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0) {
        reinterpret_cast<uint32_t*>(a.ws + a.words_off)[blockIdx.x] = *status;
        if (*abort_flag)                         // copies that nobody waited for land before the CTA goes
            for (const uint64_t t0 = globaltimer_ns(); globaltimer_ns() - t0 < 1000000ull;) {}
    }
    cluster_sync();                              // no CTA leaves while the other may still reach its memory
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, kTmemCols);
    }
}

}  // namespace

namespace {

template <int MODE>
cudaError_t launch_mode(const ChunkArgs& a, const ChunkMaps& maps, cudaStream_t stream) {
    const cudaError_t e = ensure_smem_optin(reinterpret_cast<const void*>(chunk_attn_kernel<MODE>), kSmem);
    if (e != cudaSuccess) return e;
    return launch_pdl(chunk_attn_kernel<MODE>, dim3(2 * a.pairs), dim3(kThreads), size_t(kSmem), stream, maps, a);
}

}  // namespace

cudaError_t launch_chunk_attn(const ChunkArgs& a, const ChunkMaps& maps, cudaStream_t stream) {
    switch (a.mode) {
        case kChunkWindow: return launch_mode<kChunkWindow>(a, maps, stream);
        case kChunkGroups: return launch_mode<kChunkGroups>(a, maps, stream);
        default: return launch_mode<kChunkPlain>(a, maps, stream);
    }
}

}  // namespace splash
