// chunk.h -- what the chunk attention's host code, plan, kernel and combine share.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace splash {

constexpr int kChunkRows = 64;         // query rows of one CTA; a pair works on 128
constexpr int kChunkKeys = 128;        // keys of one tile
constexpr int kChunkKBlocks = 3;       // 64-dim blocks of the keys loaded and released together
constexpr int kChunkMaxGroups = 1024;
constexpr int kEarlyUnits = 2;         // units of 64 keys that a CTA asks for before the plan
constexpr int kChunkSlotsPerPair = 8;  // partial results the workspace holds, per CTA pair

// What a call's kernels are compiled for.  Each form has its own code, so that the plain one pays for nothing else.
enum ChunkMode {
    kChunkPlain,     // every key before a token, in one range
    kChunkWindow,    // the keys of a sliding window and some first ones
    kChunkGroups     // groups of requests share a prefix, which is worked on for all rows of a group at once
};

// n / d for 0 <= n < 2^31 and a d that the host knows: a product and a shift.  (The plan is a chain of such steps, and a
// division takes some 100 clocks, one of 64 bits some 500.)  With s = 31 + ceil(log2 d) and m = ceil(2^s / d) the
// product is off by less than n d / 2^s < 1 / d.
struct FastDiv {
    uint32_t m;
    int32_t s;
    __host__ __device__ int operator()(int n) const { return int(uint64_t(uint32_t(n)) * m >> s); }
};
inline FastDiv fast_div(int d) {
    int k = 0;
    while ((int64_t(1) << k) < d) ++k;
    return FastDiv{uint32_t(((uint64_t(1) << (31 + k)) + uint64_t(d) - 1) / uint64_t(d)), 31 + k};
}

// How query rows are laid over the rows of CTA pairs.
// flat: the call has all heads, so a request's (token, head) rows are consecutive rows of q and a pair
//   takes 128 of them, wherever tokens begin (head counts that do not divide 64 waste nothing).
// else (a head slice): a CTA's rows are `tokens` consecutive new tokens times `heads` consecutive heads
//   (head fastest), at most 64.  With one head group the pair's CTAs take consecutive token blocks,
//   with several (then an even number) they take consecutive head groups of the same tokens.
struct ChunkTiling {
    int flat;
    int groups;   // head groups of a token block: 1 or an even number (flat: 1)
    int heads;    // heads of a group (the last may have fewer); flat: all heads
    int tokens;   // tokens of a CTA's block (flat: unused)
    int per;      // new tokens whose rows fill a pair's, if the first one's begin with them
    int span;     // new tokens that a row tile's rows belong to, at most.  Flat: row tiles begin wherever 128 i falls, so 128 rows
                  //   of 80 heads are of two tokens or of three
    FastDiv by_heads, by_per;
    __host__ __device__ int pair_groups() const { return groups == 1 ? 1 : groups / 2; }
    __host__ __device__ int pair_tokens() const { return per; }
    // row tiles of n new tokens (n times the call's heads is below 2^31)
    __host__ __device__ int row_tiles(int n) const {
        if (flat) return int((uint32_t(n) * uint32_t(heads) + (2 * kChunkRows - 1)) / (2 * kChunkRows));
        return by_per(n + per - 1) * pair_groups();
    }
    __host__ __device__ int box_rows() const { return flat ? kChunkRows : heads * tokens; }
};

inline ChunkTiling chunk_tiling(int H, int Hs) {
    ChunkTiling t;
    t.flat = H == Hs;
    t.groups = t.flat || Hs <= kChunkRows ? 1 : 2 * ((Hs + 2 * kChunkRows - 1) / (2 * kChunkRows));
    t.heads = (Hs + t.groups - 1) / t.groups;
    t.tokens = t.flat ? 0 : kChunkRows / t.heads;
    t.per = t.flat ? (2 * kChunkRows + t.heads - 1) / t.heads : (t.groups == 1 ? 2 * t.tokens : t.tokens);
    // (rows 128 i begin at multiples of gcd(heads, 128) within a token: the last of these leaves the fewest rows to the first token)
    int gcd = 2 * kChunkRows;
    while (t.heads % gcd != 0) gcd /= 2;
    t.span = t.flat ? (t.heads - gcd + 2 * kChunkRows - 1) / t.heads + 1 : t.per;
    t.by_heads = fast_div(t.heads);
    t.by_per = fast_div(t.per);
    return t;
}

// The token (counted from the item's first) and head (of the slice) of a row of CTA `cta` of a pair.
struct ChunkRow {
    int token, head;
    bool live;    // a row of the call, not padding
};
__host__ __device__ inline ChunkRow chunk_row(const ChunkTiling& t, int Hs, int row0, int ntok, int pair_group,
                                              int cta, int row) {
    ChunkRow r;
    if (t.flat) {
        const int x = row0 + cta * kChunkRows + row;
        r.token = t.by_heads(x);
        r.head = x - r.token * Hs;
        r.live = r.token < ntok;
    } else {
        const int in = t.by_heads(row);
        r.token = in + (t.groups == 1 ? cta * t.tokens : 0);
        r.head = row - in * t.heads + (t.groups == 1 ? 0 : (2 * pair_group + cta) * t.heads);
        r.live = in < t.tokens && r.token < ntok && r.head < Hs;
    }
    return r;
}

// Workspace: header, a status word per CTA, work items, split row tiles, partial lse,
// partial out (256-byte aligned each).
constexpr uint32_t kChunkMagic = 0x4b4e4843u;   // tells the header from a decode plan's (whose second word is a small count)
constexpr size_t kChunkWordsOff = 256;
struct ChunkHeader {
    uint32_t status;      // SPLASH_DEVICE_* bits that the plan set; the CTAs' words hold the others
    uint32_t magic;
    int32_t num_splits;   // row tiles cut into several items
    int32_t words;        // status words
    int32_t split_rows;   // grouped: rows of a request's row tile, at most
};

// One pair's work: the rows of one token block and head group pair against key tiles
// [t_lo, t_hi).  A tile is two blocks of 64 keys.  In the windowed form the first tokens' blocks and the window's
// are counted as one sequence, with `base` between a block's number in it and its place in the context.
// In the grouped form an item's keys begin at `base`, its tiles are counted from that key's block, and a group's own item is
// one of all its requests' rows.
constexpr int kItemAlone = 1;    // few row tiles share these keys: they are prefetched into L2
constexpr int kItemPrefix = 2;   // every row sees every key up to ctx: a group's rows over its prefix
struct alignas(16) ChunkItem {
    int32_t r;            // request
    int32_t tok;          // first new token (flat: of the request)
    int32_t ntok;         // tokens of the request from there on
    int32_t row0;         // flat: the tile's first row, counted from token `tok`
    int32_t seen;         // keys that token `tok` sees: its position + 1
    int32_t pair_group;   // head groups 2 * pair_group and the next one (one group: 0)
    int32_t t_lo, t_hi;   // key tiles
    int32_t slot;         // partial slot, or -1: the result goes to out
    int32_t ctx;          // context length (keys at or past it do not exist)
    int32_t flags;
    int32_t base;         // windowed, grouped: see above
};
static_assert(sizeof(ChunkItem) == 48, "ChunkItem layout");

// A row tile whose results lie in partial slots.  pre: 0; -1 for a group's row tile, which is merged into its
// requests' ones; n + 1 for the row tile of a request whose group's row tiles begin at split n, with rows counted
// from row c0 of q.
struct alignas(16) ChunkSplit {
    int32_t tok, ntok, row0, pair_group, slot, pieces, pre, c0;
};
static_assert(sizeof(ChunkSplit) == 32, "ChunkSplit layout");

struct ChunkArgs {
    const uint8_t* kv;    // the pool
    const int32_t* cu_q;
    const int32_t* block_table;
    const int32_t* ctx_lens;
    void* out;
    float* lse;
    uint8_t* ws;
    size_t words_off, items_off, splits_off, plse_off, pout_off;
    int64_t cap_items;
    int cap_slots;
    int B, total_q, H, head_lo, Hs;
    int P, P_log, num_pages, max_pages, max_ctx;   // P = 2^P_log
    int past_row;         // a row of the pool's maps that does not exist: copies from there fill zeros
    int tok_lo, tok_hi;   // tok_hi: INT32_MAX for "to the end"
    int mode;             // ChunkMode
    int window, sinks;    // windowed: a token sees the last `window` keys up to its own, and the first `sinks`
    int sink_blocks;      // blocks of first tokens from tok_lo's block on
    const int32_t* cu_groups;     // grouped: [groups + 1], requests of group g from cu_groups[g] on
    const int32_t* prefix_lens;   // [groups]
    int groups;
    int early;            // units of 64 keys that are asked for before the plan, per request
    FastDiv by_early;
    int pairs;            // CTA pairs of the grid
    FastDiv by_pairs;
    ChunkTiling tile;
    int out_f32;
    float scale;
};

// (for host programs too, which have no min and max without a namespace)
__host__ __device__ inline int lesser(int x, int y) { return x < y ? x : y; }
__host__ __device__ inline int greater(int x, int y) { return x < y ? y : x; }

// Key tiles of a row tile whose tokens see the keys from `lo` on before `first` .. `last` (positions + 1).  Windowed: the
// blocks of the first tokens, then those from the first token's window on; *base is the item's.
template <int MODE>
__host__ __device__ inline int key_tiles(const ChunkArgs& a, int lo, int first, int last, int* base = nullptr) {
    const int e = lesser(last, a.tok_hi);
    if (MODE == kChunkGroups && base) *base = lo;
    if (e <= lo) return 0;
    if constexpr (MODE == kChunkWindow) {
        const int b0 = lo / kChunkRows, end = (e + kChunkRows - 1) / kChunkRows;
        const int w = greater(b0 + a.sink_blocks, greater(greater(first, 1) - a.window, 0) / kChunkRows);
        if (base) *base = w - a.sink_blocks;
        return (lesser(end - b0, a.sink_blocks) + greater(end - w, 0) + 1) / 2;
    }
    // (grouped: from the block in which the prefix ends, not from the tile)
    if constexpr (MODE == kChunkGroups) return (e - lo / kChunkRows * kChunkRows + kChunkKeys - 1) / kChunkKeys;
    return (e + kChunkKeys - 1) / kChunkKeys - lo / kChunkKeys;
}

// Windowed: the key tiles of any row tile, at most.  Its tokens' windows span window + tokens - 1 keys, wherever those begin.
__host__ __device__ inline int most_window_tiles(const ChunkArgs& a) {
    return (a.sink_blocks + (a.window + a.tile.span - 1 + 2 * (kChunkRows - 1)) / kChunkRows + 1) / 2;
}

struct ChunkMaps {
    CUtensorMap q;        // [9][total_q][H][64] box {64, heads, tokens, 1}; flat: [9][1][total_q * H][64] box {64, 64, 1, 1}
    CUtensorMap k;        // pool as [9][rows][64]: box {64, 64, 3}, or {64, P, 1} for pages below 64
    CUtensorMap v;        // box {64, min(P, 64), 4}
    CUtensorMap rows[3];  // box {64, 4^i, 1}
};

// Capacities for the shape (cap_items, cap_slots), and the offsets; returns the bytes.
size_t chunk_layout(ChunkArgs& a);
cudaError_t launch_chunk_attn(const ChunkArgs& a, const ChunkMaps& maps, cudaStream_t stream);
cudaError_t launch_chunk_combine(const ChunkArgs& a, int sms, cudaStream_t stream);

}  // namespace splash
