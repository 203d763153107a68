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
constexpr int kChunkSlotsPerPair = 8;  // partial results the workspace holds, per CTA pair

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
    __host__ __device__ int pair_groups() const { return groups == 1 ? 1 : groups / 2; }
    // new tokens that a pair's rows span, at most
    __host__ __device__ int pair_tokens() const {
        return flat ? (2 * kChunkRows + heads - 1) / heads : (groups == 1 ? 2 * tokens : tokens);
    }
    // row tiles of n new tokens
    __host__ __device__ int64_t row_tiles(int64_t n) const {
        if (flat) return (n * heads + 2 * kChunkRows - 1) / (2 * kChunkRows);
        return (n + pair_tokens() - 1) / pair_tokens() * pair_groups();
    }
    __host__ __device__ int box_rows() const { return flat ? kChunkRows : heads * tokens; }
};

inline ChunkTiling chunk_tiling(int H, int Hs) {
    ChunkTiling t;
    t.flat = H == Hs;
    t.groups = t.flat || Hs <= kChunkRows ? 1 : 2 * ((Hs + 2 * kChunkRows - 1) / (2 * kChunkRows));
    t.heads = (Hs + t.groups - 1) / t.groups;
    t.tokens = t.flat ? 0 : kChunkRows / t.heads;
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
        r.token = x / Hs;
        r.head = x - r.token * Hs;
        r.live = r.token < ntok;
    } else {
        const int in = row / t.heads;
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
};

// One pair's work: the rows of one token block and head group pair against key tiles
// [t_lo, t_hi).
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
    int32_t alone;        // few row tiles share these keys: they are prefetched into L2
    int32_t pad;
};
static_assert(sizeof(ChunkItem) == 48, "ChunkItem layout");

struct alignas(16) ChunkSplit {
    int32_t tok, ntok, row0, pair_group, slot, pieces, pad[2];
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
    int pairs;            // CTA pairs of the grid
    ChunkTiling tile;
    int out_f32;
    float scale;
};

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
