"""The chunk attention's bounds on a row tile's tokens and key tiles (csrc/chunk.h), against every row tile's own
(CPU only)."""
import os
import subprocess
import tempfile

from layout_agnostic_paged_gb300 import build as B

SOURCE = r"""
#include <stdio.h>
#include <algorithm>
using std::max;
using std::min;
#include "chunk.h"
using namespace splash;

// First and last token of each row tile of n new tokens, from the rows themselves.
struct Tile { int first, last; };
static int tiles_of(const ChunkTiling& t, int Hs, int n, Tile* out) {
    const int count = t.row_tiles(n);
    for (int i = 0; i < count; ++i) {
        const int block = t.flat ? 0 : i / t.pair_groups() * t.per;
        Tile x = {n, -1};
        for (int cta = 0; cta < 2; ++cta)
            for (int row = 0; row < kChunkRows; ++row) {
                const ChunkRow at = chunk_row(t, Hs, t.flat ? i * 2 * kChunkRows : 0, n - block, t.flat ? 0 : i % t.pair_groups(), cta, row);
                if (!at.live) continue;
                x.first = min(x.first, block + at.token);
                x.last = max(x.last, block + at.token);
            }
        out[i] = x;
    }
    return count;
}

int main() {
    static Tile tiles[1 << 16];
    const int windows[] = {1, 2, 40, 55, 59, 62, 63, 64, 65, 127, 128, 129, 512, 1024}, sinks[] = {0, 4, 64, 70};
    // all heads of every count, and slices of 256 and of 128 heads
    for (int x = 1; x <= 256 + 255 + 127; ++x) {
        const int H = x <= 256 ? x : (x <= 511 ? 256 : 128), Hs = x <= 256 ? x : (x <= 511 ? x - 256 : x - 511);
        const ChunkTiling t = chunk_tiling(H, Hs);
        const int n = 300, count = tiles_of(t, Hs, n, tiles);
        int span = 0;
        for (int i = 0; i < count; ++i) span = max(span, tiles[i].last - tiles[i].first + 1);
        if (span != t.span) return printf("%d of %d heads: row tiles of %d tokens, not %d\n", Hs, H, span, t.span), 1;
        for (int w : windows)
            for (int s : sinks)
                for (int tok_lo : {0, 40, 200}) {
                    ChunkArgs a = {};
                    a.tile = t;
                    a.tok_lo = tok_lo;
                    a.tok_hi = 2147483647;
                    a.window = w;
                    a.sinks = s;
                    a.sink_blocks = max(0, (s + kChunkRows - 1) / kChunkRows - tok_lo / kChunkRows);
                    const int most = most_window_tiles(a);
                    for (int past = 0; past < 64; past += w == 63 || w == 64 || w == 128 ? 1 : 7)
                        for (int i = 0; i < count; ++i) {
                            const int k = key_tiles<kChunkWindow>(a, tok_lo, past + tiles[i].first + 1, past + tiles[i].last + 1);
                            if (k > most)
                                return printf("%d of %d heads, window %d, %d first tokens, from %d, past %d: row tile %d has %d key "
                                              "tiles, not %d\n", Hs, H, w, s, tok_lo, past, i, k, most), 1;
                        }
                }
    }
    return 0;
}
"""


def test_row_tiles_stay_in_their_bounds():
    cuda = os.path.join(os.path.dirname(os.path.dirname(B.nvcc())), "include")
    with tempfile.TemporaryDirectory() as d:
        src, exe = os.path.join(d, "t.cpp"), os.path.join(d, "t")
        with open(src, "w") as f:
            f.write(SOURCE)
        subprocess.run(["g++", "-std=c++17", "-O2", "-I", cuda, "-I", B.INCLUDE, "-I", B.CSRC, src, "-o", exe], check=True)
        r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout
