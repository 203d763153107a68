// rope.cuh -- rotary positions: frequencies as exact fractions of a turn, and the
// rotation of one pair.
//
// The angle of pair i at position p is p * f_i radians.  In fp32 that product loses all
// of its fraction for far positions, and fp64 is slow on this GPU.  So the host turns f_i
// into turns per position in 64-bit fixed point, F_i = round(f_i / (2 pi) * 2^64): the
// low 64 bits of the integer product p * F_i are then the fraction of a turn, whole turns
// dropped by the wrap itself, with an error of |p| / 2 units of 2^-64 turns (F_i is rounded once,
// see rope_table.h): 2^-34 turns at the farthest position, far below fp32's share.  One integer multiply
// per pair, the same accuracy at every position.
#pragma once

#include <stdint.h>

#include "splash.h"

namespace splash {

constexpr int kMaxRopePairs = 128;

// Passed to the kernels by value.
struct RopeTable {
    uint64_t turns[kMaxRopePairs];  // F_i
    float amplitude;
};

struct RopeTable32 {                // the 64-dim table of the cache's keys
    uint64_t turns[32];
    float amplitude;
};

// The table by its generic address: as kernel parameters its entries come through the constant
// cache, one address at a time, and a warp reads 32 (an append of 36,600 rows took 15.5 us that way and
// takes 12.4).
__device__ __forceinline__ const uint64_t* generic_table(const uint64_t* turns) {
    asm("" : "+l"(turns));
    return turns;
}

// cos and sin (times the amplitude) at position p of a pair with F turns.  The quadrant
// is split off in integers, so the float angle is at most 1/4 half turn and its rounding at most
// 2^-26 half turns.
__device__ __forceinline__ float2 rope_cos_sin(uint64_t F, int32_t p, float amplitude) {
    const int64_t x = static_cast<int64_t>(F * static_cast<uint64_t>(static_cast<int64_t>(p)));
    const int64_t quarter = static_cast<int64_t>(static_cast<uint64_t>(x) + (1ull << 61)) >> 62;
    const int64_t rest = static_cast<int64_t>(static_cast<uint64_t>(x) - (static_cast<uint64_t>(quarter) << 62));
    float s, c;
    sincospif(static_cast<float>(rest) * 1.0842021724855044e-19f, &s, &c);   // 2^-63: half turns
    const int q = static_cast<int>(quarter) & 3;
    if (q & 1) {
        const float t = c;
        c = -s;
        s = t;
    }
    if (q & 2) {
        c = -c;
        s = -s;
    }
    return make_float2(c * amplitude, s * amplitude);
}

__device__ __forceinline__ float2 rope_rotate(float a, float b, float2 cs) {
    return make_float2(a * cs.x - b * cs.y, a * cs.y + b * cs.x);
}

}  // namespace splash
