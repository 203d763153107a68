// norm_rope.cu -- splash_norm_rope: RMS norm of query and key head rows and the rotation of a part of
// each row, in one pass.
//
//   y_j = x_j * rsqrt(mean(x_0^2 .. x_{n-1}^2) + eps) * (w_j + offset)  for j < n, x_j behind them,
//   then pairs of dims [lo, lo + d) are rotated by the token's position.
//
// Every element is read and written once, where a norm and a rotation one after the other move it twice.  G lanes
// hold a row in registers: each has "units" of two vectors, and the two vectors of a rotated unit are the halves of its
// pairs (d / 2 apart), so that no element crosses lanes and only the sum of squares does.  A block owns a run of one
// side's rows, several to a lane one after the other, the next one's loads under way while one is worked on: a lane's place
// in the row, the weights and the tokens' cos / sin are worked out once for all of them.
//
// What bounds it is the issue of instructions, not HBM: 73% of all issue slots in the large case.  With a block per
// token it took 25 instructions an element; now 18, the products and sums two to an instruction.  8,191 tokens x 72
// heads x 128 dims in bf16, half of them rotated (302 MB): 50.2 us, 6.0 TB/s, 90% of the copy bandwidth (47.3 us in fp32 with half
// the tokens); 1,024 tokens x 129 latent heads x 576 dims 54.6 us (82%); 32,768 latent rows of 576 dims, whose 32 angles
// serve one row each: 19.0 us (60%: a block works out the angles of all its rows before it starts on the first); 256 tokens x 18 heads: 3.2 us.
#include <limits.h>

#include <algorithm>
#include <atomic>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"
#include "kernels.h"
#include "rope.cuh"

namespace splash {
namespace {

constexpr int kNormThreads = 128;    // a block's, at most
constexpr int kNormPasses = 8;       // rows of a lane one after the other, at most
constexpr int kNormUnits = 4;        // units of a lane, at most
// Blocks an SM has room for: one more than the compiler's choice of registers leaves (a unit a lane: 52.5 to 50.6 us for
// the large prompt; three: 24.1 to 21.7 for 2,000 tokens x 17 heads x 576 dims at that time; one more still takes
// 22 us there where this takes 17.8).
template <int K>
constexpr int kNormBlocks = K == 1 ? 8 : (K == 3 ? 4 : 1);
constexpr int kNormPairs = 2048;     // cos / sin a block holds, at most (one token has 128 at most)

__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ void from_f32(__nv_bfloat16& d, float v) { d = __float2bfloat16_rn(v); }
__device__ __forceinline__ void from_f32(__half& d, float v) { d = __float2half_rn(v); }
__device__ __forceinline__ void from_f32(float& d, float v) { d = v; }
// Two at a time, where there are two.
__device__ __forceinline__ void from_f32x2(__nv_bfloat16* d, float a, float b) {
    *reinterpret_cast<__nv_bfloat162*>(d) = __floats2bfloat162_rn(a, b);
}
__device__ __forceinline__ void from_f32x2(__half* d, float a, float b) { *reinterpret_cast<__half2*>(d) = __floats2half2_rn(a, b); }
__device__ __forceinline__ void from_f32x2(float* d, float a, float b) {
    d[0] = a;
    d[1] = b;
}

// Two fp32 products, multiply-adds or differences in one instruction.
__device__ __forceinline__ void mul2(float* d, const float* a, float b0, float b1) {
    asm("{\n\t.reg .b64 p, q;\n\tmov.b64 p, {%2, %3};\n\tmov.b64 q, {%4, %5};\n\tmul.rn.f32x2 p, p, q;\n\tmov.b64 {%0, %1}, p;\n\t}"
        : "=f"(d[0]), "=f"(d[1])
        : "f"(a[0]), "f"(a[1]), "f"(b0), "f"(b1));
}
__device__ __forceinline__ void fma2(float* d, const float* a, const float* b, const float* c) {
    asm("{\n\t.reg .b64 p, q, r;\n\tmov.b64 p, {%2, %3};\n\tmov.b64 q, {%4, %5};\n\tmov.b64 r, {%6, %7};\n\t"
        "fma.rn.f32x2 p, p, q, r;\n\tmov.b64 {%0, %1}, p;\n\t}"
        : "=f"(d[0]), "=f"(d[1])
        : "f"(a[0]), "f"(a[1]), "f"(b[0]), "f"(b[1]), "f"(c[0]), "f"(c[1]));
}
__device__ __forceinline__ void sub2(float* d, const float* a, const float* b) {
    asm("{\n\t.reg .b64 p, q;\n\tmov.b64 p, {%2, %3};\n\tmov.b64 q, {%4, %5};\n\tsub.rn.f32x2 p, p, q;\n\tmov.b64 {%0, %1}, p;\n\t}"
        : "=f"(d[0]), "=f"(d[1])
        : "f"(a[0]), "f"(a[1]), "f"(b[0]), "f"(b[1]));
}

// 16 bytes, or one element.
template <typename T, int VE>
__device__ __forceinline__ void load_vec(T* v, const T* p) {
    if constexpr (VE > 1) *reinterpret_cast<uint4*>(v) = __ldcs(reinterpret_cast<const uint4*>(p));
    else *v = *p;
}
template <typename T, int VE>
__device__ __forceinline__ void store_vec(T* p, const T* v) {
    if constexpr (VE > 1) __stcs(reinterpret_cast<uint4*>(p), *reinterpret_cast<const uint4*>(v));
    else *p = *v;
}

__device__ __forceinline__ float weight_at(const void* w, int dtype, int i) {
    if (dtype == SPLASH_F32) return static_cast<const float*>(w)[i];
    if (dtype == SPLASH_F16) return __half2float(static_cast<const __half*>(w)[i]);
    return __bfloat162float(static_cast<const __nv_bfloat16*>(w)[i]);
}

// A power of two for rows whose squares leave fp32's range, else 1.  Sums above 2^120 are taken from x 2^-100,
// sums below 2^-110 from x 2^100, unless eps is large enough (2^-80) for such a sum not to show beside it.
__device__ __forceinline__ float range_scale(float ss, float eps) {
    const float up = __uint_as_float((127u + 100u) << 23), down = __uint_as_float((127u - 100u) << 23);
    if (!(ss <= __uint_as_float((127u + 120u) << 23))) return down;
    return ss < __uint_as_float((127u - 110u) << 23) && eps < __uint_as_float((127u - 80u) << 23) ? up : 1.f;
}

// VE elements a vector, K units a lane.  SINGLE: the last of them has one vector, which leaves out the other's
// instructions (576 dims are five places on 16 lanes, not six: 1,024 tokens x 129 heads 59.2 to 54.6 us.  Left out at run time
// they cost 3 us more than they save).
template <typename T, bool INTER, int VE, int K, bool SINGLE>
__global__ void __launch_bounds__(kNormThreads, kNormBlocks<K>) norm_rope_kernel(const __grid_constant__ NormArgs a) {
    // Weights and cos / sin in runs with gaps, so that lanes at different runs read different banks.
    constexpr int kWRun = VE >= 8 ? VE + 4 : VE;
    constexpr int RN = INTER && VE > 1 ? VE / 2 : VE;  // pairs whose cos / sin a lane reads together
    constexpr int kCRun = 2 * RN + (RN >= 4 ? 4 : 0);  // their cosines, then their sines
    extern __shared__ __align__(16) float sm[];        // weights; then cos / sin
    pdl_wait();
    float* wts = sm;
    float* cs = sm + a.weight_len;
    const int tid = threadIdx.x, NT = blockDim.x;
    const bool key = int(blockIdx.x) >= a.q.blocks;
    const NormRows& side = key ? a.k : a.q;
    const int H = side.H;
    // rows of the side, token by token
    const int row0 = (int(blockIdx.x) - (key ? a.q.blocks : 0)) * side.rows_per_block;
    const int rows = min(side.rows_per_block, a.T * H - row0);      // (a side has fewer than 2^31)
    const int t0 = row0 / H, h0 = row0 - t0 * H;
    const int lane = tid & (a.G - 1), groups = NT >> a.G_log;
    const int half = a.dims >> 1;

    // first elements of a unit's vectors (-1: none)
    int ea[K], eb[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int u = lane + k * a.G;
        ea[k] = eb[k] = -1;
        if (u < a.rot_units) {
            ea[k] = a.rope_lo + (INTER && VE == 1 ? 2 * u : u * VE);
            eb[k] = ea[k] + (INTER && VE == 1 ? 1 : half);
        } else if (u < a.units) {
            // (the later half first: with half of a row rotated, lanes then meet in no bank of the weights)
            const int p = u - a.rot_units, first = p < a.plain_pairs ? p : p + a.plain_pairs, other = p + a.plain_pairs;
            eb[k] = first * VE < a.rope_lo ? first * VE : first * VE + a.dims;
            if (p < a.plain_pairs) ea[k] = other * VE < a.rope_lo ? other * VE : other * VE + a.dims;
        }
    }
    // no lane has the vector (k, s)
    auto none = [](int k, int s) constexpr { return SINGLE && k == K - 1 && s == 0; };
    // the lane's next row: token and head counted from t0 and 0, and where it lies
    int i = tid >> a.G_log, token = (h0 + i) / H, h = h0 + i - token * H;
    const T* px = static_cast<const T*>(side.x) + int64_t(t0 + token) * side.xt + int64_t(h) * side.xh;
    T* py = static_cast<T*>(side.y) + int64_t(t0 + token) * side.yt + int64_t(h) * side.yh;
    struct Row {
        alignas(16) T v[K][2][VE];
        T* out;
        int token;
    };
    auto load = [&](Row& r) {
        r.out = nullptr;
        if (i >= rows) return;
        r.out = py;
        r.token = token;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if (!none(k, 0) && ea[k] >= 0) load_vec<T, VE>(r.v[k][0], px + ea[k]);
            if (eb[k] >= 0) load_vec<T, VE>(r.v[k][1], px + eb[k]);
        }
        i += groups;
        h += side.step_heads;
        token += side.step_tokens;
        px += side.x_step;
        py += side.y_step;
        if (h >= H) {
            h -= H;
            ++token;
            px += side.x_wrap;
            py += side.y_wrap;
        }
    };
    Row one = {}, two = {};                            // (a lane without a vector keeps zeros)
    load(one);
    // behind the first loads
    for (int j = tid; j < a.norm_dims; j += NT)
        wts[j / VE * kWRun + j % VE] = side.weight ? weight_at(side.weight, a.weight_dtype, j) + a.weight_offset : 1.f;
    if (half > 0) {
        const uint64_t* turns = generic_table(a.table.turns);
        const int pairs = ((h0 + rows - 1) / H + 1) * half;
        for (int j = tid; j < pairs; j += NT) {
            const int t = j / half;
            const float2 v = rope_cos_sin(turns[j - t * half], a.positions[t0 + t], a.table.amplitude);
            cs[j / RN * kCRun + j % RN] = v.x;
            cs[j / RN * kCRun + j % RN + RN] = v.y;
        }
    }
    __syncthreads();

    auto work = [&](Row& row) {
        float x[K][2][VE];
        float ss = 0.f;
        auto squares = [&]() {
            float sum[2] = {};
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int s = 0; s < 2; ++s)
                    if (!none(k, s) && (s ? eb[k] : ea[k]) < a.norm_dims) {
                        if constexpr (VE == 1) sum[0] = fmaf(x[k][s][0], x[k][s][0], sum[0]);
                        else {
#pragma unroll
                            for (int e = 0; e < VE; e += 2) fma2(sum, &x[k][s][e], &x[k][s][e], sum);
                        }
                    }
            ss = sum[0] + sum[1];
            for (int o = a.G >> 1; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        };
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int s = 0; s < 2; ++s)
                if (!none(k, s))
#pragma unroll
                    for (int e = 0; e < VE; ++e) x[k][s][e] = to_f32(row.v[k][s][e]);
        squares();
        const float scale = range_scale(ss, a.eps);
        if (__any_sync(0xffffffffu, scale != 1.f)) {
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int s = 0; s < 2; ++s)
                    if (!none(k, s) && (s ? eb[k] : ea[k]) < a.norm_dims)
#pragma unroll
                        for (int e = 0; e < VE; ++e) x[k][s][e] *= scale;
            squares();
        }
        const float mean = ss * a.inv_n + a.eps * scale * scale;
        const float r = sizeof(T) == 4 ? __frsqrt_rn(mean) : rsqrtf(mean);   // (2 ulp more do not show in 16 bits)
        if (row.out == nullptr) return;
        const float* turn = cs + row.token * (half / RN * kCRun);
#pragma unroll
        for (int k = 0; k < K; ++k) {
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const int e0 = s ? eb[k] : ea[k];
                if (!none(k, s) && e0 >= 0 && e0 < a.norm_dims) {
                    alignas(16) float w[VE];
                    const float* from = wts + e0 / VE * kWRun;
#pragma unroll
                    for (int e = 0; e < VE; ++e) w[e] = from[e];
                    // (the root first: x r is of size one, where r w may leave fp32's range for a weight that y has room for)
                    if constexpr (VE == 1) x[k][s][0] = x[k][s][0] * r * w[0];
                    else {
#pragma unroll
                        for (int e = 0; e < VE; e += 2) {
                            mul2(&x[k][s][e], &x[k][s][e], r, r);
                            mul2(&x[k][s][e], &x[k][s][e], w[e], w[e + 1]);
                        }
                    }
                }
            }
            const int unit = lane + k * a.G;
            if (!none(k, 0) && unit < a.rot_units) {
                if constexpr (INTER && VE > 1) {
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        const float* t = turn + (unit + s * a.rot_units) * kCRun;
#pragma unroll
                        for (int e = 0; e < VE; e += 2) {
                            const float2 v = rope_rotate(x[k][s][e], x[k][s][e + 1], make_float2(t[e >> 1], t[RN + (e >> 1)]));
                            x[k][s][e] = v.x;
                            x[k][s][e + 1] = v.y;
                        }
                    }
                } else if constexpr (VE == 1) {
                    const float2 v = rope_rotate(x[k][0][0], x[k][1][0], make_float2(turn[unit * kCRun], turn[unit * kCRun + 1]));
                    x[k][0][0] = v.x;
                    x[k][1][0] = v.y;
                } else {
                    alignas(16) float c[VE], sn[VE];
#pragma unroll
                    for (int e = 0; e < VE; ++e) {
                        c[e] = turn[unit * kCRun + e];
                        sn[e] = turn[unit * kCRun + RN + e];
                    }
#pragma unroll
                    for (int e = 0; e < VE; e += 2) {
                        float ac[2], as[2], bs[2];
                        mul2(ac, &x[k][0][e], c[e], c[e + 1]);
                        mul2(as, &x[k][0][e], sn[e], sn[e + 1]);
                        mul2(bs, &x[k][1][e], sn[e], sn[e + 1]);
                        sub2(&x[k][0][e], ac, bs);
                        fma2(&x[k][1][e], &x[k][1][e], c + e, as);
                    }
                }
            }
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const int e0 = s ? eb[k] : ea[k];
                if (!none(k, s) && e0 >= 0) {
                    alignas(16) T o[VE];
                    if constexpr (VE == 1) from_f32(o[0], x[k][s][0]);
                    else {
#pragma unroll
                        for (int e = 0; e < VE; e += 2) from_f32x2(o + e, x[k][s][e], x[k][s][e + 1]);
                    }
                    store_vec<T, VE>(row.out + e0, o);
                }
            }
        }
    };
    // the next row's loads are under way while one is worked on (lanes of a warp run out of rows together or
    // keep its exchanges company)
    for (;;) {
        load(two);
        work(one);
        if (!__any_sync(0xffffffffu, two.out != nullptr)) break;
        load(one);
        work(two);
        if (!__any_sync(0xffffffffu, one.out != nullptr)) break;
    }
}

// The rows of a side's blocks, `passes` to a lane.
void plan_side(const NormArgs& a, int64_t passes, NormRows* s) {
    s->blocks = 0;
    if (s->H == 0) return;
    const int64_t rows = int64_t(a.T) * s->H;
    const int groups = kNormThreads / a.G;
    int64_t per = passes * groups;
    // the tokens that so many rows can touch have to fit the table
    if (a.dims > 0) {
        const int64_t tokens = kNormPairs / (a.dims / 2);
        if (per > (tokens - 1) * s->H) per = (tokens - 1) * s->H;
    }
    s->rows_per_block = int(per < rows ? per : rows);
    s->blocks = int((rows + s->rows_per_block - 1) / s->rows_per_block);
    s->step_tokens = groups / s->H;
    s->step_heads = groups % s->H;
    s->x_step = s->step_tokens * s->xt + s->step_heads * s->xh;
    s->y_step = s->step_tokens * s->yt + s->step_heads * s->yh;
    s->x_wrap = s->xt - s->H * s->xh;
    s->y_wrap = s->yt - s->H * s->yh;
}

template <typename T, bool INTER, int VE, int K, bool SINGLE>
cudaError_t launch_units(NormArgs& a, int sms, cudaStream_t stream) {
    const auto kernel = norm_rope_kernel<T, INTER, VE, K, SINGLE>;
    static std::atomic<int> most{0};                   // blocks that an SM's registers have room for
    int per_sm = most.load(std::memory_order_relaxed);
    if (per_sm == 0) {
        const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, kNormThreads, 0);
        if (e != cudaSuccess) return e;
        most.store(per_sm, std::memory_order_relaxed);
    }
    // As many rows a lane as make whole waves of blocks
    const int64_t wave = int64_t(per_sm) * sms, work = int64_t(a.T) * (a.q.H + a.k.H) * a.G / kNormThreads + 1;
    const int64_t waves = (work + wave * kNormPasses - 1) / (wave * kNormPasses);
    int64_t passes = (work + wave * waves - 1) / (wave * waves);
    for (;; ++passes) {
        plan_side(a, passes, &a.q);
        plan_side(a, passes, &a.k);
        if (passes >= kNormPasses || a.q.blocks + a.k.blocks <= wave * waves) break;
    }
    // (with room for the gaps between runs)
    a.weight_len = (a.norm_dims + 7) / 8 * 12;
    auto pairs = [&](const NormRows& s) { return s.blocks ? ((s.rows_per_block + s.H - 2) / s.H + 1) * (a.dims / 2) : 0; };
    const int held = std::max(pairs(a.q), pairs(a.k));
    const size_t smem = (size_t(a.weight_len) + size_t(held + 7) / 8 * 24) * sizeof(float);
    return launch_pdl(kernel, dim3(static_cast<unsigned>(a.q.blocks + a.k.blocks)), dim3(kNormThreads), smem, stream, a);
}

template <typename T, bool INTER>
cudaError_t launch_typed(NormArgs& a, bool vectors, int sms, cudaStream_t stream) {
    constexpr int V16 = 16 / int(sizeof(T));
    const int ve = vectors ? V16 : 1;
    a.rot_units = a.dims / 2 / ve;
    const int plain = (a.width - a.dims) / ve;
    a.plain_pairs = plain / 2;
    a.units = a.rot_units + plain - a.plain_pairs;
    // lanes and units a lane: as few idle places as can be, then as few units
    int per_lane = 16;
    bool single = false;
    if (vectors) {
        int best = INT_MAX;
        for (int k = 1; k <= kNormUnits; ++k) {
            int g = 0;
            while (g < 5 && (k << g) < a.units) ++g;
            if ((k << g) >= a.units && (2 * k << g) < best) {
                best = 2 * k << g;
                per_lane = k;
                a.G_log = g;
            }
        }
        // if one vector each does for the last units, the other's place is left out
        const int before = ((per_lane - 1) << a.G_log) - a.rot_units;
        if (per_lane == 3 && before >= 0 && plain - 2 * before <= 1 << a.G_log) {
            single = true;
            a.plain_pairs = before;
            a.units = a.rot_units + plain - before;
        }
    } else {
        a.G_log = 0;
        while (a.G_log < 5 && (1 << a.G_log) < a.units) ++a.G_log;
    }
    a.G = 1 << a.G_log;
    if (!vectors) return launch_units<T, INTER, 1, 16, false>(a, sms, stream);
    if (per_lane == 1) return launch_units<T, INTER, V16, 1, false>(a, sms, stream);
    if (per_lane == 2) return launch_units<T, INTER, V16, 2, false>(a, sms, stream);
    if (per_lane == 3 && single) return launch_units<T, INTER, V16, 3, true>(a, sms, stream);
    if (per_lane == 3) return launch_units<T, INTER, V16, 3, false>(a, sms, stream);
    return launch_units<T, INTER, V16, 4, false>(a, sms, stream);
}
static_assert(kMaxNormWidth <= 2 * 16 * 32, "a row of single elements: 16 units a lane");
static_assert(kMaxNormWidth * 4 <= 2 * kNormUnits * 32 * 16, "a row of vectors");

}  // namespace

cudaError_t launch_norm_rope(NormArgs& a, int dtype, bool interleaved, bool vectors, int sms, cudaStream_t stream) {
    a.inv_n = 1.f / float(a.norm_dims);
    switch (dtype) {
        case SPLASH_F16:
            return interleaved ? launch_typed<__half, true>(a, vectors, sms, stream) : launch_typed<__half, false>(a, vectors, sms, stream);
        case SPLASH_F32:
            return interleaved ? launch_typed<float, true>(a, vectors, sms, stream) : launch_typed<float, false>(a, vectors, sms, stream);
        default:
            return interleaved ? launch_typed<__nv_bfloat16, true>(a, vectors, sms, stream)
                               : launch_typed<__nv_bfloat16, false>(a, vectors, sms, stream);
    }
}

}  // namespace splash
