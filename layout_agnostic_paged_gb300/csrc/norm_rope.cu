// norm_rope.cu -- splash_norm_rope: RMS norm of query and key head rows and the rotation of a part of
// each row, in one pass.
//
//   y_j = x_j * rsqrt(mean(x_0^2 .. x_{n-1}^2) + eps) * (w_j + offset)  for j < n, x_j behind them,
//   then pairs of dims [lo, lo + d) are rotated by the token's position.
//
// HBM-bound: every element is read and written once, where a norm and a rotation one after the other move
// it twice.  G lanes hold a row in registers: each has "units" of two vectors, and the two vectors of a
// rotated unit are the halves of its pairs (d / 2 apart), so that no element crosses lanes and only the sum
// of squares does.  A block owns a run of one token's rows, queries and keys alike, or all rows of a few
// tokens where one's are few; its tokens' cos / sin and the weights lie in shared memory.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"
#include "kernels.h"
#include "rope.cuh"

namespace splash {
namespace {

constexpr int kNormThreads = 256;    // a block's, at most
constexpr int kNormPairs = 256;      // cos / sin a block holds, at most (one token has 128 at most)
template <int K>
constexpr int norm_rows_per_lane = K == 1 ? 2 : 1;   // 32 to 64 bytes of loads in flight

__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ void from_f32(__nv_bfloat16& d, float v) { d = __float2bfloat16_rn(v); }
__device__ __forceinline__ void from_f32(__half& d, float v) { d = __float2half_rn(v); }
__device__ __forceinline__ void from_f32(float& d, float v) { d = v; }

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

// VE elements a vector, K units a lane, U rows of a lane in flight (a block has no more rows than that).
template <typename T, bool INTER, int VE, int K>
__global__ void __launch_bounds__(kNormThreads) norm_rope_kernel(const __grid_constant__ NormArgs a) {
    constexpr int U = norm_rows_per_lane<K>;
    // Weights and cos / sin in runs with gaps, so that lanes at different runs read different banks.
    constexpr int kWRun = VE >= 8 ? VE + 4 : VE;
    constexpr int RN = INTER && VE > 1 ? VE / 2 : VE;  // pairs whose cos / sin a lane reads together
    constexpr int kCRun = RN >= 4 ? RN + 2 : RN;
    extern __shared__ __align__(16) float sm[];        // weights of q and of k; then cos / sin
    pdl_wait();
    float* wts = sm;
    float2* cs = reinterpret_cast<float2*>(sm + 2 * a.weight_len);
    const int tid = threadIdx.x, NT = blockDim.x;
    const int t0 = blockIdx.x / a.chunks * a.tokens_per_block;
    const int ntok = min(a.tokens_per_block, a.T - t0);
    const int j0 = (blockIdx.x % a.chunks) * a.rows_per_block;
    const int nrow = min(a.rows_per_block, a.q.H + a.k.H - j0);
    const int rows = ntok * nrow;                      // of the block
    const int lane = tid & (a.G - 1), groups = NT >> a.G_log;
    const int half = a.dims >> 1;
    const uint64_t* turns = generic_table(a.table.turns);

    // first elements of a unit's vectors; -1: none
    int ea[K], eb[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int u = lane + k * a.G;
        ea[k] = eb[k] = -1;
        if (u < a.rot_units) {
            ea[k] = a.rope_lo + (INTER && VE == 1 ? 2 * u : u * VE);
            eb[k] = ea[k] + (INTER && VE == 1 ? 1 : half);
        } else if (u < a.units) {
            const int p = u - a.rot_units, other = p + a.plain_units;
            ea[k] = p * VE < a.rope_lo ? p * VE : p * VE + a.dims;
            if (other * VE < a.width - a.dims) eb[k] = other * VE < a.rope_lo ? other * VE : other * VE + a.dims;
        }
    }
    alignas(16) T in[U][K][2][VE];
    T* out[U];
    int token[U];
    bool key[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int i = (tid >> a.G_log) + u * groups;
        out[u] = nullptr;
        token[u] = 0;
        key[u] = false;
        if (i < rows) {
            token[u] = ntok == 1 ? 0 : i / nrow;
            const int j = j0 + i - token[u] * nrow;
            key[u] = j >= a.q.H;
            const NormRows& s = key[u] ? a.k : a.q;
            const int h = key[u] ? j - a.q.H : j;
            const T* x = static_cast<const T*>(s.x) + int64_t(t0 + token[u]) * s.xt + int64_t(h) * s.xh;
            out[u] = static_cast<T*>(s.y) + int64_t(t0 + token[u]) * s.yt + int64_t(h) * s.yh;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                if (ea[k] >= 0) load_vec<T, VE>(in[u][k][0], x + ea[k]);
                if (eb[k] >= 0) load_vec<T, VE>(in[u][k][1], x + eb[k]);
            }
        }
    }
    // behind the loads
    for (int i = tid; i < a.norm_dims; i += NT) {
        const int at = i / VE * kWRun + i % VE;
        wts[at] = a.q.weight ? weight_at(a.q.weight, a.weight_dtype, i) + a.weight_offset : 1.f;
        wts[a.weight_len + at] = a.k.weight ? weight_at(a.k.weight, a.weight_dtype, i) + a.weight_offset : 1.f;
    }
    for (int i = tid; i < ntok * half; i += NT) {
        const int tok = ntok == 1 ? 0 : i / half;
        cs[i / RN * kCRun + i % RN] = rope_cos_sin(turns[i - tok * half], a.positions[t0 + tok], a.table.amplitude);
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < U; ++u) {
        float x[K][2][VE];
        float ss = 0.f;
        auto squares = [&]() {
            ss = 0.f;
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int s = 0; s < 2; ++s)
                    if ((s ? eb[k] : ea[k]) < a.norm_dims)
#pragma unroll
                        for (int e = 0; e < VE; ++e) ss = fmaf(x[k][s][e], x[k][s][e], ss);
            for (int o = a.G >> 1; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        };
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int e = 0; e < VE; ++e)
                    x[k][s][e] = out[u] != nullptr && (s ? eb[k] : ea[k]) >= 0 ? to_f32(in[u][k][s][e]) : 0.f;
        squares();
        const float scale = range_scale(ss, a.eps);
        if (__any_sync(0xffffffffu, scale != 1.f)) {
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int s = 0; s < 2; ++s)
                    if ((s ? eb[k] : ea[k]) < a.norm_dims)
#pragma unroll
                        for (int e = 0; e < VE; ++e) x[k][s][e] *= scale;
            squares();
        }
        const float r = rsqrtf(ss * a.inv_n + a.eps * scale * scale);
        if (out[u] == nullptr) continue;
        const float* w = wts + (key[u] ? a.weight_len : 0);
        const float2* turn = cs + token[u] * (half / RN * kCRun);
#pragma unroll
        for (int k = 0; k < K; ++k) {
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const int e0 = s ? eb[k] : ea[k];
                if (e0 >= 0 && e0 < a.norm_dims) {
#pragma unroll
                    for (int e = 0; e < VE; ++e) x[k][s][e] *= r * w[e0 / VE * kWRun + e];
                }
            }
            const int unit = lane + k * a.G;
            if (unit < a.rot_units) {
                if constexpr (INTER && VE > 1) {
#pragma unroll
                    for (int s = 0; s < 2; ++s)
#pragma unroll
                        for (int e = 0; e < VE; e += 2) {
                            const float2 v = rope_rotate(x[k][s][e], x[k][s][e + 1], turn[(unit + s * a.rot_units) * kCRun + (e >> 1)]);
                            x[k][s][e] = v.x;
                            x[k][s][e + 1] = v.y;
                        }
                } else {
#pragma unroll
                    for (int e = 0; e < VE; ++e) {
                        const float2 v = rope_rotate(x[k][0][e], x[k][1][e], turn[unit * kCRun + e]);
                        x[k][0][e] = v.x;
                        x[k][1][e] = v.y;
                    }
                }
            }
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const int e0 = s ? eb[k] : ea[k];
                if (e0 >= 0) {
                    alignas(16) T o[VE];
#pragma unroll
                    for (int e = 0; e < VE; ++e) from_f32(o[e], x[k][s][e]);
                    store_vec<T, VE>(out[u] + e0, o);
                }
            }
        }
    }
}

template <typename T, bool INTER, int VE, int K>
cudaError_t launch_units(NormArgs& a, int sms, cudaStream_t stream) {
    constexpr int U = norm_rows_per_lane<K>;
    const int R = a.q.H + a.k.H;
    // rows that a block's threads hold at once; a token's rows in equal runs of at most so many
    const int fit = kNormThreads / a.G * U;
    a.chunks = (R + fit - 1) / fit;
    a.rows_per_block = (R + a.chunks - 1) / a.chunks;
    // more tokens a block where one leaves threads without work, as long as the blocks fill the GPU
    a.tokens_per_block = 1;
    if (a.chunks == 1) {
        const int64_t spread = a.T / (int64_t(sms) * 4);
        int most = fit / R;
        if (a.dims > 0 && most > kNormPairs / (a.dims / 2)) most = kNormPairs / (a.dims / 2);
        a.tokens_per_block = spread < 1 || most < 1 ? 1 : (spread < most ? int(spread) : most);
    }
    const int groups = (a.tokens_per_block * a.rows_per_block + U - 1) / U;
    const int threads = (groups * a.G + 31) / 32 * 32;
    // (with room for the gaps between runs)
    a.weight_len = (a.norm_dims + 7) / 8 * 12;
    const size_t smem = 2 * size_t(a.weight_len) * sizeof(float) +
                        size_t(a.tokens_per_block) * ((a.dims / 2 + 3) / 4 * 6) * sizeof(float2);
    const int64_t grid = (int64_t(a.T) + a.tokens_per_block - 1) / a.tokens_per_block * a.chunks;
    return launch_pdl(norm_rope_kernel<T, INTER, VE, K>, dim3(static_cast<unsigned>(grid)), dim3(threads), smem, stream, a);
}

template <typename T, bool INTER>
cudaError_t launch_typed(NormArgs& a, bool vectors, int sms, cudaStream_t stream) {
    constexpr int V16 = 16 / int(sizeof(T));
    const int ve = vectors ? V16 : 1;
    a.rot_units = a.dims / 2 / ve;
    const int plain = (a.width - a.dims) / ve;
    a.plain_units = (plain + 1) / 2;
    a.units = a.rot_units + a.plain_units;
    a.G_log = 0;
    while (a.G_log < 5 && (1 << a.G_log) < a.units) ++a.G_log;
    a.G = 1 << a.G_log;
    const int per_lane = (a.units + a.G - 1) / a.G;
    if (!vectors) return launch_units<T, INTER, 1, 16>(a, sms, stream);
    if (per_lane == 1) return launch_units<T, INTER, V16, 1>(a, sms, stream);
    if constexpr (sizeof(T) == 4)
        if (per_lane > 2) return launch_units<T, INTER, V16, 4>(a, sms, stream);
    return launch_units<T, INTER, V16, 2>(a, sms, stream);
}
static_assert(kMaxNormWidth <= 2 * 16 * 32, "a row of single elements: 16 units a lane");
static_assert(kMaxNormWidth * 4 <= 2 * 4 * 32 * 16, "a row of vectors: 4 units a lane in fp32, 2 in 16 bits");

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
