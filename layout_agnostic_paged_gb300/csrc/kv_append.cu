// kv_append.cu -- writing new tokens' keys into the paged cache (bf16 or MXFP8), and
// reading MXFP8 pages back into bf16 pages.
//
// Both are HBM-bound copies with a little arithmetic.  A warp owns one token row: 512
// latents are 16 consecutive ones per lane, so that an MXFP8 group of 32 is a pair of
// lanes, and the 64 rope dims are one pair per lane.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "common.cuh"
#include "kernels.h"
#include "rope.cuh"

namespace splash {
namespace {

constexpr int kAppendThreads = 256;
constexpr int kUnpackThreads = 256;
constexpr int kUnpackRows = 4;                   // rows whose loads a warp has in flight
constexpr int kScaleBytes = kDv / 32;            // 16
constexpr int kRopeDims = kDqk - kDv;            // 64

struct AppendArgs {
    const __nv_bfloat16* latent;
    const __nv_bfloat16* k_rope;
    const int32_t* cu_q;
    const int32_t* block_table;
    const int32_t* ctx_lens;
    uint8_t* pool;
    int64_t latent_stride, rope_stride;
    int B, total_q, P, num_pages, max_pages;
    int rotate, interleaved;
    RopeTable32 table;
};

// The request that owns row t: the last r with cu[r] <= t.  32 probes a step, so that the
// 256 requests of a decode batch take two dependent loads instead of eight.
__device__ __forceinline__ int find_request(const int32_t* cu, int B, int t, int lane) {
    int lo = 0, hi = B;                           // cu[lo] <= t assumed, checked by the caller
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32;
        const int i = lo + lane * step;
        const bool le = lane == 0 || (i < hi && cu[i] <= t);
        const uint32_t m = __ballot_sync(0xffffffffu, le);
        const int k = 31 - __clz(m);              // the last probe at or below t
        lo += k * step;
        hi = min(hi, lo + step);
    }
    return lo;
}

template <bool MXFP8>
__global__ void __launch_bounds__(kAppendThreads) kv_append_kernel(const __grid_constant__ AppendArgs a) {
    constexpr int kRow = MXFP8 ? kMxRowBytes : kDqk * 2;
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int t = blockIdx.x * (kAppendThreads / 32) + (threadIdx.x >> 5);
    if (t >= a.total_q) return;
    // the row's data is on its way while the slot is looked up
    const uint4* lp = reinterpret_cast<const uint4*>(a.latent + int64_t(t) * a.latent_stride) + 2 * lane;
    uint4 in[2];
    if (MXFP8) {
        in[0] = __ldcs(lp);
        in[1] = __ldcs(lp + 1);
    } else {                                      // whole 512-byte runs per load
        in[0] = __ldcs(lp - lane);
        in[1] = __ldcs(lp - lane + 32);
    }
    const __nv_bfloat16* kp = a.k_rope + int64_t(t) * a.rope_stride;
    const int ia = a.interleaved ? 2 * lane : lane, ib = a.interleaved ? 2 * lane + 1 : lane + 32;
    __nv_bfloat16 ra = kp[ia], rb = kp[ib];

    const int r = find_request(a.cu_q, a.B, t, lane);
    const int c0 = a.cu_q[r], c1 = a.cu_q[r + 1];
    if (t < c0 || t >= c1) return;                // padding
    const int64_t pos = int64_t(a.ctx_lens[r]) - (int64_t(c1) - t);
    if (pos < 0 || pos >= int64_t(a.max_pages) * a.P) return;
    const int id = a.block_table[int64_t(r) * a.max_pages + pos / a.P];
    if (id < 0 || id >= a.num_pages) return;
    uint8_t* row = a.pool + (int64_t(id) * a.P + pos % a.P) * kRow;

    if (a.rotate) {
        const float2 y = rope_rotate(__bfloat162float(ra), __bfloat162float(rb),
                                     rope_cos_sin(a.table.turns[lane], int32_t(pos), a.table.amplitude));
        ra = __float2bfloat16_rn(y.x);
        rb = __float2bfloat16_rn(y.y);
    }
    __nv_bfloat16* kr = reinterpret_cast<__nv_bfloat16*>(row + kRow - 2 * kRopeDims);
    if (a.interleaved) {
        *reinterpret_cast<__nv_bfloat162*>(kr + 2 * lane) = __nv_bfloat162(ra, rb);
    } else {
        kr[ia] = ra;
        kr[ib] = rb;
    }
    if (!MXFP8) {
        uint4* dst = reinterpret_cast<uint4*>(row);
        dst[lane] = in[0];
        dst[32 + lane] = in[1];
        return;
    }
    float x[16];
    const uint32_t* w = reinterpret_cast<const uint32_t*>(in);
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const float m = fabsf(x[i]);
        if (m < INFINITY) top = fmaxf(top, m);    // false for NaN
    }
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
    // least e with top <= 448 * 2^e: 448 = 1.75 * 2^8, so one more when the mantissa is above 1.75
    const uint32_t bits = __float_as_uint(top);
    int e = int(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
    e = max(e, -127);
    const float inv = __uint_as_float(uint32_t(127 - e) << 23);      // 2^-e, exact
    uint32_t q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t l = __nv_cvt_float2_to_fp8x2(make_float2(x[4 * i] * inv, x[4 * i + 1] * inv), __NV_SATFINITE, __NV_E4M3);
        const uint32_t h = __nv_cvt_float2_to_fp8x2(make_float2(x[4 * i + 2] * inv, x[4 * i + 3] * inv), __NV_SATFINITE, __NV_E4M3);
        q[i] = l | (h << 16);
    }
    reinterpret_cast<uint4*>(row)[lane] = make_uint4(q[0], q[1], q[2], q[3]);
    // lane 2g holds group g's scale: pack four at a time into lanes 0, 8, 16 and 24
    uint32_t s = uint32_t(e + 127);
    s |= __shfl_down_sync(0xffffffffu, s, 2) << 8;
    s |= __shfl_down_sync(0xffffffffu, s, 4) << 16;
    if ((lane & 7) == 0) reinterpret_cast<uint32_t*>(row + kDv)[lane >> 3] = s;
}

// Two e4m3 codes times a power of two, as packed bf16.
__device__ __forceinline__ uint32_t mx_pair(uint32_t codes, float scale) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(__nv_fp8x2_storage_t(codes & 0xffffu), __NV_E4M3);
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    const __nv_bfloat162 v = __floats2bfloat162_rn(f.x * scale, f.y * scale);
    return *reinterpret_cast<const uint32_t*>(&v);
}

__global__ void __launch_bounds__(kUnpackThreads) kv_unpack_kernel(
    const uint8_t* __restrict__ src, uint8_t* __restrict__ dst, int P, int groups_per_page,
    const int32_t* __restrict__ src_ids, const int32_t* __restrict__ dst_ids, int64_t items,
    int src_np, int dst_np) {
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int64_t warps = int64_t(gridDim.x) * (kUnpackThreads / 32);
    for (int64_t i = int64_t(blockIdx.x) * (kUnpackThreads / 32) + (threadIdx.x >> 5); i < items; i += warps) {
        const int64_t pg = i / groups_per_page;
        const int r0 = int(i % groups_per_page) * kUnpackRows;
        const int s = src_ids[pg], d = dst_ids[pg];
        if (s < 0 || s >= src_np || d < 0 || d >= dst_np) continue;
        const uint8_t* sp = src + (int64_t(s) * P + r0) * kMxRowBytes;
        uint8_t* dp = dst + (int64_t(d) * P + r0) * (kDqk * 2);
        const int n = min(kUnpackRows, P - r0);
        uint4 c[kUnpackRows], k[kUnpackRows];
        uint32_t b[kUnpackRows];
#pragma unroll
        for (int u = 0; u < kUnpackRows; ++u)
            if (u < n) {
                const uint8_t* row = sp + u * kMxRowBytes;
                c[u] = __ldcs(reinterpret_cast<const uint4*>(row) + lane);
                b[u] = __ldcs(row + kDv + (lane >> 1));
                if (lane < 8) k[u] = __ldcs(reinterpret_cast<const uint4*>(row + kDv + kScaleBytes) + lane);
            }
#pragma unroll
        for (int u = 0; u < kUnpackRows; ++u)
            if (u < n) {
                // 2^(b - 127): the byte is the exponent field, 0 is 2^-127 (a subnormal), 255 NaN
                const uint32_t sb = b[u] == 255 ? 0x7fc00000u : (b[u] << 23) | (b[u] == 0 ? 0x400000u : 0u);
                const float scale = __uint_as_float(sb);
                uint4 o[2];
                const uint32_t w[4] = {c[u].x, c[u].y, c[u].z, c[u].w};
                uint32_t* ow = reinterpret_cast<uint32_t*>(o);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    ow[2 * j] = mx_pair(w[j], scale);
                    ow[2 * j + 1] = mx_pair(w[j] >> 16, scale);
                }
                uint4* row = reinterpret_cast<uint4*>(dp + u * (kDqk * 2));
                __stcs(row + 2 * lane, o[0]);
                __stcs(row + 2 * lane + 1, o[1]);
                if (lane < 8) __stcs(row + kDv / 8 + lane, k[u]);
            }
    }
}

}  // namespace

cudaError_t launch_kv_append(const RopeTable32* table, bool interleaved, bool mxfp8, const void* latent,
                             int64_t latent_stride, const void* k_rope, int64_t rope_stride,
                             const int32_t* cu_q, int B, int total_q, const int32_t* block_table,
                             const int32_t* ctx_lens, int P, int num_pages, int max_pages, void* pool,
                             cudaStream_t stream) {
    AppendArgs a = {};
    a.latent = static_cast<const __nv_bfloat16*>(latent);
    a.k_rope = static_cast<const __nv_bfloat16*>(k_rope);
    a.cu_q = cu_q;
    a.block_table = block_table;
    a.ctx_lens = ctx_lens;
    a.pool = static_cast<uint8_t*>(pool);
    a.latent_stride = latent_stride;
    a.rope_stride = rope_stride;
    a.B = B;
    a.total_q = total_q;
    a.P = P;
    a.num_pages = num_pages;
    a.max_pages = max_pages;
    a.rotate = table != nullptr;
    a.interleaved = interleaved;
    if (table) a.table = *table;
    const int per_block = kAppendThreads / 32;
    const dim3 g((total_q + per_block - 1) / per_block), b(kAppendThreads);
    if (mxfp8) return launch_pdl(kv_append_kernel<true>, g, b, 0, stream, a);
    return launch_pdl(kv_append_kernel<false>, g, b, 0, stream, a);
}

cudaError_t launch_kv_unpack(const void* src, void* dst, int P, const int32_t* src_ids,
                             const int32_t* dst_ids, int n, int src_np, int dst_np, int sms,
                             cudaStream_t stream) {
    const int gpp = (P + kUnpackRows - 1) / kUnpackRows;
    const int64_t items = int64_t(n) * gpp;
    const int64_t blocks = (items + kUnpackThreads / 32 - 1) / (kUnpackThreads / 32);
    const int64_t most = int64_t(sms) * 8;
    return launch_pdl(kv_unpack_kernel, dim3(unsigned(blocks < most ? blocks : most)), dim3(kUnpackThreads),
                      0, stream, static_cast<const uint8_t*>(src), static_cast<uint8_t*>(dst), P, gpp,
                      src_ids, dst_ids, items, src_np, dst_np);
}

}  // namespace splash
