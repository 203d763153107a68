// kv_append.cu -- writing new tokens' keys into the paged cache (bf16 or MXFP8), and
// reading MXFP8 pages back into bf16 pages.
//
// Both are HBM-bound copies with a little arithmetic.  A warp owns one token row: 512
// latents are 16 consecutive ones per lane, so that an MXFP8 group of 32 is a pair of
// lanes, and the 64 rope dims are one pair per lane.  An append's warp is a chain of two to three
// dependent loads (the owner of the row, its page, the stores), so many warps with one row each
// beat fewer with more: 36,600 rows to MXFP8 (66 MB) in 12.5 us (78% of the copy bandwidth; four rows a
// warp took half as long again) and to bf16 (84 MB) in 14.5 us (86%); one row of each of 256 requests in
// 1.9 us.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "common.cuh"
#include "kernels.h"
#include "rope.cuh"
#include "vec32.cuh"

namespace splash {
namespace {

constexpr int kAppendThreads = 256;
constexpr int kUnpackThreads = 256;
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
    int B, total_q, P_log, num_pages, max_pages;
    int rotate, interleaved;
    RopeTable32 table;
};

// The request that owns row t (the last r with cu[r] <= t), its rows [c0, c1) and context.  32
// probes a step, and the last step brings the offsets and lengths along: a batch of 31 requests takes one
// round trip to memory, 256 requests two.
struct Owner {
    int r, c0, c1, ctx;
};
__device__ __forceinline__ Owner find_owner(const int32_t* cu, const int32_t* ctx_lens, int B, int t, int lane) {
    int lo = 0, hi = B;                           // cu[lo] <= t assumed, checked by the caller
    while (hi - lo > 31) {
        const int step = (hi - lo + 31) / 32;
        const int i = lo + lane * step;
        const uint32_t m = __ballot_sync(0xffffffffu, lane == 0 || (i < hi && cu[i] <= t));
        lo += (31 - __clz(m)) * step;             // the last probe at or below t
        hi = min(hi, lo + step);
    }
    const int c = cu[min(lo + lane, B)];
    const int len = ctx_lens[min(lo + lane, B - 1)];
    const uint32_t m = __ballot_sync(0xffffffffu, lane == 0 || (lane < hi - lo && c <= t));
    const int k = 31 - __clz(m);                  // k + 1 <= hi - lo <= 31
    Owner o;
    o.r = lo + k;
    o.c0 = __shfl_sync(0xffffffffu, c, k);
    o.c1 = __shfl_sync(0xffffffffu, c, k + 1);
    o.ctx = __shfl_sync(0xffffffffu, len, k);
    return o;
}

template <bool MXFP8>
__global__ void __launch_bounds__(kAppendThreads) kv_append_kernel(const __grid_constant__ AppendArgs a) {
    constexpr int kRow = MXFP8 ? kMxRowBytes : kDqk * 2;
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int t = blockIdx.x * (kAppendThreads / 32) + (threadIdx.x >> 5);
    if (t >= a.total_q) return;
    // the row's data is on its way while its slot is looked up.  MXFP8: 16 consecutive latents a
    // lane; bf16: whole 512-byte runs per load
    const uint4* lp = reinterpret_cast<const uint4*>(a.latent + int64_t(t) * a.latent_stride);
    const uint4 v0 = __ldcs(lp + (MXFP8 ? 2 * lane : lane)), v1 = __ldcs(lp + (MXFP8 ? 2 * lane + 1 : lane + 32));
    const __nv_bfloat16* kp = a.k_rope + int64_t(t) * a.rope_stride;
    const int ia = a.interleaved ? 2 * lane : lane, ib = a.interleaved ? 2 * lane + 1 : lane + 32;
    __nv_bfloat16 ra = kp[ia], rb = kp[ib];
    const uint64_t F = a.rotate ? generic_table(a.table.turns)[lane] : 0;

    const Owner o = find_owner(a.cu_q, a.ctx_lens, a.B, t, lane);
    const int pos = o.ctx - (o.c1 - t);
    // padding, or a position without a place
    if (t < o.c0 || t >= o.c1 || pos < 0 || (pos >> a.P_log) >= a.max_pages) return;
    const int id = a.block_table[int64_t(o.r) * a.max_pages + (pos >> a.P_log)];
    if (id < 0 || id >= a.num_pages) return;
    uint8_t* row = a.pool + ((int64_t(id) << a.P_log) + (pos & ((1 << a.P_log) - 1))) * kRow;

    if (a.rotate) {
        const float2 y = rope_rotate(__bfloat162float(ra), __bfloat162float(rb),
                                     rope_cos_sin(F, pos, a.table.amplitude));
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
        dst[lane] = v0;
        dst[32 + lane] = v1;
        return;
    }
    // the group's largest magnitude: bf16 bits without the sign order like the values, and anything from
    // 0x7f80 on is not finite
    const uint32_t w[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = __vmaxu2(top, w[i] & 0x7fff7fffu);
    top = max(top & 0xffffu, top >> 16);
    if (top >= 0x7f80u) {
        top = 0;
        for (int i = 0; i < 16; ++i) {
            const uint32_t m = (w[i >> 1] >> (16 * (i & 1))) & 0x7fffu;
            if (m < 0x7f80u) top = max(top, m);
        }
    }
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    // least e with top <= 448 * 2^e: 448 = 1.75 * 2^8, so one more when the mantissa is above 1.75
    const int e = max(int(top >> 7) - 127 - 8 + ((top & 0x7fu) > 0x60u ? 1 : 0), -127);
    const float inv = __uint_as_float(uint32_t(127 - e) << 23);      // 2^-e, exact
    uint32_t q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 lo = make_float2(__uint_as_float(w[2 * i] << 16) * inv, __uint_as_float(w[2 * i] & 0xffff0000u) * inv);
        const float2 hi = make_float2(__uint_as_float(w[2 * i + 1] << 16) * inv, __uint_as_float(w[2 * i + 1] & 0xffff0000u) * inv);
        q[i] = uint32_t(__nv_cvt_float2_to_fp8x2(lo, __NV_SATFINITE, __NV_E4M3)) |
               uint32_t(__nv_cvt_float2_to_fp8x2(hi, __NV_SATFINITE, __NV_E4M3)) << 16;
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

template <int ROWS>   // rows whose loads a warp has in flight
__global__ void __launch_bounds__(kUnpackThreads) kv_unpack_kernel(
    const uint8_t* __restrict__ src, uint8_t* __restrict__ dst, int P, int groups_per_page,
    const int32_t* __restrict__ src_ids, const int32_t* __restrict__ dst_ids, int64_t items,
    int src_np, int dst_np) {
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const bool wide = (reinterpret_cast<uintptr_t>(dst) & 31) == 0;   // whole sectors per store
    const int64_t warps = int64_t(gridDim.x) * (kUnpackThreads / 32);
    for (int64_t i = int64_t(blockIdx.x) * (kUnpackThreads / 32) + (threadIdx.x >> 5); i < items; i += warps) {
        const int64_t pg = i / groups_per_page;
        const int r0 = int(i % groups_per_page) * ROWS;
        const int s = src_ids[pg], d = dst_ids[pg];
        if (s < 0 || s >= src_np || d < 0 || d >= dst_np) continue;
        const uint8_t* sp = src + (int64_t(s) * P + r0) * kMxRowBytes;
        uint8_t* dp = dst + (int64_t(d) * P + r0) * (kDqk * 2);
        const int n = min(ROWS, P - r0);
        uint4 c[ROWS], k[ROWS];
        uint32_t b[ROWS];
#pragma unroll
        for (int u = 0; u < ROWS; ++u)
            if (u < n) {
                const uint8_t* row = sp + u * kMxRowBytes;
                c[u] = __ldcs(reinterpret_cast<const uint4*>(row) + lane);
                b[u] = __ldcs(row + kDv + (lane >> 1));
                if (lane < 8) k[u] = __ldcs(reinterpret_cast<const uint4*>(row + kDv + kScaleBytes) + lane);
            }
#pragma unroll
        for (int u = 0; u < ROWS; ++u)
            if (u < n) {
                // 2^(b - 127): the byte is the exponent field, 0 is 2^-127 (a subnormal), 255 NaN
                const uint32_t sb = b[u] == 255 ? 0x7fc00000u : (b[u] << 23) | (b[u] == 0 ? 0x400000u : 0u);
                const float scale = __uint_as_float(sb);
                uint32_t o[8];
                const uint32_t w[4] = {c[u].x, c[u].y, c[u].z, c[u].w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    o[2 * j] = mx_pair(w[j], scale);
                    o[2 * j + 1] = mx_pair(w[j] >> 16, scale);
                }
                uint4* row = reinterpret_cast<uint4*>(dp + u * (kDqk * 2));
                if (wide) {
                    store32_cs(row + 2 * lane, o);
                } else {
                    __stcs(row + 2 * lane, make_uint4(o[0], o[1], o[2], o[3]));
                    __stcs(row + 2 * lane + 1, make_uint4(o[4], o[5], o[6], o[7]));
                }
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
    for (a.P_log = 4; (1 << a.P_log) < P; ++a.P_log) {}      // P is 16, 32, 64 or 128
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
    // Four rows a warp and one pass of the grid (8,192 pages of 64 tokens: 146 us, 95% of the copy
    // bandwidth; eight blocks an SM in a loop took 158, 16-byte stores 189); a row a warp when those
    // warps would not fill the SMs (8 pages: 1.8 against 2.1 us).
    const bool few = int64_t(n) * P < int64_t(sms) * 64 * 4;
    const int rows = few ? 1 : 4;
    const int gpp = (P + rows - 1) / rows;
    const int64_t items = int64_t(n) * gpp;
    int64_t blocks = (items + kUnpackThreads / 32 - 1) / (kUnpackThreads / 32);
    if (blocks > (int64_t(1) << 30)) blocks = int64_t(1) << 30;
    const dim3 g(static_cast<unsigned>(blocks)), b(kUnpackThreads);
    const uint8_t* s = static_cast<const uint8_t*>(src);
    uint8_t* o = static_cast<uint8_t*>(dst);
    if (few) return launch_pdl(kv_unpack_kernel<1>, g, b, 0, stream, s, o, P, gpp, src_ids, dst_ids, items, src_np, dst_np);
    return launch_pdl(kv_unpack_kernel<4>, g, b, 0, stream, s, o, P, gpp, src_ids, dst_ids, items, src_np, dst_np);
}

}  // namespace splash
