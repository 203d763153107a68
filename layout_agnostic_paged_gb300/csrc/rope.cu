// rope.cu -- splash_rope: rotary positions of head rows, in place or from one strided
// tensor to another.
//
// HBM-bound: every rotated element is read and written once.  A block owns a run of one token's
// heads, or all heads of a few tokens where a token's are too few for its threads.  The cos / sin of
// its tokens' d / 2 pairs are computed once per block into shared memory, behind its first loads, and
// serve all of its heads.  Threads move
// 32 bytes at a time, so that a sector is written by one store.  8,191 tokens x 64 heads x 128
// dims of fp16 (268 MB): 39.5 us, the copy bandwidth; 256 tokens x 128 heads x 64 dims inside wider
// rows (8.4 MB): 2.4 us (16-byte vectors: 2.9 us).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"
#include "kernels.h"
#include "rope.cuh"
#include "vec32.cuh"

namespace splash {
namespace {

constexpr int kRopeThreads = 128;   // (64 and 256 take the same time, within 2%)

__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ void from_f32(__nv_bfloat16& d, float v) { d = __float2bfloat16_rn(v); }
__device__ __forceinline__ void from_f32(__half& d, float v) { d = __float2half_rn(v); }
__device__ __forceinline__ void from_f32(float& d, float v) { d = v; }

// N elements between registers and global memory: 32 or 16 bytes, or one element.
template <typename T, int N>
__device__ __forceinline__ void load_vec(T* v, const T* p) {
    if constexpr (N * sizeof(T) == 32) load32_cs(reinterpret_cast<uint32_t*>(v), p);
    else if constexpr (N * sizeof(T) == 16) *reinterpret_cast<uint4*>(v) = __ldcs(reinterpret_cast<const uint4*>(p));
    else *v = *p;
}
template <typename T, int N>
__device__ __forceinline__ void store_vec(T* p, const T* v) {
    if constexpr (N * sizeof(T) == 32) store32_cs(p, reinterpret_cast<const uint32_t*>(v));
    else if constexpr (N * sizeof(T) == 16) __stcs(reinterpret_cast<uint4*>(p), *reinterpret_cast<const uint4*>(v));
    else *p = *v;
}

struct RopeArgs {
    const void* x;
    void* y;
    const int32_t* positions;
    int64_t xt, xh, yt, yh;   // strides in elements
    int T, H, heads_per_block, dims;
    int chunks;               // runs of heads per token
    int tokens_per_block;     // above 1 only with one run
    RopeTable table;
};

// Work items whose loads a thread has in flight: 64 bytes.
template <typename T, int NP>
constexpr int kRopeUnroll = 2 * NP * sizeof(T) >= 64 ? 1 : (2 * NP * sizeof(T) >= 32 ? 2 : 4);

// VE elements a vector: 32 or 16 bytes, or 1 element where alignment or d forbids them.  A work item is
// VE / 2 pairs of one head in the interleaved layout (at least one pair) and VE pairs in the half layout.
constexpr int kRopeTablePairs = 256;   // of a block's tokens: 2 KB to 3 KB

template <typename T, bool INTER, int VE>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeArgs a) {
    constexpr int W = INTER && VE == 1 ? 2 : VE;       // elements of one load group
    constexpr int NP = INTER ? W / 2 : VE;             // pairs of a work item
    constexpr int U = kRopeUnroll<T, NP>;
    // runs of NP pairs, 16 bytes apart: threads at different runs of a head read different banks (without
    // the gap four of them met in one, and the large case took 46 us)
    constexpr int kRun = NP >= 4 ? NP + 2 : NP;
    __shared__ alignas(16) float2 cs[kRopeTablePairs / NP * kRun];
    pdl_wait();
    const int t = blockIdx.x / a.chunks * a.tokens_per_block;
    const int ntok = min(a.tokens_per_block, a.T - t);
    const int h0 = (blockIdx.x % a.chunks) * a.heads_per_block;
    const int nh = min(a.heads_per_block, a.H - h0);
    const int half = a.dims >> 1;
    const int per_head = half / NP;                    // work items of a head
    const int per_token = nh * per_head;
    const int items = ntok * per_token;
    const T* x = static_cast<const T*>(a.x) + int64_t(t) * a.xt + int64_t(h0) * a.xh;
    T* y = static_cast<T*>(a.y) + int64_t(t) * a.yt + int64_t(h0) * a.yh;
    const uint64_t* turns = generic_table(a.table.turns);
    struct Item {
        int token, head, run;
    };
    auto item = [&](int i) -> Item {
        const int token = ntok == 1 ? 0 : i / per_token;
        i -= token * per_token;
        return Item{token, i / per_head, i % per_head};
    };
    bool ready = false;
    for (int i0 = threadIdx.x; !ready || i0 < items; i0 += kRopeThreads * U) {
        alignas(32) T in[U][2 * NP];                     // the pairs' elements, as loaded
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = i0 + u * kRopeThreads;
            if (i < items) {
                const Item w = item(i);
                const T* p = x + w.token * a.xt + w.head * a.xh + (INTER ? w.run * 2 * NP : w.run * NP);
                if (INTER) {
#pragma unroll
                    for (int e = 0; e < 2 * NP; e += VE) load_vec<T, VE>(&in[u][e], p + e);
                } else {
                    load_vec<T, VE>(&in[u][0], p);
                    load_vec<T, VE>(&in[u][NP], p + half);
                }
            }
        }
        if (!ready) {
            for (int j = threadIdx.x; j < ntok * half; j += kRopeThreads) {
                const int token = ntok == 1 ? 0 : j / half;
                cs[j / NP * kRun + j % NP] =
                    rope_cos_sin(turns[j - token * half], a.positions[t + token], a.table.amplitude);
            }
            __syncthreads();
            ready = true;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = i0 + u * kRopeThreads;
            if (i < items) {
                const Item w = item(i);
                T* p = y + w.token * a.yt + w.head * a.yh + (INTER ? w.run * 2 * NP : w.run * NP);
                const float2* turn = cs + (w.token * per_head + w.run) * kRun;
#pragma unroll
                for (int e = 0; e < NP; ++e) {
                    T& ea = in[u][INTER ? 2 * e : e];
                    T& eb = in[u][INTER ? 2 * e + 1 : NP + e];
                    const float2 r = rope_rotate(to_f32(ea), to_f32(eb), turn[e]);
                    from_f32(ea, r.x);
                    from_f32(eb, r.y);
                }
                if (INTER) {
#pragma unroll
                    for (int e = 0; e < 2 * NP; e += VE) store_vec<T, VE>(p + e, &in[u][e]);
                } else {
                    store_vec<T, VE>(p, &in[u][0]);
                    store_vec<T, VE>(p + half, &in[u][NP]);
                }
            }
        }
    }
}

template <typename T, bool INTER, int VE>
cudaError_t launch_vec(RopeArgs& a, int T_, int sms, cudaStream_t stream) {
    constexpr int NP = INTER && VE > 1 ? VE / 2 : VE;
    const int per_head = (a.dims / 2) / NP;
    // One pass of a block covers kRopeThreads * U work items.  Fewer heads a block
    // when the tokens alone would not fill the GPU.
    int heads = (kRopeThreads * kRopeUnroll<T, NP>) / per_head;
    if (heads < 1) heads = 1;
    const int64_t want = int64_t(sms) * 4;
    while (heads > 1 && int64_t(T_) * ((a.H + heads - 1) / heads) < want &&
           int64_t(heads) * per_head > kRopeThreads)
        heads = (heads + 1) / 2;
    if (heads > a.H) heads = a.H;
    a.heads_per_block = heads;
    a.chunks = (a.H + heads - 1) / heads;
    // More tokens a block where one leaves threads without work, as long as the blocks fill the GPU
    // (6,139 tokens of 5 heads x 32 fp32 dims: 3.3 us, with a block per token 5.9; 36,585 tokens of one head
    // x 64 bf16 dims inside wider rows: 8.0 against 27.5).
    a.tokens_per_block = 1;
    if (a.chunks == 1) {
        const int fit = (kRopeThreads * kRopeUnroll<T, NP>) / (a.H * per_head), table = kRopeTablePairs / (a.dims / 2);
        const int64_t spread = T_ / want;
        const int most = fit < table ? fit : table;
        a.tokens_per_block = spread < 1 || most < 1 ? 1 : (spread < most ? int(spread) : most);
    }
    const int64_t grid = (int64_t(T_) + a.tokens_per_block - 1) / a.tokens_per_block * a.chunks;
    return launch_pdl(rope_kernel<T, INTER, VE>, dim3(static_cast<unsigned>(grid)), dim3(kRopeThreads), 0, stream, a);
}

template <typename T>
cudaError_t launch_typed(RopeArgs& a, int T_, bool inter, int vec_bytes, int sms, cudaStream_t stream) {
    constexpr int V32 = 32 / int(sizeof(T)), V16 = 16 / int(sizeof(T));
    if (inter) {
        if (vec_bytes == 32) return launch_vec<T, true, V32>(a, T_, sms, stream);
        if (vec_bytes == 16) return launch_vec<T, true, V16>(a, T_, sms, stream);
        return launch_vec<T, true, 1>(a, T_, sms, stream);
    }
    if (vec_bytes == 32) return launch_vec<T, false, V32>(a, T_, sms, stream);
    if (vec_bytes == 16) return launch_vec<T, false, V16>(a, T_, sms, stream);
    return launch_vec<T, false, 1>(a, T_, sms, stream);
}

}  // namespace

cudaError_t launch_rope(const RopeTable& table, int dtype, int dims, bool interleaved, int vec_bytes,
                        const void* x, int64_t xt, int64_t xh, void* y, int64_t yt, int64_t yh,
                        const int32_t* positions, int T, int H, int sms, cudaStream_t stream) {
    RopeArgs a;
    a.x = x;
    a.y = y;
    a.positions = positions;
    a.xt = xt;
    a.xh = xh;
    a.yt = yt;
    a.yh = yh;
    a.T = T;
    a.H = H;
    a.dims = dims;
    a.heads_per_block = a.chunks = a.tokens_per_block = 1;
    a.table = table;
    switch (dtype) {
        case SPLASH_F16: return launch_typed<__half>(a, T, interleaved, vec_bytes, sms, stream);
        case SPLASH_F32: return launch_typed<float>(a, T, interleaved, vec_bytes, sms, stream);
        default: return launch_typed<__nv_bfloat16>(a, T, interleaved, vec_bytes, sms, stream);
    }
}

}  // namespace splash
