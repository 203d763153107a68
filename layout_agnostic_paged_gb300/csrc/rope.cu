// rope.cu -- splash_rope: rotary positions of head rows, in place or from one strided
// tensor to another.
//
// HBM-bound: every rotated element is read and written once.  A block owns one token and a
// run of its heads.  The cos / sin of the token's d / 2 pairs are computed once per block
// into shared memory, behind the block's first loads, and serve all of its heads.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"
#include "kernels.h"
#include "rope.cuh"

namespace splash {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeUnroll = 4;   // work items whose loads a thread has in flight

__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ void from_f32(__nv_bfloat16& d, float v) { d = __float2bfloat16_rn(v); }
__device__ __forceinline__ void from_f32(__half& d, float v) { d = __float2half_rn(v); }
__device__ __forceinline__ void from_f32(float& d, float v) { d = v; }

template <typename T, int N>
struct alignas(N * sizeof(T)) Vec {
    T v[N];
};

struct RopeArgs {
    const void* x;
    void* y;
    const int32_t* positions;
    int64_t xt, xh, yt, yh;   // strides in elements
    int H, heads_per_block, dims;
    int chunks;               // runs of heads per token
    RopeTable table;
};

// VE elements a vector: 16 bytes, or 1 where alignment or d forbids it.  A work item is
// VE / 2 pairs of one head in the interleaved layout (at least one pair) and VE pairs in the half layout.
template <typename T, bool INTER, int VE>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeArgs a) {
    constexpr int W = INTER && VE == 1 ? 2 : VE;       // elements of one load group
    constexpr int NP = INTER ? W / 2 : VE;             // pairs of a work item
    using V = Vec<T, VE>;
    __shared__ float2 cs[kMaxRopePairs];
    pdl_wait();
    const int t = blockIdx.x / a.chunks;
    const int h0 = (blockIdx.x % a.chunks) * a.heads_per_block;
    const int nh = min(a.heads_per_block, a.H - h0);
    const int half = a.dims >> 1;
    const int per_head = half / NP;                    // work items of a head
    const int items = nh * per_head;
    const T* x = static_cast<const T*>(a.x) + int64_t(t) * a.xt + int64_t(h0) * a.xh;
    T* y = static_cast<T*>(a.y) + int64_t(t) * a.yt + int64_t(h0) * a.yh;
    bool ready = false;
    for (int i0 = threadIdx.x; !ready || i0 < items; i0 += kRopeThreads * kRopeUnroll) {
        T in[kRopeUnroll][2 * NP];                     // the pairs' elements, as loaded
#pragma unroll
        for (int u = 0; u < kRopeUnroll; ++u) {
            const int i = i0 + u * kRopeThreads;
            if (i < items) {
                const int h = i / per_head, k = i % per_head;
                const T* p = x + int64_t(h) * a.xh + (INTER ? k * 2 * NP : k * NP);
                if (INTER) {
#pragma unroll
                    for (int e = 0; e < 2 * NP; e += VE) *reinterpret_cast<V*>(&in[u][e]) = *reinterpret_cast<const V*>(p + e);
                } else {
                    *reinterpret_cast<V*>(&in[u][0]) = *reinterpret_cast<const V*>(p);
                    *reinterpret_cast<V*>(&in[u][NP]) = *reinterpret_cast<const V*>(p + half);
                }
            }
        }
        if (!ready) {
            const int32_t pos = a.positions[t];
            for (int j = threadIdx.x; j < half; j += kRopeThreads)
                cs[j] = rope_cos_sin(a.table.turns[j], pos, a.table.amplitude);
            __syncthreads();
            ready = true;
        }
#pragma unroll
        for (int u = 0; u < kRopeUnroll; ++u) {
            const int i = i0 + u * kRopeThreads;
            if (i < items) {
                const int h = i / per_head, k = i % per_head;
                T* p = y + int64_t(h) * a.yh + (INTER ? k * 2 * NP : k * NP);
#pragma unroll
                for (int e = 0; e < NP; ++e) {
                    T& ea = in[u][INTER ? 2 * e : e];
                    T& eb = in[u][INTER ? 2 * e + 1 : NP + e];
                    const float2 r = rope_rotate(to_f32(ea), to_f32(eb), cs[k * NP + e]);
                    from_f32(ea, r.x);
                    from_f32(eb, r.y);
                }
                if (INTER) {
#pragma unroll
                    for (int e = 0; e < 2 * NP; e += VE) *reinterpret_cast<V*>(p + e) = *reinterpret_cast<const V*>(&in[u][e]);
                } else {
                    *reinterpret_cast<V*>(p) = *reinterpret_cast<const V*>(&in[u][0]);
                    *reinterpret_cast<V*>(p + half) = *reinterpret_cast<const V*>(&in[u][NP]);
                }
            }
        }
    }
}

template <typename T>
cudaError_t launch_typed(RopeArgs& a, int T_, bool inter, bool vec, int sms, cudaStream_t stream) {
    constexpr int VE = 16 / int(sizeof(T));
    const int np = vec ? (inter ? VE / 2 : VE) : 1;
    const int per_head = (a.dims / 2) / np;
    // One pass of a block covers kRopeThreads * kRopeUnroll work items.  Fewer heads a block
    // when the tokens alone would not fill the GPU.
    int heads = (kRopeThreads * kRopeUnroll) / per_head;
    if (heads < 1) heads = 1;
    const int64_t want = int64_t(sms) * 4;
    while (heads > 1 && int64_t(T_) * ((a.H + heads - 1) / heads) < want &&
           int64_t(heads) * per_head > kRopeThreads)
        heads = (heads + 1) / 2;
    if (heads > a.H) heads = a.H;
    a.heads_per_block = heads;
    a.chunks = (a.H + heads - 1) / heads;
    const int64_t grid = int64_t(T_) * a.chunks;
    const dim3 g(static_cast<unsigned>(grid)), b(kRopeThreads);
    if (inter) {
        if (vec) return launch_pdl(rope_kernel<T, true, VE>, g, b, 0, stream, a);
        return launch_pdl(rope_kernel<T, true, 1>, g, b, 0, stream, a);
    }
    if (vec) return launch_pdl(rope_kernel<T, false, VE>, g, b, 0, stream, a);
    return launch_pdl(rope_kernel<T, false, 1>, g, b, 0, stream, a);
}

}  // namespace

cudaError_t launch_rope(const RopeTable& table, int dtype, int dims, bool interleaved, bool vec,
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
    a.H = H;
    a.dims = dims;
    a.heads_per_block = a.chunks = 1;
    a.table = table;
    switch (dtype) {
        case SPLASH_F16: return launch_typed<__half>(a, T, interleaved, vec, sms, stream);
        case SPLASH_F32: return launch_typed<float>(a, T, interleaved, vec, sms, stream);
        default: return launch_typed<__nv_bfloat16>(a, T, interleaved, vec, sms, stream);
    }
}

}  // namespace splash
