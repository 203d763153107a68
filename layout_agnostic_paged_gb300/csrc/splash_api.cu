// splash_api.cu -- the C ABI (include/splash.h): host-side validation, workspace
// sizing, per-device state and kernel launches.  No allocation, no stream
// synchronisation (except splash_workspace_status, which is documented to sync).
#include <stdlib.h>
#include <string.h>

#include <math.h>

#include <initializer_list>
#include <mutex>
#include <unordered_map>

#include "chunk.h"
#include "common.cuh"
#include "kernels.h"
#include "rope.cuh"
#include "rope_table.h"

namespace splash {
namespace {

std::mutex g_mu;
int g_sm_count[128];
std::unordered_map<uint64_t, int> g_smem_optin;  // (kernel ptr ^ device) -> bytes set

int current_device(int* dev) {
    return cudaGetDevice(dev) == cudaSuccess ? 0 : -1;
}

int sm_count(int dev) {
    if (dev < 0 || dev >= 128) return 0;
    std::lock_guard<std::mutex> lk(g_mu);
    if (g_sm_count[dev] == 0) {
        int n = 0;
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
        g_sm_count[dev] = n;
    }
    return g_sm_count[dev];
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

int validate_desc(const splash_attn_desc* d) {
    if (!d) return SPLASH_ERR_INVALID_ARG;
    if (d->num_reqs < 0 || d->num_heads <= 0 || d->num_pages < 0 || d->max_pages_per_req < 0)
        return SPLASH_ERR_INVALID_ARG;
    if (!(d->scale == d->scale)) return SPLASH_ERR_INVALID_ARG;  // NaN scale
    if (d->d_qk != kDqk || d->d_v != kDv) return SPLASH_ERR_UNSUPPORTED;
    const int P = d->page_size;
    if (P != 16 && P != 32 && P != 64 && P != 128) return SPLASH_ERR_UNSUPPORTED;
    if (int64_t(d->num_pages) * P >= (int64_t(1) << 31)) return SPLASH_ERR_UNSUPPORTED;
    if (int64_t(d->max_pages_per_req) * P >= (int64_t(1) << 31)) return SPLASH_ERR_UNSUPPORTED;
    if (int64_t(d->num_reqs) * d->num_heads >= (int64_t(1) << 31)) return SPLASH_ERR_UNSUPPORTED;
    return SPLASH_OK;
}

// A call without work leaves a workspace that reports no status bits (the first 16 bytes of either header).
constexpr size_t kHeadBytes = 16;
int clear_status(void* workspace, cudaStream_t stream) {
    return cudaMemsetAsync(workspace, 0, kHeadBytes, stream) == cudaSuccess ? SPLASH_OK : SPLASH_ERR_CUDA;
}

// Launch geometry of the decode kernel for a head slice of Hs heads.
struct Geometry {
    int head_groups;  // CTAs per CTA group (one per head group)
    int group_heads;  // heads per head group (the last group may have fewer)
    int num_groups;   // CTA groups G' (the tile sequence is cut into G' ranges)
};

// kv_group_heads > 0 forces head groups of that size (several KV heads: a group must
// stay within one KV head's query heads).
Geometry decode_geometry(int Hs, int sms, int kv_group_heads = 0) {
    Geometry g;
    if (kv_group_heads > 0) {
        g.group_heads = kv_group_heads;
        g.head_groups = (Hs + kv_group_heads - 1) / kv_group_heads;
        g.num_groups = sms / g.head_groups;
    } else {
        g.head_groups = (Hs + kTcMaxGroupHeads - 1) / kTcMaxGroupHeads;
        g.group_heads = (Hs + g.head_groups - 1) / g.head_groups;
        g.num_groups = sms / g.head_groups;  // one persistent CTA per SM
    }
    if (g.num_groups < 1) g.num_groups = 1;
    return g;
}

// cuTensorMapEncodeTiled through the runtime's driver entry point (no libcuda link).
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
    static EncodeTiledFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                             &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(p);
    });
    return fn;
}

// 2D bf16 map over [rows][576] with a {64, box_rows} box and the 128-byte swizzle.
bool encode_rows_576(CUtensorMap* m, const void* base, uint64_t rows, uint32_t box_rows) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[2] = {uint64_t(kDqk), rows};
    cuuint64_t strides[1] = {uint64_t(kDqk) * 2};
    cuuint32_t box[2] = {64u, box_rows};
    cuuint32_t es[2] = {1u, 1u};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box,
              es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// bf16 map over rows of 576 seen as [9 blocks][...][64], innermost first: box {64, rest...} and
// the 128-byte swizzle.  dims / strides (bytes) / box of the rank - 1 outer dims.
bool encode_blocks(CUtensorMap* m, const void* base, int rank, const uint64_t* dims, const uint64_t* strides,
                   const uint32_t* box) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    cuuint64_t d[5] = {64}, s[5];
    cuuint32_t b[5] = {64}, es[5] = {1, 1, 1, 1, 1};
    for (int i = 1; i < rank; ++i) {
        d[i] = dims[i - 1];
        s[i - 1] = strides[i - 1];
        b[i] = box[i - 1];
    }
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, cuuint32_t(rank), const_cast<void*>(base), d, s, b, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Pool map [9][rows][64] with a {64, box_rows, box_blocks} box.
bool encode_pool(CUtensorMap* m, const void* base, uint64_t rows, uint32_t box_rows, uint32_t box_blocks) {
    const uint64_t dims[2] = {rows, 9}, strides[2] = {uint64_t(kDqk) * 2, 128};
    const uint32_t box[2] = {box_rows, box_blocks};
    return encode_blocks(m, base, 3, dims, strides, box);
}

// The frequencies of a rope description as 64-bit fractions of a turn per position.
// Returns SPLASH_OK or the argument error.
int rope_turns(const splash_rope_desc* d, RopeTable* table) {
    // a model has one description: each thread keeps the table of the last one it saw (its 64 bytes)
    thread_local splash_rope_desc last;
    thread_local RopeTable last_table;
    thread_local bool valid = false;
    if (!d) return SPLASH_ERR_INVALID_ARG;
    if (valid && memcmp(d, &last, sizeof(last)) == 0) {
        *table = last_table;
        return SPLASH_OK;
    }
    valid = false;
    if (d->dims < 2 || d->dims % 2 != 0) return SPLASH_ERR_INVALID_ARG;
    if (d->dims > 2 * kMaxRopePairs) return SPLASH_ERR_UNSUPPORTED;
    if (d->scaling < SPLASH_ROPE_PLAIN || d->scaling > SPLASH_ROPE_YARN) return SPLASH_ERR_INVALID_ARG;
    if (!(d->base >= 1.0) || !isfinite(d->base) || !isfinite(d->amplitude)) return SPLASH_ERR_INVALID_ARG;
    if (d->scaling != SPLASH_ROPE_PLAIN && (!(d->factor >= 1.0) || !isfinite(d->factor)))
        return SPLASH_ERR_INVALID_ARG;
    if (d->scaling == SPLASH_ROPE_YARN &&
        (!(d->base > 1.0) || !(d->orig_ctx > 0) || !(d->beta_fast > 0) || !(d->beta_slow > 0) ||
         !isfinite(d->orig_ctx) || !isfinite(d->beta_fast) || !isfinite(d->beta_slow)))
        return SPLASH_ERR_INVALID_ARG;
    rope_table(*d, last_table.turns);
    last_table.amplitude = float(d->amplitude);
    last = *d;
    valid = true;
    *table = last_table;
    return SPLASH_OK;
}

}  // namespace

cudaError_t ensure_smem_optin(const void* kernel, int bytes) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t key = reinterpret_cast<uint64_t>(kernel) * 131u + uint64_t(dev);
    std::lock_guard<std::mutex> lk(g_mu);
    auto it = g_smem_optin.find(key);
    if (it != g_smem_optin.end() && it->second >= bytes) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) g_smem_optin[key] = bytes;
    return e;
}

}  // namespace splash

using namespace splash;

extern "C" {

const char* splash_status_string(int status) {
    switch (status) {
        case SPLASH_OK: return "SPLASH_OK";
        case SPLASH_ERR_INVALID_ARG: return "SPLASH_ERR_INVALID_ARG: invalid argument";
        case SPLASH_ERR_UNSUPPORTED: return "SPLASH_ERR_UNSUPPORTED: shape not supported";
        case SPLASH_ERR_WORKSPACE: return "SPLASH_ERR_WORKSPACE: workspace too small";
        case SPLASH_ERR_CUDA: return "SPLASH_ERR_CUDA: CUDA call failed";
        default: return "unknown splash status";
    }
}

size_t splash_decode_workspace_size(const splash_attn_desc* desc, int head_lo, int head_hi) {
    if (validate_desc(desc) != SPLASH_OK) return 0;
    if (head_lo < 0 || head_hi > desc->num_heads || head_lo >= head_hi) return 0;
    int dev = 0;
    if (current_device(&dev) != 0) return 0;
    const int sms = sm_count(dev);
    if (sms <= 0) return 0;
    const int Hs = head_hi - head_lo;
    const Geometry g = decode_geometry(Hs, sms);
    return WorkspaceLayout(desc->num_reqs, Hs, g.num_groups,
                           status_capacity(sms, g.num_groups * g.head_groups)).total;
}

int splash_decode_attn(const splash_attn_desc* desc, const void* q, const void* kv_pool,
                       const int32_t* block_table, const int32_t* ctx_lens, int head_lo,
                       int head_hi, int64_t tok_lo, int64_t tok_hi, float* out, float* lse,
                       void* workspace, size_t ws_bytes, splash_stream_t stream_) {
    return splash_decode_attn_ex(desc, nullptr, q, kv_pool, block_table, ctx_lens, head_lo, head_hi,
                                 tok_lo, tok_hi, out, lse, workspace, ws_bytes, stream_);
}

int splash_decode_attn_ex(const splash_attn_desc* desc, const splash_decode_ext* ext,
                          const void* q, const void* kv_pool, const int32_t* block_table,
                          const int32_t* ctx_lens, int head_lo, int head_hi, int64_t tok_lo,
                          int64_t tok_hi, float* out, float* lse, void* workspace,
                          size_t ws_bytes, splash_stream_t stream_) {
    int st = validate_desc(desc);
    if (st != SPLASH_OK) return st;
    if (head_lo < 0 || head_hi > desc->num_heads || head_lo >= head_hi) return SPLASH_ERR_INVALID_ARG;
    if (tok_lo < 0 || (tok_hi >= 0 && tok_hi < tok_lo)) return SPLASH_ERR_INVALID_ARG;
    if (tok_lo >= (int64_t(1) << 31)) tok_lo = (int64_t(1) << 31) - 1;   // beyond any context
    if (tok_hi >= (int64_t(1) << 31)) tok_hi = (int64_t(1) << 31) - 1;
    if (!workspace || !aligned(workspace, 256)) return SPLASH_ERR_INVALID_ARG;
    const int B = desc->num_reqs;
    const int32_t* lo_arr = ext ? ext->tok_lo : nullptr;
    const int32_t* hi_arr = ext ? ext->tok_hi : nullptr;
    const int32_t* rows = ext ? ext->rows : nullptr;
    const int num_rows = rows ? ext->num_rows : B;   // rows of q / block_table / ... / lse
    if (rows && num_rows < 1) return SPLASH_ERR_INVALID_ARG;
    const int max_sms = ext ? ext->max_sms : 0;
    if (max_sms < 0) return SPLASH_ERR_INVALID_ARG;
    const int kv_heads = ext && ext->num_kv_heads > 1 ? ext->num_kv_heads : 1;
    if (ext && ext->num_kv_heads < 0) return SPLASH_ERR_INVALID_ARG;
    int kv_group_heads = 0;   // head-group size forced by several KV heads
    if (kv_heads > 1) {
        if (desc->num_heads % kv_heads != 0) return SPLASH_ERR_INVALID_ARG;
        const int per_kv = desc->num_heads / kv_heads;
        if (per_kv > kTcMaxGroupHeads && per_kv % kTcMaxGroupHeads != 0) return SPLASH_ERR_UNSUPPORTED;
        kv_group_heads = per_kv < kTcMaxGroupHeads ? per_kv : kTcMaxGroupHeads;
        if (head_lo % kv_group_heads != 0) return SPLASH_ERR_UNSUPPORTED;
        if (int64_t(desc->num_pages) * kv_heads * desc->page_size >= (int64_t(1) << 31))
            return SPLASH_ERR_UNSUPPORTED;
    }
    if (!aligned(lo_arr, 4) || !aligned(hi_arr, 4) || !aligned(rows, 4)) return SPLASH_ERR_INVALID_ARG;
    if (B > 0) {
        if (!q || !block_table || !ctx_lens || !out || !lse) return SPLASH_ERR_INVALID_ARG;
        if (!aligned(q, 16) || !aligned(out, 16) || !aligned(lse, 4) || !aligned(block_table, 4) ||
            !aligned(ctx_lens, 4))
            return SPLASH_ERR_INVALID_ARG;
        if (desc->num_pages > 0 && (!kv_pool || !aligned(kv_pool, 16))) return SPLASH_ERR_INVALID_ARG;
    }
    int dev = 0;
    if (current_device(&dev) != 0) return SPLASH_ERR_CUDA;
    const int sms = sm_count(dev);
    if (sms <= 0) return SPLASH_ERR_CUDA;
    const int Hs = head_hi - head_lo;
    const Geometry g = decode_geometry(Hs, max_sms > 0 && max_sms < sms ? max_sms : sms,
                                       kv_group_heads);
    const int ctas = g.num_groups * g.head_groups;
    const int sts_cap = status_capacity(sms, ctas);
    const WorkspaceLayout lay(B, Hs, g.num_groups, sts_cap);
    if (ws_bytes < lay.total) return SPLASH_ERR_WORKSPACE;
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    if (B == 0) return clear_status(workspace, stream);

    DecodeArgs a;
    a.q = q;
    a.kv_pool = kv_pool;
    a.block_table = block_table;
    a.ctx_lens = ctx_lens;
    a.lo_arr = lo_arr;
    a.hi_arr = hi_arr;
    a.rows = rows;
    a.out = out;
    a.lse = lse;
    a.ws = workspace;
    a.tok_lo = tok_lo;
    a.tok_hi = tok_hi;
    a.B = B;
    a.H = desc->num_heads;
    a.P = desc->page_size;
    a.num_pages = desc->num_pages;
    a.max_pages = desc->max_pages_per_req;
    a.num_rows = num_rows;
    a.max_ctx = desc->max_pages_per_req * desc->page_size;
    a.head_lo = head_lo;
    a.Hs = Hs;
    a.num_groups = g.num_groups;
    a.ctas = ctas;
    a.sts_cap = sts_cap;
    a.kv_heads = kv_heads;
    a.q_per_kv = desc->num_heads / kv_heads;
    a.scale = desc->scale;
    {
        CUtensorMap mq, mkv;
        const uint32_t qbox = uint32_t(tc_pad_heads(g.group_heads));
        if (!encode_rows_576(&mq, q, uint64_t(num_rows) * desc->num_heads, qbox)) return SPLASH_ERR_CUDA;
        // an empty pool still needs a valid map: point it at the workspace (never read,
        // every page id is then out of range)
        const void* kv = desc->num_pages > 0 ? kv_pool : workspace;
        const uint64_t kv_rows = desc->num_pages > 0
                                     ? uint64_t(desc->num_pages) * kv_heads * desc->page_size
                                     : uint64_t(1);
        if (!encode_rows_576(&mkv, kv, kv_rows, uint32_t(desc->page_size))) return SPLASH_ERR_CUDA;
        if (launch_decode_tc(a, mq, mkv, g.head_groups, g.group_heads, stream) != cudaSuccess)
            return SPLASH_ERR_CUDA;
    }
    if (launch_combine(workspace, B, desc->num_heads, head_lo, Hs, g.num_groups, ctas, sts_cap, out,
                       lse, stream) != cudaSuccess)
        return SPLASH_ERR_CUDA;
    return SPLASH_OK;
}

int splash_lse_merge(const float* part_out, const float* part_lse, int S, int B, int H, int d_v,
                     float* out, float* lse, splash_stream_t stream) {
    if (S < 1 || B < 0 || H < 0 || d_v <= 0 || (d_v % 4) != 0) return SPLASH_ERR_INVALID_ARG;
    const int64_t rows = int64_t(B) * H;
    if (rows == 0) return SPLASH_OK;
    if (!part_out || !part_lse || !out || !lse) return SPLASH_ERR_INVALID_ARG;
    if (!aligned(part_out, 16) || !aligned(out, 16) || !aligned(part_lse, 4) || !aligned(lse, 4))
        return SPLASH_ERR_INVALID_ARG;
    // out must not overlap part_out
    const uintptr_t po0 = reinterpret_cast<uintptr_t>(part_out);
    const uintptr_t po1 = po0 + uintptr_t(S) * rows * d_v * sizeof(float);
    const uintptr_t o0 = reinterpret_cast<uintptr_t>(out);
    const uintptr_t o1 = o0 + uintptr_t(rows) * d_v * sizeof(float);
    if (o0 < po1 && po0 < o1) return SPLASH_ERR_INVALID_ARG;
    if (launch_lse_merge(part_out, part_lse, S, rows, d_v, out, lse,
                         reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess)
        return SPLASH_ERR_CUDA;
    return SPLASH_OK;
}

int splash_kv_migrate(const void* src_pool, void* dst_pool, size_t page_bytes,
                      const int32_t* src_ids, const int32_t* dst_ids, int n_pages,
                      int32_t src_num_pages, int32_t dst_num_pages, splash_stream_t stream) {
    if (n_pages < 0 || page_bytes == 0 || (page_bytes % 16) != 0 || src_num_pages < 0 ||
        dst_num_pages < 0)
        return SPLASH_ERR_INVALID_ARG;
    if (n_pages == 0) return SPLASH_OK;
    if (!src_pool || !dst_pool || !src_ids || !dst_ids) return SPLASH_ERR_INVALID_ARG;
    if (!aligned(src_pool, 16) || !aligned(dst_pool, 16) || !aligned(src_ids, 4) ||
        !aligned(dst_ids, 4))
        return SPLASH_ERR_INVALID_ARG;
    int dev = 0;
    if (current_device(&dev) != 0) return SPLASH_ERR_CUDA;
    const int sms = sm_count(dev);
    if (sms <= 0) return SPLASH_ERR_CUDA;
    if (launch_kv_migrate(src_pool, dst_pool, page_bytes, src_ids, dst_ids, n_pages, src_num_pages,
                          dst_num_pages, sms, reinterpret_cast<cudaStream_t>(stream)) !=
        cudaSuccess)
        return SPLASH_ERR_CUDA;
    return SPLASH_OK;
}

int splash_rope(const splash_rope_desc* rope, int dtype, const void* x, int64_t x_token_stride,
                int64_t x_head_stride, void* y, int64_t y_token_stride, int64_t y_head_stride,
                const int32_t* positions, int T, int H, splash_stream_t stream) {
    RopeTable table;
    const int st = rope_turns(rope, &table);
    if (st != SPLASH_OK) return st;
    if (dtype != SPLASH_BF16 && dtype != SPLASH_F16 && dtype != SPLASH_F32) return SPLASH_ERR_UNSUPPORTED;
    if (T < 0 || H < 0 || x_token_stride < 0 || x_head_stride < 0 || y_token_stride < 0 || y_head_stride < 0)
        return SPLASH_ERR_INVALID_ARG;
    if (T == 0 || H == 0) return SPLASH_OK;
    // rows of y may not share elements: the head rows of a token, then the tokens, or the other way round
    const int64_t d = rope->dims, yt = y_token_stride, yh = y_head_stride;
    if ((H > 1 && yh < d) || (T > 1 && yt < d)) return SPLASH_ERR_INVALID_ARG;
    if (T > 1 && H > 1 && yt < (H - 1) * yh + d && yh < (T - 1) * yt + d) return SPLASH_ERR_INVALID_ARG;
    if (!x || !y || !positions || !aligned(positions, 4)) return SPLASH_ERR_INVALID_ARG;
    const int size = dtype == SPLASH_F32 ? 4 : 2;
    if (!aligned(x, size) || !aligned(y, size)) return SPLASH_ERR_INVALID_ARG;
    if (int64_t(T) * H >= (int64_t(1) << 31)) return SPLASH_ERR_UNSUPPORTED;
    // the widest vectors that every head row allows: the interleaved layout takes them from the d dims, the
    // half layout from each half
    auto fits = [&](int bytes) {
        const int ve = bytes / size;
        return aligned(x, bytes) && aligned(y, bytes) && x_token_stride % ve == 0 && x_head_stride % ve == 0 &&
               yt % ve == 0 && yh % ve == 0 && (rope->interleaved ? d : d / 2) % ve == 0;
    };
    const int vec_bytes = fits(32) ? 32 : (fits(16) ? 16 : 0);
    int dev = 0;
    if (current_device(&dev) != 0) return SPLASH_ERR_CUDA;
    const int sms = sm_count(dev);
    if (sms <= 0) return SPLASH_ERR_CUDA;
    if (launch_rope(table, dtype, rope->dims, rope->interleaved != 0, vec_bytes, x, x_token_stride, x_head_stride, y, yt,
                    yh, positions, T, H, sms, reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess)
        return SPLASH_ERR_CUDA;
    return SPLASH_OK;
}

namespace {

// Checks one side's rows of splash_norm_rope and copies them; `vectors` stays true if 16-byte vectors fit them.
int norm_rows(const splash_norm_rows* r, const splash_norm_desc* norm, int size, int T, NormRows* out, bool* vectors) {
    if (r->heads < 0 || r->reserved != 0 || r->x_token_stride < 0 || r->x_head_stride < 0 || r->y_token_stride < 0 ||
        r->y_head_stride < 0)
        return SPLASH_ERR_INVALID_ARG;
    out->H = r->heads;
    if (r->heads == 0 || T == 0) return SPLASH_OK;
    // rows of y may not share elements: the head rows of a token, then the tokens, or the other way round
    const int64_t D = norm->width, yt = r->y_token_stride, yh = r->y_head_stride, H = r->heads;
    if ((H > 1 && yh < D) || (T > 1 && yt < D)) return SPLASH_ERR_INVALID_ARG;
    if (T > 1 && H > 1 && yt < (H - 1) * yh + D && yh < (T - 1) * yt + D) return SPLASH_ERR_INVALID_ARG;
    if (!r->x || !r->y || !aligned(r->x, size) || !aligned(r->y, size)) return SPLASH_ERR_INVALID_ARG;
    if (!aligned(r->weight, norm->weight_dtype == SPLASH_F32 ? 4 : 2)) return SPLASH_ERR_INVALID_ARG;
    out->x = r->x;
    out->y = r->y;
    out->weight = r->weight;
    out->xt = r->x_token_stride;
    out->xh = r->x_head_stride;
    out->yt = yt;
    out->yh = yh;
    const int ve = 16 / size;
    *vectors = *vectors && aligned(r->x, 16) && aligned(r->y, 16) && out->xt % ve == 0 && out->xh % ve == 0 &&
               yt % ve == 0 && yh % ve == 0;
    return SPLASH_OK;
}

}  // namespace

int splash_norm_rope(const splash_norm_desc* norm, const splash_rope_desc* rope, int dtype, const splash_norm_rows* q,
                     const splash_norm_rows* k, const int32_t* positions, int T, splash_stream_t stream) {
    if (!norm || !q) return SPLASH_ERR_INVALID_ARG;
    if (dtype != SPLASH_BF16 && dtype != SPLASH_F16 && dtype != SPLASH_F32) return SPLASH_ERR_UNSUPPORTED;
    if (norm->weight_dtype != SPLASH_BF16 && norm->weight_dtype != SPLASH_F16 && norm->weight_dtype != SPLASH_F32)
        return SPLASH_ERR_UNSUPPORTED;
    if (norm->width < 1 || norm->norm_dims < 1 || norm->norm_dims > norm->width || T < 0) return SPLASH_ERR_INVALID_ARG;
    if (norm->width > kMaxNormWidth) return SPLASH_ERR_UNSUPPORTED;
    if (!(norm->eps >= 0.f) || !isfinite(norm->eps) || !isfinite(norm->weight_offset)) return SPLASH_ERR_INVALID_ARG;
    NormArgs a = {};
    if (rope) {
        const int st = rope_turns(rope, &a.table);
        if (st != SPLASH_OK) return st;
        if (norm->rope_lo < 0 || norm->rope_lo > norm->width - rope->dims) return SPLASH_ERR_INVALID_ARG;
        a.rope_lo = norm->rope_lo;
        a.dims = rope->dims;
    }
    const int size = dtype == SPLASH_F32 ? 4 : 2, ve = 16 / size;
    // every part of a row, and each half of the rotated dims, is whole vectors
    bool vectors = norm->width % ve == 0 && norm->norm_dims % ve == 0 && a.rope_lo % ve == 0 && a.dims / 2 % ve == 0;
    int st = norm_rows(q, norm, size, T, &a.q, &vectors);
    if (st == SPLASH_OK && k) st = norm_rows(k, norm, size, T, &a.k, &vectors);
    if (st != SPLASH_OK) return st;
    if (int64_t(T) * (int64_t(a.q.H) + a.k.H) >= (int64_t(1) << 31)) return SPLASH_ERR_UNSUPPORTED;
    if (T == 0 || a.q.H + a.k.H == 0) return SPLASH_OK;
    if (rope && (!positions || !aligned(positions, 4))) return SPLASH_ERR_INVALID_ARG;
    a.positions = positions;
    a.T = T;
    a.width = norm->width;
    a.norm_dims = norm->norm_dims;
    a.weight_dtype = norm->weight_dtype;
    a.eps = norm->eps;
    a.weight_offset = norm->weight_offset;
    int dev = 0;
    if (current_device(&dev) != 0) return SPLASH_ERR_CUDA;
    const int sms = sm_count(dev);
    if (sms <= 0) return SPLASH_ERR_CUDA;
    if (launch_norm_rope(a, dtype, rope && rope->interleaved, vectors, sms, reinterpret_cast<cudaStream_t>(stream)) !=
        cudaSuccess)
        return SPLASH_ERR_CUDA;
    return SPLASH_OK;
}

int splash_kv_append(const splash_attn_desc* desc, const splash_rope_desc* rope, int format, const void* latent,
                     int64_t latent_stride, const void* k_rope, int64_t k_rope_stride, const int32_t* cu_q,
                     int total_q, const int32_t* block_table, const int32_t* ctx_lens, void* kv_pool,
                     splash_stream_t stream) {
    int st = validate_desc(desc);
    if (st != SPLASH_OK) return st;
    if (format != SPLASH_KV_BF16 && format != SPLASH_KV_MXFP8) return SPLASH_ERR_UNSUPPORTED;
    RopeTable wide;
    RopeTable32 table;
    if (rope) {
        st = rope_turns(rope, &wide);
        if (st != SPLASH_OK) return st;
        table.amplitude = wide.amplitude;
        if (rope->dims != kDqk - kDv) return SPLASH_ERR_UNSUPPORTED;
        for (int i = 0; i < 32; ++i) table.turns[i] = wide.turns[i];
    }
    if (total_q < 0 || latent_stride < 0 || k_rope_stride < 0) return SPLASH_ERR_INVALID_ARG;
    if (total_q == 0 || desc->num_reqs == 0 || desc->num_pages == 0 || desc->max_pages_per_req == 0) return SPLASH_OK;
    if (latent_stride % 8 != 0 || k_rope_stride % 2 != 0) return SPLASH_ERR_INVALID_ARG;
    if (!latent || !k_rope || !cu_q || !block_table || !ctx_lens || !kv_pool) return SPLASH_ERR_INVALID_ARG;
    if (!aligned(latent, 16) || !aligned(k_rope, 4) || !aligned(cu_q, 4) || !aligned(block_table, 4) ||
        !aligned(ctx_lens, 4) || !aligned(kv_pool, 16))
        return SPLASH_ERR_INVALID_ARG;
    if (launch_kv_append(rope ? &table : nullptr, rope ? rope->interleaved != 0 : true, format == SPLASH_KV_MXFP8,
                         latent, latent_stride, k_rope, k_rope_stride, cu_q, desc->num_reqs, total_q, block_table,
                         ctx_lens, desc->page_size, desc->num_pages, desc->max_pages_per_req, kv_pool,
                         reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess)
        return SPLASH_ERR_CUDA;
    return SPLASH_OK;
}

int splash_kv_unpack(const void* src_pool, void* dst_pool, int page_size, const int32_t* src_ids,
                     const int32_t* dst_ids, int n_pages, int32_t src_num_pages, int32_t dst_num_pages,
                     splash_stream_t stream) {
    if (n_pages < 0 || page_size <= 0 || src_num_pages < 0 || dst_num_pages < 0) return SPLASH_ERR_INVALID_ARG;
    if (n_pages == 0) return SPLASH_OK;
    if (!src_pool || !dst_pool || !src_ids || !dst_ids) return SPLASH_ERR_INVALID_ARG;
    if (!aligned(src_pool, 16) || !aligned(dst_pool, 16) || !aligned(src_ids, 4) || !aligned(dst_ids, 4))
        return SPLASH_ERR_INVALID_ARG;
    const uintptr_t s0 = reinterpret_cast<uintptr_t>(src_pool), d0 = reinterpret_cast<uintptr_t>(dst_pool);
    const uintptr_t s1 = s0 + uintptr_t(src_num_pages) * page_size * kMxRowBytes;
    const uintptr_t d1 = d0 + uintptr_t(dst_num_pages) * page_size * (kDqk * 2);
    if (s0 < d1 && d0 < s1) return SPLASH_ERR_INVALID_ARG;
    int dev = 0;
    if (current_device(&dev) != 0) return SPLASH_ERR_CUDA;
    const int sms = sm_count(dev);
    if (sms <= 0) return SPLASH_ERR_CUDA;
    if (launch_kv_unpack(src_pool, dst_pool, page_size, src_ids, dst_ids, n_pages, src_num_pages, dst_num_pages, sms,
                         reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess)
        return SPLASH_ERR_CUDA;
    return SPLASH_OK;
}

namespace {

int page_log(int P) { return P == 16 ? 4 : (P == 32 ? 5 : (P == 64 ? 6 : 7)); }

}  // namespace

namespace {

int batch_shape_error(int reqs, int page_size, int num_pages, int max_pages) {
    const splash_attn_desc d = {reqs, 1, kDqk, kDv, page_size, num_pages, max_pages, 1.f};
    return validate_desc(&d);
}

}  // namespace

int splash_batch_tables(const splash_batch* b, splash_stream_t stream) {
    if (!b) return SPLASH_ERR_INVALID_ARG;
    const int st = batch_shape_error(b->num_reqs, b->page_size, b->num_pages, b->max_pages_per_req);
    if (st != SPLASH_OK) return st;
    if (b->total_q < 0 || b->reserved != 0) return SPLASH_ERR_INVALID_ARG;
    if (b->total_q > 1 << 30) return SPLASH_ERR_UNSUPPORTED;
    if (!b->cu_q || !b->left || !b->free_count) return SPLASH_ERR_INVALID_ARG;
    if (b->num_reqs > 0 && (!b->past_lens || !b->new_lens || !b->ctx_lens)) return SPLASH_ERR_INVALID_ARG;
    if (b->num_reqs > 0 && b->max_pages_per_req > 0 && !b->block_table) return SPLASH_ERR_INVALID_ARG;
    if ((b->num_pages > 0 && !b->free_pages) || (b->total_q > 0 && (!b->positions || !b->slots)))
        return SPLASH_ERR_INVALID_ARG;
    for (const int32_t* p : {b->past_lens, b->new_lens, b->free_pages, b->free_count,
                             static_cast<const int32_t*>(b->block_table), static_cast<const int32_t*>(b->cu_q),
                             static_cast<const int32_t*>(b->ctx_lens), static_cast<const int32_t*>(b->positions),
                             static_cast<const int32_t*>(b->slots), static_cast<const int32_t*>(b->left)})
        if (!aligned(p, 4)) return SPLASH_ERR_INVALID_ARG;
    BatchTablesArgs a = {};
    a.past = b->past_lens;
    a.fresh = b->new_lens;
    a.table = b->block_table;
    a.free_pages = b->free_pages;
    a.free_count = b->free_count;
    a.cu = b->cu_q;
    a.ctx = b->ctx_lens;
    a.positions = b->positions;
    a.slots = b->slots;
    a.left = b->left;
    a.B = b->num_reqs;
    a.total_q = b->total_q;
    a.P_log = page_log(b->page_size);
    a.num_pages = b->num_pages;
    a.max_pages = b->max_pages_per_req;
    a.wide = aligned(b->positions, 16) && aligned(b->slots, 16);
    if (launch_batch_tables(a, reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess) return SPLASH_ERR_CUDA;
    return SPLASH_OK;
}

int splash_batch_release(const splash_batch_drop* d, splash_stream_t stream) {
    if (!d) return SPLASH_ERR_INVALID_ARG;
    const int st = batch_shape_error(d->num_reqs, d->page_size, d->num_pages, d->max_pages_per_req);
    if (st != SPLASH_OK) return st;
    if (d->window < 0 || d->sinks < 0) return SPLASH_ERR_INVALID_ARG;
    if (int64_t(d->num_reqs) * d->max_pages_per_req >= (int64_t(1) << 31)) return SPLASH_ERR_UNSUPPORTED;
    if (d->num_reqs == 0 || d->max_pages_per_req == 0) return SPLASH_OK;
    if (!d->ctx_lens || !d->block_table || !d->free_count || (d->num_pages > 0 && !d->free_pages))
        return SPLASH_ERR_INVALID_ARG;
    if (!aligned(d->ctx_lens, 4) || !aligned(d->keep_lens, 4) || !aligned(d->block_table, 4) ||
        !aligned(d->free_pages, 4) || !aligned(d->free_count, 4))
        return SPLASH_ERR_INVALID_ARG;
    BatchReleaseArgs a = {};
    a.ctx = d->ctx_lens;
    a.keep = d->keep_lens;
    a.table = d->block_table;
    a.free_pages = d->free_pages;
    a.free_count = d->free_count;
    a.B = d->num_reqs;
    a.P_log = page_log(d->page_size);
    a.num_pages = d->num_pages;
    a.max_pages = d->max_pages_per_req;
    a.window = d->window;
    a.sinks = d->sinks;
    if (launch_batch_release(a, reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess) return SPLASH_ERR_CUDA;
    return SPLASH_OK;
}

namespace {

// Positions rounded up to whole tiles, and a tile ahead, stay below 2^31.
bool chunk_too_long(const splash_attn_desc* d) {
    return int64_t(d->max_pages_per_req) * d->page_size > (int64_t(1) << 31) - 1024;
}

int chunk_ext_error(const splash_chunk_ext* ext) {
    if (!ext) return SPLASH_OK;
    if (ext->window < 0 || ext->sinks < 0 || ext->num_groups < 0 || ext->reserved != 0) return SPLASH_ERR_INVALID_ARG;
    return ext->num_groups > kChunkMaxGroups || (ext->num_groups > 0 && ext->window > 0) ? SPLASH_ERR_UNSUPPORTED : SPLASH_OK;
}

// Shape, tiling and workspace layout of a chunk call; returns its workspace bytes, 0 for a bad shape.
size_t chunk_shape(const splash_attn_desc* desc, const splash_chunk_ext* ext, int total_q, int head_lo, int head_hi,
                   ChunkArgs* a, int* sms) {
    if (validate_desc(desc) != SPLASH_OK || chunk_too_long(desc) || total_q < 0) return 0;
    if (head_lo < 0 || head_hi > desc->num_heads || head_lo >= head_hi) return 0;
    int dev = 0;
    if (current_device(&dev) != 0) return 0;
    *sms = sm_count(dev);
    if (*sms < 2) return 0;
    a->B = desc->num_reqs;
    a->total_q = total_q;
    a->H = desc->num_heads;
    a->head_lo = head_lo;
    a->Hs = head_hi - head_lo;
    a->P = desc->page_size;
    a->P_log = page_log(a->P);
    a->num_pages = desc->num_pages;
    a->max_pages = desc->max_pages_per_req;
    a->max_ctx = desc->max_pages_per_req * desc->page_size;
    a->past_row = desc->num_pages > 0 ? desc->num_pages * desc->page_size : 1;
    a->pairs = *sms / 2;
    a->by_pairs = fast_div(a->pairs);
    a->tile = chunk_tiling(a->H, a->Hs);
    a->scale = desc->scale;
    if (ext) {
        // a window that reaches back from the last position to the first hides nothing, and requests whose every
        // token fills a pair's rows have nothing to share
        if (ext->window > 0 && ext->window < a->max_ctx) {
            a->mode = kChunkWindow;
            a->window = ext->window;
            a->sinks = min(ext->sinks, a->max_ctx);
        } else if (ext->num_groups > 0 && a->tile.pair_tokens() > 1) {
            a->mode = kChunkGroups;
            a->groups = ext->num_groups;
            a->cu_groups = ext->cu_groups;
            a->prefix_lens = ext->prefix_lens;
        }
    }
    a->early = max(1, 2 * a->pairs * kEarlyUnits / max(1, a->mode == kChunkGroups ? a->groups : a->B));
    a->by_early = fast_div(a->early);
    const size_t bytes = chunk_layout(*a);
    if (a->cap_items >= (int64_t(1) << 31)) return 0;
    return bytes;
}

}  // namespace

size_t splash_chunk_workspace_size(const splash_attn_desc* desc, int total_q, int head_lo, int head_hi) {
    return splash_chunk_workspace_size_ex(desc, nullptr, total_q, head_lo, head_hi);
}

size_t splash_chunk_workspace_size_ex(const splash_attn_desc* desc, const splash_chunk_ext* ext, int total_q, int head_lo,
                                      int head_hi) {
    if (chunk_ext_error(ext) != SPLASH_OK) return 0;
    ChunkArgs a = {};
    int sms = 0;
    return chunk_shape(desc, ext, total_q, head_lo, head_hi, &a, &sms);
}

int splash_chunk_attn(const splash_attn_desc* desc, const void* q, const void* kv_pool, const int32_t* cu_q,
                      int total_q, const int32_t* block_table, const int32_t* ctx_lens, int head_lo, int head_hi,
                      int64_t tok_lo, int64_t tok_hi, int out_dtype, void* out, float* lse, void* workspace,
                      size_t ws_bytes, splash_stream_t stream) {
    return splash_chunk_attn_ex(desc, nullptr, q, kv_pool, cu_q, total_q, block_table, ctx_lens, head_lo, head_hi, tok_lo,
                                tok_hi, out_dtype, out, lse, workspace, ws_bytes, stream);
}

int splash_chunk_attn_ex(const splash_attn_desc* desc, const splash_chunk_ext* ext, const void* q, const void* kv_pool,
                         const int32_t* cu_q, int total_q, const int32_t* block_table, const int32_t* ctx_lens, int head_lo,
                         int head_hi, int64_t tok_lo, int64_t tok_hi, int out_dtype, void* out, float* lse, void* workspace,
                         size_t ws_bytes, splash_stream_t stream_) {
    int st = validate_desc(desc);
    if (st == SPLASH_OK) st = chunk_ext_error(ext);
    if (st != SPLASH_OK) return st;
    if (total_q < 0 || head_lo < 0 || head_hi > desc->num_heads || head_lo >= head_hi) return SPLASH_ERR_INVALID_ARG;
    if (tok_lo < 0 || (tok_hi >= 0 && tok_hi < tok_lo)) return SPLASH_ERR_INVALID_ARG;
    if (out_dtype != SPLASH_BF16 && out_dtype != SPLASH_F32) return SPLASH_ERR_UNSUPPORTED;
    if (int64_t(total_q) * desc->num_heads >= (int64_t(1) << 31) || chunk_too_long(desc)) return SPLASH_ERR_UNSUPPORTED;
    if (!workspace || !aligned(workspace, 256)) return SPLASH_ERR_INVALID_ARG;
    const bool work = desc->num_reqs > 0 && total_q > 0;
    if (work) {
        if (!q || !cu_q || !block_table || !ctx_lens || !out || !lse) return SPLASH_ERR_INVALID_ARG;
        if (!aligned(q, 16) || !aligned(out, 32) || !aligned(lse, 4) || !aligned(cu_q, 4) ||
            !aligned(block_table, 4) || !aligned(ctx_lens, 4))
            return SPLASH_ERR_INVALID_ARG;
        if (desc->num_pages > 0 && (!kv_pool || !aligned(kv_pool, 16))) return SPLASH_ERR_INVALID_ARG;
        if (ext && ext->num_groups > 0 && (!ext->cu_groups || !ext->prefix_lens || !aligned(ext->cu_groups, 4) ||
                                           !aligned(ext->prefix_lens, 4)))
            return SPLASH_ERR_INVALID_ARG;
    }
    ChunkArgs a = {};
    int sms = 0;
    const size_t need = chunk_shape(desc, ext, total_q, head_lo, head_hi, &a, &sms);
    if (need == 0) return sms < 2 ? SPLASH_ERR_CUDA : SPLASH_ERR_UNSUPPORTED;
    if (ws_bytes < need) return SPLASH_ERR_WORKSPACE;
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    if (!work) return clear_status(workspace, stream);

    const int64_t most = (int64_t(1) << 31) - 1;
    a.kv = static_cast<const uint8_t*>(kv_pool);
    a.cu_q = cu_q;
    a.block_table = block_table;
    a.ctx_lens = ctx_lens;
    a.out = out;
    a.lse = lse;
    a.ws = static_cast<uint8_t*>(workspace);
    a.tok_lo = int(tok_lo < most ? tok_lo : most);
    a.tok_hi = int(tok_hi >= 0 && tok_hi < most ? tok_hi : most);
    if (a.mode == kChunkWindow)
        a.sink_blocks = max(0, (a.sinks + kChunkRows - 1) / kChunkRows - a.tok_lo / kChunkRows);
    a.out_f32 = out_dtype == SPLASH_F32;
    ChunkMaps maps;
    const uint64_t row = uint64_t(kDqk) * 2;
    const uint64_t qd[3] = {a.tile.flat ? uint64_t(a.H) * total_q : uint64_t(a.H), a.tile.flat ? uint64_t(1) : uint64_t(total_q), 9};
    const uint64_t qs[3] = {row, row * a.H, 128};
    const uint32_t qb[3] = {a.tile.flat ? uint32_t(kChunkRows) : uint32_t(a.tile.heads), a.tile.flat ? 1u : uint32_t(a.tile.tokens), 1};
    // an empty pool still needs a valid map: one row of the workspace, which no copy reads
    const void* kv = desc->num_pages > 0 ? kv_pool : workspace;
    const uint64_t rows = uint64_t(a.past_row);
    const uint32_t R = uint32_t(a.P < kChunkRows ? a.P : kChunkRows);
    bool ok = encode_blocks(&maps.q, q, 4, qd, qs, qb) &&
              encode_pool(&maps.k, kv, rows, R, R == uint32_t(kChunkRows) ? kChunkKBlocks : 1) &&
              encode_pool(&maps.v, kv, rows, R, 4);
    for (int i = 0; ok && i < 3; ++i) ok = encode_pool(&maps.rows[i], kv, rows, 1u << (2 * i), 1);
    if (!ok) return SPLASH_ERR_CUDA;
    if (launch_chunk_attn(a, maps, stream) != cudaSuccess || launch_chunk_combine(a, sms, stream) != cudaSuccess)
        return SPLASH_ERR_CUDA;
    return SPLASH_OK;
}

int splash_workspace_status(const void* workspace, uint32_t* flags, splash_stream_t stream) {
    if (!workspace || !flags) return SPLASH_ERR_INVALID_ARG;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (cudaStreamSynchronize(s) != cudaSuccess) return SPLASH_ERR_CUDA;
    uint32_t head[kHeadBytes / 4];
    if (cudaMemcpy(head, workspace, sizeof(head), cudaMemcpyDeviceToHost) != cudaSuccess) return SPLASH_ERR_CUDA;
    uint32_t bits = head[0];
    if (head[1] == kChunkMagic) {   // a chunk call: its CTAs' words hold the rest
        int dev = 0;
        if (current_device(&dev) != 0) return SPLASH_ERR_CUDA;
        constexpr uint32_t kMost = 1024;
        uint32_t words[kMost];
        const uint32_t sms = uint32_t(sm_count(dev));            // a word per CTA, a CTA per SM at most
        const uint32_t n = min(head[3], min(sms, kMost));
        if (cudaMemcpy(words, static_cast<const uint8_t*>(workspace) + kChunkWordsOff, n * sizeof(uint32_t),
                       cudaMemcpyDeviceToHost) != cudaSuccess)
            return SPLASH_ERR_CUDA;
        for (uint32_t i = 0; i < n; ++i) bits |= words[i];
    }
    *flags = bits;
    return SPLASH_OK;
}

}  // extern "C"
