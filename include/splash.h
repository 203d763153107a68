/*
 * splash.h -- C ABI of the GB300 (sm_103a) paged MLA decode-attention hot path.
 *
 * Method: "SPLASH: Switching Parallel Layouts of Attention with Seamless Handoff
 * for LLM Serving".
 *   Abstract -- with few or no KV heads (MLA: one shared latent KV head), where a
 *     request's KV cache lives is decoupled from how attention weights are
 *     sharded, so the four attention layouts (TP, CP, DP-attention and DOP)
 *     differ only in who owns weights and cache; a layout switch moves the state
 *     that is not yet in place and hands off at a batch boundary.
 *   Appendix, Table 2 -- per-layout ownership: TP reads every request's history
 *     for a share of the heads; CP reads a B/T share of every request's tokens
 *     ("ideal token partitioning"); DP-attention and DOP own whole requests.
 *
 * One call of splash_decode_attn computes any of those ownership slices on one
 * GPU: a head range [head_lo, head_hi) (TP / DOP shard), a token range
 * [tok_lo, tok_hi) returning partial output plus log-sum-exp (CP), or whole
 * requests (DP-attention / DOP: pass only the owned requests' rows).
 * splash_lse_merge combines CP partials; splash_kv_migrate moves KV pages
 * between block pools for a handoff.
 *
 * Conventions shared by every entry point
 *   - Every pointer argument is DEVICE memory owned by the caller, unless stated
 *     otherwise.  The library allocates no device memory, keeps no reference to
 *     any buffer after the call returns, and never synchronises the stream.
 *   - Work is enqueued on `stream` (a cudaStream_t; NULL is the legacy default
 *     stream).  Buffers must stay alive until that work completes.
 *   - Arguments are validated on the host before anything is enqueued; a call
 *     that returns an error has enqueued nothing.  Launch failures are reported
 *     as SPLASH_ERR_CUDA (the CUDA error is not cleared from the device).
 *   - Calls are thread-safe; the only library state is a per-device cache of
 *     the SM count and of the dynamic shared memory opt-in, and each thread's
 *     frequency table of the last splash_rope_desc it passed (compared by value).
 *   - The calling thread's current CUDA device must be the device that owns
 *     the pointers and the stream.
 */
#ifndef SPLASH_H_
#define SPLASH_H_

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define SPLASH_API __attribute__((visibility("default")))
#else
#define SPLASH_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

/* ABI-identical to cudaStream_t / CUstream. */
typedef struct CUstream_st* splash_stream_t;

typedef enum {
    SPLASH_OK = 0,
    SPLASH_ERR_INVALID_ARG = -1, /* null pointer, bad range, misaligned pointer   */
    SPLASH_ERR_UNSUPPORTED = -2, /* shape outside what the kernels implement      */
    SPLASH_ERR_WORKSPACE = -3,   /* workspace smaller than the size query returns */
    SPLASH_ERR_CUDA = -4         /* a CUDA runtime / driver call failed           */
} splash_status;

/* Bits of the device-side status word (see splash_workspace_status). */
enum {
    SPLASH_DEVICE_TIMEOUT = 1u << 0,   /* a bounded wait gave up; outputs are invalid  */
    SPLASH_DEVICE_BAD_INPUT = 1u << 1  /* a needed page id or a context length was out of range */
};

/*
 * Shape of one paged decode batch.
 *   num_reqs          B, requests in this call (rows of q, block_table, ctx_lens, out, lse)
 *   num_heads         H, query heads per request (rows per request in q / out / lse)
 *   d_qk              key / query width: must be 576 (512 latent + 64 rope dims)
 *   d_v               value width: must be 512 (values are the latent prefix of the key)
 *   page_size         P, tokens per KV page: 16, 32, 64 or 128
 *   num_pages         pages in kv_pool
 *   max_pages_per_req row stride of block_table (entries per request)
 *   scale             softmax temperature applied to q.k (e.g. 1/sqrt(192)), fp32
 */
typedef struct {
    int32_t num_reqs;
    int32_t num_heads;
    int32_t d_qk;
    int32_t d_v;
    int32_t page_size;
    int32_t num_pages;
    int32_t max_pages_per_req;
    float scale;
} splash_attn_desc;

/*
 * Bytes of device workspace splash_decode_attn needs for this shape and head
 * range on the current device (it depends on B, head_hi - head_lo and the
 * device's SM count, not on the context lengths).  Returns 0 when the shape is
 * invalid or unsupported.
 */
SPLASH_API size_t splash_decode_workspace_size(const splash_attn_desc* desc, int head_lo, int head_hi);

/*
 * Paged decode attention for one ownership slice (Abstract; Appendix, Table 2).
 *
 * For every request r < B and head h in [head_lo, head_hi), over the token set
 *   T_r = [tok_lo, min(tok_hi < 0 ? ctx_lens[r] : tok_hi, ctx_lens[r]))
 * with key k_t = kv_pool[block_table[r][t / P]][t % P][0:576] and value
 * v_t = k_t[0:512]:
 *   s_t = scale * q[r][h] . k_t
 *   out[r][h][j] = sum_t exp(s_t - m) v_t[j] / sum_t exp(s_t - m)
 *   lse[r][h]    = m + ln sum_t exp(s_t - m)          (natural log, m = max_t s_t)
 * An empty T_r gives out = 0 and lse = -inf.  A token range [tok_lo, tok_hi)
 * that is a share of the context yields the CP partial (out normalised over the
 * share, lse of the share) that splash_lse_merge combines.
 *
 *   q           bf16 [B][H][576], 16-byte aligned rows (contiguous)
 *   kv_pool     bf16 [num_pages][P][576], 16-byte aligned, contiguous
 *   block_table int32 [B][max_pages_per_req]; entries for pages at or beyond
 *               ceil(ctx_len / P) are never read
 *   ctx_lens    int32 [B], 0 <= ctx_lens[r] <= max_pages_per_req * P
 *   head_lo/hi  0 <= head_lo < head_hi <= H
 *   tok_lo      >= 0;  tok_hi < 0 means "to the end of each context", else tok_hi >= tok_lo
 *   out         fp32 [B][H][512]: only rows [head_lo, head_hi) are written
 *   lse         fp32 [B][H]:      only rows [head_lo, head_hi) are written
 *   workspace   >= splash_decode_workspace_size(...) bytes, 256-byte aligned; reused
 *               across calls on one stream; must not be shared by calls that may
 *               overlap on the device
 * Slot contents of KV pages beyond ctx_len (tail slots, unused pages) may hold
 * any bits, NaN included: they never reach an output.  A block-table id outside
 * [0, num_pages) for a needed page is not read: that page's tokens are left out of
 * T_r.  A context length outside [0, max_pages_per_req * P] is clamped into it.
 * Both set SPLASH_DEVICE_BAD_INPUT.
 * Returns SPLASH_OK or a splash_status error (nothing enqueued on error).
 */
SPLASH_API int splash_decode_attn(const splash_attn_desc* desc, const void* q, const void* kv_pool,
                       const int32_t* block_table, const int32_t* ctx_lens, int head_lo,
                       int head_hi, int64_t tok_lo, int64_t tok_hi, float* out, float* lse,
                       void* workspace, size_t ws_bytes, splash_stream_t stream);

/*
 * Per-request token ranges and storage rows for splash_decode_attn_ex.  Every
 * pointer may be NULL, and NULL restores the splash_decode_attn behaviour for
 * that field.
 *   tok_lo, tok_hi  int32 [B] device: request r's token set is
 *                   [tok_lo[r], min(tok_hi[r] < 0 ? ctx_len : tok_hi[r], ctx_len)),
 *                   for CP with an uneven share per request (the "ideal token
 *                   partitioning" of Appendix, Table 2, for ragged contexts).  A NULL
 *                   array uses the call's scalar for every request.  A negative
 *                   tok_lo[r] is bad input: it is taken as 0 and sets
 *                   SPLASH_DEVICE_BAD_INPUT.
 *   rows            int32 [B] device: request r of the call reads row rows[r] of q,
 *                   block_table and ctx_lens and writes row rows[r] of out and lse.
 *                   Those arrays then have num_rows rows.  This lets a DP-attention /
 *                   DOP owner decode its subset of a batch in place.  The rows must be
 *                   distinct.  A row outside [0, num_rows) is bad input: nothing is
 *                   read or written for that request, and SPLASH_DEVICE_BAD_INPUT is set.
 *   num_rows        rows of q / block_table / ctx_lens / out / lse when rows != NULL
 *                   (>= 1); ignored otherwise (the arrays then have B rows).
 *   max_sms         at most this many SMs run the call's persistent decode grid (0: all
 *                   of them), leaving the rest to work on other streams, e.g. a
 *                   background splash_kv_migrate of a layout handoff.  Must be >= 0.
 *   num_kv_heads    KV heads per token, Hkv (0 or 1: the one shared latent head).  With
 *                   Hkv > 1 (grouped-query attention, the Abstract's "few KV heads") the
 *                   pool is bf16 [num_pages][Hkv][P][576] and query head h reads KV head
 *                   h / (H / Hkv).  H must be a multiple of Hkv.  H / Hkv must be at most 64
 *                   or a multiple of 64, and head_lo a multiple of min(H / Hkv, 64); other
 *                   shapes return SPLASH_ERR_UNSUPPORTED.
 */
typedef struct {
    const int32_t* tok_lo;
    const int32_t* tok_hi;
    const int32_t* rows;
    int32_t num_rows;
    int32_t max_sms;
    int32_t num_kv_heads;
} splash_decode_ext;

/*
 * splash_decode_attn with per-request token ranges and storage rows.
 * `ext` may be NULL.  desc->num_reqs is B, the number of requests in the call
 * and the length of the ext arrays.  The scalars tok_lo / tok_hi apply to every
 * request whose array is NULL, and are validated as in splash_decode_attn.  The
 * workspace size is splash_decode_workspace_size(desc, head_lo, head_hi), as
 * for splash_decode_attn.  Alignment: the ext arrays 4 bytes.  Otherwise the
 * same arguments, results and errors as splash_decode_attn.
 */
SPLASH_API int splash_decode_attn_ex(const splash_attn_desc* desc, const splash_decode_ext* ext,
                          const void* q, const void* kv_pool, const int32_t* block_table,
                          const int32_t* ctx_lens, int head_lo, int head_hi, int64_t tok_lo,
                          int64_t tok_hi, float* out, float* lse, void* workspace,
                          size_t ws_bytes, splash_stream_t stream);

/*
 * splash_decode_attn without a caller workspace.  This entry point has no
 * counterpart in the paper; it exists for callers that cannot allocate device
 * memory at the point where they decode: code inside CUDA stream capture (a
 * cudaMalloc there is not captured and can invalidate the capture), serving loops
 * whose memory is owned by another allocator or capped by a fixed budget, and
 * plugins that are handed only input and output buffers.
 *
 * Same arguments, results and errors as splash_decode_attn, minus the workspace:
 * the scratch is a 32 MiB array inside the library, resident on every GPU that
 * loads the library until the process exits.  No cudaMalloc, cudaFree or other
 * allocating routine is called.
 *   - A shape whose splash_decode_workspace_size exceeds 32 MiB is rejected with
 *     SPLASH_ERR_WORKSPACE.  With 128 heads on a 152-SM GB300 that is more than
 *     51 requests per call; a 16-head shard takes up to 868.
 *   - The first call on a device resolves the array's device address
 *     (cudaGetSymbolAddress with that device current); make that first call
 *     before any stream capture.
 *   - Every call on a device shares the one array and it keeps the last call's
 *     contents (each call rewrites all of it that it reads).  Calls that may
 *     overlap on the GPU (different streams, or graphs replayed concurrently)
 *     race on it: serialise them.
 *   - The device status word (SPLASH_DEVICE_* bits) of the last call on the
 *     device is read with splash_noalloc_status.
 */
SPLASH_API int splash_decode_attn_noalloc(const splash_attn_desc* desc, const void* q,
                                          const void* kv_pool, const int32_t* block_table,
                                          const int32_t* ctx_lens, int head_lo, int head_hi,
                                          int64_t tok_lo, int64_t tok_hi, float* out, float* lse,
                                          splash_stream_t stream);

/*
 * Device status word of the most recent splash_decode_attn_noalloc call on the
 * current device (the SPLASH_DEVICE_* bits that splash_workspace_status reports
 * for a caller workspace).  Like splash_decode_attn_noalloc it has no counterpart
 * in the paper.  Synchronises `stream` (the stream of that call), then copies 4
 * bytes from the library's scratch to *flags (host pointer).  The word belongs to
 * the last call on the device, whichever stream issued it.  Allocates nothing.
 * Returns SPLASH_OK or an error.
 */
SPLASH_API int splash_noalloc_status(uint32_t* flags, splash_stream_t stream);

/*
 * Log-sum-exp merge of S partial results over disjoint token sets (the CP
 * combine; Appendix, Table 2, ideal token partitioning):
 *   m = max_s part_lse[s][b][h], w_s = exp(part_lse[s][b][h] - m),
 *   out[b][h] = sum_s w_s part_out[s][b][h] / sum_s w_s,  lse[b][h] = m + ln sum_s w_s;
 *   rows whose parts are all empty (-inf) give out = 0, lse = -inf.
 *   part_out fp32 [S][B][H][d_v], part_lse fp32 [S][B][H]; out fp32 [B][H][d_v],
 *   lse fp32 [B][H].  S >= 1, d_v a positive multiple of 4, 16-byte aligned
 *   part_out / out.  out may not alias part_out.
 */
SPLASH_API int splash_lse_merge(const float* part_out, const float* part_lse, int S, int B, int H, int d_v,
                     float* out, float* lse, splash_stream_t stream);

/*
 * KV-page migration between block pools (Abstract: a switch moves the state
 * that is not yet where the next layout needs it):
 *   dst_pool page dst_ids[i]  <-  byte copy of src_pool page src_ids[i],  i < n_pages.
 *   page_bytes  size of one page (P * 576 * 2 for this cache), multiple of 16
 *   src_ids, dst_ids int32 [n_pages] (device); dst_ids must be distinct; when
 *               src_pool == dst_pool the two id sets must be disjoint
 *   src_num_pages, dst_num_pages  pool sizes: a pair with an id outside its pool
 *               is skipped (no byte of either pool is touched for it)
 * Pools must be 16-byte aligned.  The caller rewrites its block tables.
 */
SPLASH_API int splash_kv_migrate(const void* src_pool, void* dst_pool, size_t page_bytes,
                      const int32_t* src_ids, const int32_t* dst_ids, int n_pages,
                      int32_t src_num_pages, int32_t dst_num_pages, splash_stream_t stream);

/* ---------------------------------------------------------------------------
 * The serving step around the attention: rotary positions, writing new tokens
 * into the paged cache (plain or quantised), reading quantised pages back, and
 * causal attention of a chunk of new tokens.
 *
 * A ragged batch of new tokens is described the same way everywhere: the new
 * tokens of all requests are packed in one array of total_q rows, and
 *   cu_q        int32 [B + 1] device, ascending, 0 <= cu_q[r] <= total_q: request r owns
 *               rows [cu_q[r], cu_q[r + 1]); rows outside every request are padding
 *   ctx_lens    int32 [B]: tokens of request r once its new tokens are written, so that
 *               row cu_q[r] + i is the token at position ctx_lens[r] - n_r + i
 *               (n_r = cu_q[r + 1] - cu_q[r])
 *   block_table int32 [B][max_pages_per_req], as for splash_decode_attn
 * ------------------------------------------------------------------------- */

/*
 * A ragged batch whose arrays the device builds (host struct, read during the call only).
 *   num_reqs, page_size, num_pages, max_pages_per_req   as in splash_attn_desc
 *   total_q      rows that positions and slots have, 2^30 at most;  reserved is 0
 *   past_lens    int32 [B]: tokens of request r in the cache;  new_lens int32 [B]: its new tokens (0 or more)
 *   free_pages   int32 [num_pages], a stack: entries [0, *free_count) are free pages' ids, the last one on top
 *   free_count   int32 [1]; a value outside [0, num_pages] is clamped into it
 *   block_table  int32 [B][max_pages_per_req]: entries for the past tokens' pages are there already; those
 *                that the new tokens add are written, the others left as they are
 *   cu_q, ctx_lens   int32 [B + 1] and [B]: as above; ctx_lens[r] = past_lens[r] + new_lens[r]
 *   positions, slots int32 [total_q]: a new token's position, and its row of the pool: page id * P + position % P
 *                (-1 where the page id is outside [0, num_pages)).  Rows past cu_q[B] are left as they are
 *   left         int32 [2]: free pages left, the next *free_count; requests served
 */
typedef struct {
    int32_t num_reqs;
    int32_t page_size;
    int32_t num_pages;
    int32_t max_pages_per_req;
    int32_t total_q;
    int32_t reserved;
    const int32_t* past_lens;
    const int32_t* new_lens;
    const int32_t* free_pages;
    const int32_t* free_count;
    int32_t* block_table;
    int32_t* cu_q;
    int32_t* ctx_lens;
    int32_t* positions;
    int32_t* slots;
    int32_t* left;
} splash_batch;

/*
 * The arrays of a ragged batch from its request lengths, with pages from a free list: what a step begins
 * with, built on the device, so that lengths and tables need not come back to the host.
 * Pages are taken from the top of the stack in the order of the requests and of their pages; the stack is read,
 * not written (left holds its new height).  The batch is served up to the first request that cannot be:
 * one for which rows or free pages do not suffice, or whose lengths are negative or add up to more than
 * max_pages_per_req * P.  That request and the ones after it get neither rows (cu_q[r + 1] = cu_q[r]) nor pages, and
 * ctx_lens[r] = past_lens[r].
 * ctx_lens may be past_lens, and left may begin at free_count; otherwise no two arrays may overlap.
 */
SPLASH_API int splash_batch_tables(const splash_batch* batch, splash_stream_t stream);

/*
 * Tokens to drop from a batch (host struct, read during the call only).
 *   num_reqs, page_size, num_pages, max_pages_per_req, block_table, free_pages, free_count: as in splash_batch;
 *                the three arrays are updated
 *   ctx_lens     int32 [B], in and out: request r keeps its first keep_lens[r] tokens (all, if it has fewer or
 *                keep_lens is NULL; a negative value keeps none), and ctx_lens[r] becomes their number k
 *   window, sinks  window > 0: also the pages all of whose tokens lie in [sinks, k + 1 - window), which no later
 *                token sees (see splash_chunk_attn_ex).  0: none; sinks is then unused
 */
typedef struct {
    int32_t num_reqs;
    int32_t page_size;
    int32_t num_pages;
    int32_t max_pages_per_req;
    int32_t window;
    int32_t sinks;
    int32_t* ctx_lens;
    const int32_t* keep_lens;
    int32_t* block_table;
    int32_t* free_pages;
    int32_t* free_count;
} splash_batch_drop;

/*
 * Gives pages back to the free list: those of tokens that are dropped (a request that ends, drafted tokens that
 * are rejected), and those that a sliding window has left behind.
 * Pages [ceil(k / P), ceil(ctx / P)) and the window's go on the stack, and their entries become -1.  An entry
 * outside [0, num_pages) has no page: it is passed over.  The pages go on so that the first request's first one lies
 * on top: after splash_batch_tables, dropping the same new tokens puts the stack back as it was.
 * A page that several requests share must be kept by all of them but one, or it is on the list more than
 * once.  Pages that do not fit on the stack are lost.  With a window, tokens are dropped in the same call or before it: what the
 * window has left behind k tokens does not come back when a later call keeps fewer.  num_reqs * max_pages_per_req is below 2^31.  No two arrays may
 * overlap (keep_lens may be ctx_lens).
 */
SPLASH_API int splash_batch_release(const splash_batch_drop* drop, splash_stream_t stream);

/* Element types of splash_rope and of splash_chunk_attn's output. */
enum { SPLASH_BF16 = 0, SPLASH_F16 = 1, SPLASH_F32 = 2 };

/* Frequency scaling of rotary positions. */
enum { SPLASH_ROPE_PLAIN = 0, SPLASH_ROPE_LINEAR = 1, SPLASH_ROPE_YARN = 2 };

/*
 * Rotary positions (host struct, read during the call only).
 *   dims         d, rotated dims of a head: even, 2..256
 *   interleaved  nonzero: pair i is dims (2i, 2i + 1); zero: dims (i, i + d / 2)
 *   scaling      SPLASH_ROPE_PLAIN   f_i = base^(-2i / d) radians per position
 *                SPLASH_ROPE_LINEAR  f_i / factor
 *                SPLASH_ROPE_YARN    f_i * ((1 - g_i) + g_i / factor), g_i = clamp((i - lo) /
 *                    max(hi - lo, 0.001), 0, 1), lo = max(floor(pair(beta_fast)), 0),
 *                    hi = min(ceil(pair(beta_slow)), d - 1), pair(b) = d ln(orig_ctx / (2 pi b))
 *                    / (2 ln base)
 *   base         >= 1 (> 1 for YARN); factor >= 1; orig_ctx, beta_fast, beta_slow > 0 (YARN only)
 *   amplitude    multiplies cos and sin (1: a pure rotation); finite
 */
typedef struct {
    int32_t dims;
    int32_t interleaved;
    int32_t scaling;
    int32_t reserved; /* 0 */
    double base;
    double factor;
    double orig_ctx;
    double beta_fast;
    double beta_slow;
    double amplitude;
} splash_rope_desc;

/*
 * Rotates the d = rope->dims leading dims of every head row:
 *   (y_a, y_b) = amplitude * (x_a cos w - x_b sin w, x_a sin w + x_b cos w),  w = positions[t] * f_i
 * for the pairs (a, b) of rope->interleaved.  Pass pointers to the first rotated dim:
 * a position part at the end of a wider head is reached through the strides.
 *   dtype       SPLASH_BF16, SPLASH_F16 or SPLASH_F32, of x and y; computed in fp32 and
 *               rounded once.  The angle is reduced exactly: its error does not grow with the position
 *   x, y        [T][H][d] with strides in elements (head rows contiguous); y may be x with
 *               the same strides, otherwise the two may not overlap
 *   positions   int32 [T]; negative positions turn the other way (amplitude 1: they undo
 *               the rotation)
 * Elements of y outside the d dims are not written.  Any alignment of the elements' own
 * size is taken; 32-byte aligned pointers and strides run fastest.
 */
SPLASH_API int splash_rope(const splash_rope_desc* rope, int dtype, const void* x,
                           int64_t x_token_stride, int64_t x_head_stride, void* y,
                           int64_t y_token_stride, int64_t y_head_stride, const int32_t* positions,
                           int T, int H, splash_stream_t stream);

/*
 * RMS norm of head rows with the rotary positions of a part of each row in the same pass (host structs,
 * read during the call only).
 *   width         D, dims of a row, 1..1024
 *   norm_dims     n, 1..D: dims [0, n) are normalised, the others are copied (a key row whose position dims
 *                 follow its latent, for instance)
 *   rope_lo       the first rotated dim: [rope_lo, rope_lo + rope->dims) lies within the row
 *   weight_dtype  SPLASH_BF16, SPLASH_F16 or SPLASH_F32, of the weights
 *   eps           >= 0, finite
 *   weight_offset added to every weight (1 for weights that are held as differences from one)
 */
typedef struct {
    int32_t width;
    int32_t norm_dims;
    int32_t rope_lo;
    int32_t weight_dtype;
    float eps;
    float weight_offset;
} splash_norm_desc;

/*
 * One side's rows: x and y [T][heads][D] of the call's dtype with strides in elements (rows dense), and
 * weight [n] (NULL: ones, without the offset).  reserved is 0.
 */
typedef struct {
    const void* x;
    int64_t x_token_stride;
    int64_t x_head_stride;
    void* y;
    int64_t y_token_stride;
    int64_t y_head_stride;
    const void* weight;
    int32_t heads;
    int32_t reserved;
} splash_norm_rows;

/*
 * For every row of q, and of k with weights of its own (k may be NULL):
 *   z_j = x_j * (mean(x_0^2, ..., x_{n-1}^2) + eps)^(-1/2) * (weight_j + weight_offset), j < n;  z_j = x_j, j >= n
 *   y = z with the dims [rope_lo, rope_lo + d) rotated as by splash_rope (rope NULL: y = z, positions unused)
 * Computed in fp32 and rounded once; the sum of squares neither over- nor underflows.  Among the first n dims a NaN
 * makes NaN of them all, an infinity NaN of itself and zeros of the others, and a row of zeros with eps = 0 is NaN.
 *   positions   int32 [T], of both sides' rows
 * A side's y may be its x with the same strides; otherwise no two of the arrays may overlap.  Any alignment of
 * the elements' own size is taken; fastest are 16-byte aligned pointers and strides with n, rope_lo, D and d / 2
 * multiples of 16 bytes.
 */
SPLASH_API int splash_norm_rope(const splash_norm_desc* norm, const splash_rope_desc* rope, int dtype,
                                const splash_norm_rows* q, const splash_norm_rows* k, const int32_t* positions,
                                int T, splash_stream_t stream);

/*
 * Cache formats of splash_kv_append:
 *   SPLASH_KV_BF16   rows of 576 bf16 (1,152 bytes), what the attention reads
 *   SPLASH_KV_MXFP8  rows of 656 bytes: 512 e4m3 latents, 16 scale bytes (one per 32 latents),
 *                    64 bf16 rope dims.  A scale byte b stands for 2^(b - 127); a group's is
 *                    the least with max |x| <= 448 * 2^(b - 127) over its finite x (0 for a group
 *                    of zeros), and its codes are x / 2^(b - 127) rounded to nearest even.  NaN stays
 *                    NaN, an infinity becomes the group's largest code.  Every held value
 *                    is exact in bf16, with two exceptions: with scale bytes below 3 values
 *                    reach below bf16's least, and a finite |x| of 248 * 2^120 or more (bf16's last
 *                    eight) rounds to 2^128, which splash_kv_unpack reads back as an infinity.
 * Pages are P consecutive rows either way, so splash_kv_migrate moves both.
 */
enum { SPLASH_KV_BF16 = 0, SPLASH_KV_MXFP8 = 1 };

/*
 * Writes new tokens' keys into the paged cache: row cu_q[r] + i goes to slot
 * p % P of page block_table[r][p / P], p = ctx_lens[r] - n_r + i.
 *   desc         num_reqs, page_size, num_pages, max_pages_per_req, d_qk = 576 and d_v = 512;
 *                num_heads must be positive and is otherwise unused, as is scale
 *   rope         rotates the 64 rope dims by the token's position (dims must be 64), or
 *                NULL: they are written as they are
 *   format       SPLASH_KV_BF16 or SPLASH_KV_MXFP8, of kv_pool
 *   latent       bf16 [total_q][512], rows latent_stride elements apart (a multiple of 8),
 *                16-byte aligned
 *   k_rope       bf16 [total_q][64], rows k_rope_stride elements apart (even), 4-byte aligned
 *   kv_pool      16-byte aligned; slots that no new token owns are left as they are
 * A token is skipped when it is padding, when its position is outside [0, max_pages_per_req
 * * P) or when its page id is outside [0, num_pages).  Two tokens may not own one slot.
 */
SPLASH_API int splash_kv_append(const splash_attn_desc* desc, const splash_rope_desc* rope, int format,
                                const void* latent, int64_t latent_stride, const void* k_rope,
                                int64_t k_rope_stride, const int32_t* cu_q, int total_q,
                                const int32_t* block_table, const int32_t* ctx_lens, void* kv_pool,
                                splash_stream_t stream);

/*
 * Reads MXFP8 pages back: dst_pool page dst_ids[i] (bf16 [P][576]) <- the values of src_pool
 * page src_ids[i] (MXFP8 [P][656]), i < n_pages, all P rows.
 *   page_size   any positive number of tokens; ids and pool sizes as in splash_kv_migrate (a
 *               pair with an id outside its pool is skipped); the pools may not overlap, and
 *               dst_ids must be distinct.  A scale byte of 255 gives NaN.
 */
SPLASH_API int splash_kv_unpack(const void* src_pool, void* dst_pool, int page_size,
                                const int32_t* src_ids, const int32_t* dst_ids, int n_pages,
                                int32_t src_num_pages, int32_t dst_num_pages, splash_stream_t stream);

/*
 * Bytes of device workspace splash_chunk_attn needs for this shape, number of new
 * tokens and head range on the current device.  Returns 0 when the shape is invalid or
 * unsupported.
 */
SPLASH_API size_t splash_chunk_workspace_size(const splash_attn_desc* desc, int total_q, int head_lo,
                                              int head_hi);

/*
 * Causal attention of new tokens over the paged cache that already holds them
 * (a prompt, a chunk of one, drafted tokens, or single tokens; any mix of them).
 *
 * For the token at row t = cu_q[r] + i and head h in [head_lo, head_hi), over the tokens
 *   T = [tok_lo, min(tok_hi < 0 ? e : tok_hi, e)),  e = ctx_lens[r] - n_r + i + 1,
 * out[t][h] and lse[t][h] are those of splash_decode_attn with q[t][h].  An empty T gives
 * out = 0 and lse = -inf.  A share [tok_lo, tok_hi) gives the partial that splash_lse_merge
 * combines (fp32 out).
 *   q           bf16 [total_q][H][576], contiguous, 16-byte aligned
 *   out         [total_q][H][512] of out_dtype (SPLASH_BF16 or SPLASH_F32), 32-byte aligned
 *   lse         fp32 [total_q][H]
 *   head_lo/hi, tok_lo/hi, kv_pool, block_table, ctx_lens: as for splash_decode_attn, desc->num_reqs
 *               = B; one shared KV head
 *   workspace   >= splash_chunk_workspace_size(...) bytes, 256-byte aligned; one call at a time
 * Only rows that a request owns and heads [head_lo, head_hi) are written.  The scores of one
 * row never depend on another row.  Slots past a context may hold any bits; a token within a
 * context whose latent is not finite can make NaN of every new row of that request, also of
 * those that precede it.
 * A cu_q that descends or leaves [0, total_q] (no row is written then), a context length
 * outside [0, max_pages_per_req * P] (clamped) and a needed page id outside [0, num_pages) (its
 * tokens are left out) set SPLASH_DEVICE_BAD_INPUT, read with splash_workspace_status.
 * max_pages_per_req * P may be 2^31 - 1024 at most.  out is summed over the keys in fp32 with truncation:
 * over a context of millions of keys it comes out small, by up to 0.5% per million.  The same call on
 * the same device gives the same bits.
 */
SPLASH_API int splash_chunk_attn(const splash_attn_desc* desc, const void* q, const void* kv_pool,
                                 const int32_t* cu_q, int total_q, const int32_t* block_table,
                                 const int32_t* ctx_lens, int head_lo, int head_hi, int64_t tok_lo,
                                 int64_t tok_hi, int out_dtype, void* out, float* lse,
                                 void* workspace, size_t ws_bytes, splash_stream_t stream);

/*
 * What splash_chunk_attn_ex knows about the keys that new tokens see.  All zero: nothing.
 *   window, sinks   window > 0: the token at position p sees the last `window` positions up to its own,
 *                   p + 1 - window .. p, and the first `sinks` ones.  window 0: every position up to its own (sinks is
 *                   then unused)
 *   num_groups      G groups of requests with a common prefix, 1,024 at most; not together with a window
 *   cu_groups       int32 [G + 1] device, ascending, 0 <= cu_groups[g] <= B: group g is the requests [cu_groups[g],
 *                   cu_groups[g + 1]); requests outside every group share nothing
 *   prefix_lens     int32 [G] device: the first prefix_lens[g] tokens of the group's requests are the same, and in the cache
 *                   before their new ones.  They are read through the table of the group's first request
 */
typedef struct {
    int32_t window;
    int32_t sinks;
    const int32_t* cu_groups;
    const int32_t* prefix_lens;
    int32_t num_groups;
    int32_t reserved; /* 0 */
} splash_chunk_ext;

/*
 * splash_chunk_attn with `ext` (NULL: without).
 * Window:  T = {t in [tok_lo, min(tok_hi < 0 ? e : tok_hi, e)) : t >= e - window or t < sinks}.  A page that holds no token
 * which a new token of its request sees is not needed: its table entry may be anything (splash_batch_release gives
 * such pages back).
 * Groups:  the results are those of splash_chunk_attn; where it pays, the rows of a group's requests are worked on
 * together over the prefix, whose keys are then read and multiplied once for up to 128 of them (16 heads of 8
 * single tokens, for instance) instead of once a request.  Where a token's own rows fill that many (a call of all heads with 128
 * of them or more, a slice of more than 64) there is nothing to gain: such calls are worked on as by splash_chunk_attn and read
 * neither array, so what follows on their values holds for the other calls.  Whether it pays goes by the numbers of rows and keys, so equal calls give equal bits.
 * The prefix's entries in the tables of the group's other requests may or may not be read.  A prefix that is negative or longer than
 * max_pages_per_req * P (clamped), or longer than the tokens that one of its requests has before its new ones (whose rows
 * may then see all of it), and cu_groups that descend or leave [0, B] (no row is written then) set SPLASH_DEVICE_BAD_INPUT.
 * The workspace is that of splash_chunk_workspace_size_ex, which takes num_groups from ext and reads neither of its
 * arrays.  So it has room for a partial result (262 KB) of every 128 rows of the requests and of as many of the groups, 4 KB a
 * row, whether a group holds them or not: prompts of many tokens are better in a call of their own.
 * Otherwise the same arguments, results and errors as splash_chunk_attn, and without groups the same workspace.
 */
SPLASH_API size_t splash_chunk_workspace_size_ex(const splash_attn_desc* desc, const splash_chunk_ext* ext, int total_q,
                                                 int head_lo, int head_hi);
SPLASH_API int splash_chunk_attn_ex(const splash_attn_desc* desc, const splash_chunk_ext* ext, const void* q,
                                    const void* kv_pool, const int32_t* cu_q, int total_q, const int32_t* block_table,
                                    const int32_t* ctx_lens, int head_lo, int head_hi, int64_t tok_lo, int64_t tok_hi,
                                    int out_dtype, void* out, float* lse, void* workspace, size_t ws_bytes,
                                    splash_stream_t stream);

/*
 * Reads the device status of a decode or chunk workspace (SPLASH_DEVICE_* bits set
 * by the most recent splash_decode_attn or splash_chunk_attn that used it; one without
 * requests or new tokens clears them): synchronises `stream`, then copies the bits to *flags (host
 * pointer).  Returns SPLASH_OK or an error.
 */
SPLASH_API int splash_workspace_status(const void* workspace, uint32_t* flags, splash_stream_t stream);

/* Static string for a splash_status value. */
SPLASH_API const char* splash_status_string(int status);

#ifdef __cplusplus
}
#endif

#endif /* SPLASH_H_ */
