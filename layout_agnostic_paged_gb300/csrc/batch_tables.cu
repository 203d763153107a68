// batch_tables.cu -- a batch's index arrays from its request lengths, with pages from a free
// list, and pages back to it.
//
// Latency-bound: a decode step of 256 requests touches 6 KB.  What counts is the chain of dependent
// steps (lengths, sums over the requests, the page, the store), so each operator is one launch of one
// cluster: every CTA computes the sums of the whole batch for itself, and only the rows are dealt out.
// Lengths and counts may be updated in place, because the cluster's barrier stands between the last
// read and the first write.  256 single tokens and 61 prompts of 31,000 tokens both take 4.4 us; giving the pages of 128
// requests back 3.8 us, of 333 requests' 2,300 pages 6 us.
#include <limits.h>

#include "common.cuh"
#include "kernels.h"
#include "pair.cuh"

namespace splash {
namespace {

constexpr int kTableThreads = 1024;   // requests of one pass
constexpr int kWarps = kTableThreads / 32;

template <int C>
__device__ __forceinline__ void sync_all() {
    if constexpr (C > 1) cluster_sync();
    else __syncthreads();
}

__device__ __forceinline__ int pages_of(int len, int P_log) {   // len >= 0
    return int((uint32_t(len) + (1u << P_log) - 1) >> P_log);
}

// a + b, at most INT_MAX (a, b >= 0)
__device__ __forceinline__ int sat_add(int a, int b) {
    const uint32_t s = uint32_t(a) + uint32_t(b);
    return s > uint32_t(INT_MAX) ? INT_MAX : int(s);
}

// Inclusive sums of two values over the block, saturating.  scratch: 2 ints per warp.
__device__ __forceinline__ void block_sums(int& x, int& y, int2* scratch) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int a = __shfl_up_sync(0xffffffffu, x, o), b = __shfl_up_sync(0xffffffffu, y, o);
        if (lane >= o) {
            x = sat_add(x, a);
            y = sat_add(y, b);
        }
    }
    if (lane == 31) scratch[warp] = make_int2(x, y);
    __syncthreads();
    int2 w = scratch[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int a = __shfl_up_sync(0xffffffffu, w.x, o), b = __shfl_up_sync(0xffffffffu, w.y, o);
        if (lane >= o) {
            w.x = sat_add(w.x, a);
            w.y = sat_add(w.y, b);
        }
    }
    const int before = warp == 0 ? 0 : warp - 1;
    const int a = __shfl_sync(0xffffffffu, w.x, before), b = __shfl_sync(0xffffffffu, w.y, before);
    if (warp > 0) {
        x = sat_add(x, a);
        y = sat_add(y, b);
    }
}
static_assert(kWarps == 32, "block_sums reads a value per lane");

// The last index in [0, n) with from[i] <= x (n >= 1, ascending, from[0] <= x).
__device__ __forceinline__ int owner(const int* from, int n, int x) {
    int lo = 0;
    for (int len = n; len > 1;) {
        const int half = len >> 1;
        if (from[lo + half] <= x) {
            lo += half;
            len -= half;
        } else {
            len = half;
        }
    }
    return lo;
}

// A batch's arrays.  A request is served if it and all before it have valid lengths, rows and pages; the
// others keep their length and get neither.
template <int C>
__global__ void __cluster_dims__(C, 1, 1) __launch_bounds__(kTableThreads, 1)
    batch_tables_kernel(const __grid_constant__ BatchTablesArgs a) {
    constexpr int NT = kTableThreads;
    __shared__ int row0[NT], page0[NT], past[NT];
    __shared__ int2 scratch[kWarps];
    __shared__ int ends[2];
    pdl_wait();
    const int tid = threadIdx.x;
    const int rank = C > 1 ? int(cluster_rank()) : 0;
    const int P_log = a.P_log, off = (1 << P_log) - 1;
    const int count = min(max(*a.free_count, 0), a.num_pages);
    const int64_t max_ctx = int64_t(a.max_pages) << P_log;
    int rows = 0, used = 0, served = 0;           // of the passes before
    bool stopped = false;
    for (int b0 = 0; b0 < a.B; b0 += NT) {
        const int r = b0 + tid, nb = min(NT, a.B - b0);
        int p = 0, n = 0;
        bool bad = false;
        if (r < a.B) {
            p = a.past[r];
            n = a.fresh[r];
            bad = p < 0 || n < 0 || int64_t(p) + n > max_ctx;
        }
        const int have = bad ? 0 : pages_of(p, P_log), need = bad ? 0 : pages_of(p + n, P_log) - have;
        int x = bad ? INT_MAX : n, y = need;       // (bad lengths end the batch: no call has INT_MAX rows)
        if (tid == 0) ends[0] = ends[1] = 0;
        block_sums(x, y, scratch);
        const bool ok = tid < nb && !stopped && sat_add(rows, x) <= a.total_q && sat_add(used, y) <= count;
        const int ns = __syncthreads_count(ok);    // served requests of this pass: the first ns
        if (ok && tid == ns - 1) {
            ends[0] = x;
            ends[1] = y;
        }
        row0[tid] = rows + x - n;
        page0[tid] = used + y - need;
        past[tid] = p;
        sync_all<C>();                             // and every CTA has read the lengths
        const int rows_end = rows + ends[0], used_end = used + ends[1];
        if (rank == 0 && r < a.B) {
            a.cu[r] = ok ? row0[tid] : rows_end;
            a.ctx[r] = ok ? p + n : p;
        }
        // new pages into the table
        for (int k = used + rank * NT + tid; k < used_end; k += C * NT) {
            const int j = owner(page0, ns, k);
            a.table[int64_t(b0 + j) * a.max_pages + pages_of(past[j], P_log) + (k - page0[j])] =
                a.free_pages[count - 1 - k];
        }
        // rows, four to a thread
        for (int g = (rows >> 2) + rank * NT + tid; 4 * g < rows_end; g += C * NT) {
            int t = max(4 * g, rows);
            const int end = min(4 * g + 4, rows_end);
            int j = owner(row0, ns, t);
            int pos[4], slot[4], id = -1, page = -1;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int at = 4 * g + e;
                if (at < t || at >= end) continue;
                bool other = page < 0;
                while (j + 1 < ns && row0[j + 1] <= at) {
                    ++j;
                    other = true;
                }
                pos[e] = past[j] + (at - row0[j]);
                if (other || pos[e] >> P_log != page) {
                    page = pos[e] >> P_log;
                    const int h = pages_of(past[j], P_log);
                    id = page >= h ? a.free_pages[count - 1 - (page0[j] + page - h)]
                                   : a.table[int64_t(b0 + j) * a.max_pages + page];
                }
                slot[e] = id >= 0 && id < a.num_pages ? (id << P_log) + (pos[e] & off) : -1;
            }
            if (a.wide && t == 4 * g && end == 4 * g + 4) {
                reinterpret_cast<int4*>(a.positions)[g] = make_int4(pos[0], pos[1], pos[2], pos[3]);
                reinterpret_cast<int4*>(a.slots)[g] = make_int4(slot[0], slot[1], slot[2], slot[3]);
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (4 * g + e >= t && 4 * g + e < end) {
                        a.positions[4 * g + e] = pos[e];
                        a.slots[4 * g + e] = slot[e];
                    }
            }
        }
        rows = rows_end;
        used = used_end;
        served += ns;
        stopped = stopped || ns < nb;
        __syncthreads();                           // the next pass writes the shared arrays
    }
    if (a.B == 0) __syncthreads();                 // every thread has read the count
    if (rank == 0 && tid == 0) {
        a.cu[a.B] = rows;
        a.left[0] = count - used;
        a.left[1] = served;
    }
}

// The pages that a request gives back: [lo0, lo0 + n0) that no later token sees, [lo1, lo1 + n1) behind the kept tokens.
struct Gone {
    int keep, lo0, n0, lo1, n1;
};
__device__ __forceinline__ Gone gone_of(const BatchReleaseArgs& a, int r) {
    Gone g = {};
    if (r >= a.B) return g;
    const int64_t max_ctx = int64_t(a.max_pages) << a.P_log;
    const int ctx = int(min(int64_t(max(a.ctx[r], 0)), max_ctx));
    g.keep = a.keep ? min(max(a.keep[r], 0), ctx) : ctx;
    g.lo1 = pages_of(g.keep, a.P_log);
    g.n1 = pages_of(ctx, a.P_log) - g.lo1;
    if (a.window > 0) {
        // the next token, at position keep, sees the keys from keep + 1 - window on
        const int first = pages_of(a.sinks, a.P_log), end = g.keep + 1 > a.window ? (g.keep + 1 - a.window) >> a.P_log : 0;
        g.lo0 = first;
        g.n0 = max(0, end - first);
    }
    return g;
}

// The warp's requests [r0, r1), 32 at a time, and their pages, 32 at a time whatever requests they belong
// to.  each(request, page, id, valid) runs converged.
template <typename F>
__device__ __forceinline__ void for_pages(const BatchReleaseArgs& a, int r0, int r1, F each) {
    const int lane = threadIdx.x & 31;
#pragma unroll 1
    for (int rb = r0; rb < r1; rb += 32) {
        const Gone g = gone_of(a, rb + lane < r1 ? rb + lane : a.B);
        uint32_t sum = uint32_t(g.n0 + g.n1);      // (a request has fewer than 2^27 pages: 32 of them fit)
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t x = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += x;
        }
        const uint32_t total = __shfl_sync(0xffffffffu, sum, 31);
        const uint32_t start = sum - uint32_t(g.n0 + g.n1);
#pragma unroll 1
        for (uint32_t i0 = 0; i0 < total; i0 += 32) {
            const uint32_t i = i0 + lane;
            int j = 0;                             // the last request with start <= i (others share a start with the next)
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                const uint32_t s = __shfl_sync(0xffffffffu, start, j + o);
                if (s <= i) j += o;
            }
            const uint32_t s = __shfl_sync(0xffffffffu, start, j);
            const int n0 = __shfl_sync(0xffffffffu, g.n0, j);
            const int lo0 = __shfl_sync(0xffffffffu, g.lo0, j), lo1 = __shfl_sync(0xffffffffu, g.lo1, j);
            const int k = int(i - s), page = k < n0 ? lo0 + k : lo1 + (k - n0);
            int id = -1;
            if (i < total) id = a.table[int64_t(rb + j) * a.max_pages + page];
            each(rb + j, page, id, i < total && id >= 0 && id < a.num_pages, i < total);
        }
    }
}

// A warp takes a run of consecutive requests; the pages' places on the list follow from the sums over all
// warps before it.
__global__ void __cluster_dims__(kReleaseCtas, 1, 1) __launch_bounds__(kTableThreads, 1)
    batch_release_kernel(const __grid_constant__ BatchReleaseArgs a) {
    __shared__ int counts[kReleaseCtas];           // every CTA's pages, in each CTA
    __shared__ int warps[kWarps];
    cluster_sync();                                // every CTA of the cluster has begun: its memory may be written
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int rank = int(cluster_rank());
    const int w = rank * kWarps + warp;
    const int r0 = int(int64_t(a.B) * w / (kReleaseCtas * kWarps)), r1 = int(int64_t(a.B) * (w + 1) / (kReleaseCtas * kWarps));
    const int top = min(max(*a.free_count, 0), a.num_pages);
    int mine = 0;
    for_pages(a, r0, r1, [&](int, int, int, bool valid, bool) { mine += __popc(__ballot_sync(0xffffffffu, valid)); });
    if (lane == 0) warps[warp] = mine;
    __syncthreads();
    if (warp == 0) {
        const int own = warps[lane];
        int sum = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += x;
        }
        warps[lane] = sum - own;
        const int total = __shfl_sync(0xffffffffu, sum, 31);
        if (lane < kReleaseCtas)
            asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(map_to_rank(smem_u32(&counts[rank]), lane)), "r"(total)
                         : "memory");
    }
    cluster_sync();
    int before = warps[warp], total = 0;
#pragma unroll
    for (int c = 0; c < kReleaseCtas; ++c) {
        if (c < rank) before += counts[c];
        total += counts[c];
    }
    // the last page goes on the list first, so that the first lies on top
    int place = top + total - 1 - before;
    for_pages(a, r0, r1, [&](int r, int page, int id, bool valid, bool live) {
        const uint32_t m = __ballot_sync(0xffffffffu, valid);
        const int at = place - __popc(m & ((1u << lane) - 1));
        if (valid && at < a.num_pages) a.free_pages[at] = id;
        if (live) a.table[int64_t(r) * a.max_pages + page] = -1;
        place -= __popc(m);
    });
    __syncwarp();
#pragma unroll 1
    for (int r = r0 + lane; r < r1; r += 32) {     // (behind the last read of the warp's lengths)
        const int keep = gone_of(a, r).keep;
        a.ctx[r] = keep;
    }
    if (rank == 0 && threadIdx.x == 0) *a.free_count = min(top + total, a.num_pages);
}

}  // namespace

cudaError_t launch_batch_tables(const BatchTablesArgs& a, cudaStream_t stream) {
    const dim3 b(kTableThreads);
    if (a.total_q <= kSmallBatchRows) return launch_pdl(batch_tables_kernel<1>, dim3(1), b, 0, stream, a);
    return launch_pdl(batch_tables_kernel<8>, dim3(8), b, 0, stream, a);
}

cudaError_t launch_batch_release(const BatchReleaseArgs& a, cudaStream_t stream) {
    return launch_pdl(batch_release_kernel, dim3(kReleaseCtas), dim3(kTableThreads), 0, stream, a);
}

}  // namespace splash
