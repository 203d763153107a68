// batch_tables.cu -- a batch's index arrays from its request lengths, with pages from a free
// list, and pages back to it.
//
// Latency-bound: a decode step of 256 requests touches 6 KB.  What counts is the chain of dependent
// steps (lengths, sums over the requests, the page, the store), so each operator is one launch of one
// cluster: every CTA computes the sums of the whole batch for itself, and only the rows are dealt out.
// Lengths and counts may be updated in place, because the cluster's barrier stands between the last
// read and the first write.  Per call in replays of a graph, 256 single tokens of ragged lengths and 61 prompts of 31,000
// tokens both take 4.5 us; giving the pages of 128
// requests back 3.6 us, of 333 requests' 2,300 pages 5.1 us; looking through the 127,000 pages of 64 requests that a window
// of 4,096 tokens has left behind at 131,072 (512 KB) 8.6 us.
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

// The pages that the batch gives back, one after the other in the order of the requests and of their pages, are dealt out
// to the warps in equal runs: a window's pages are looked through in every step, whether they went back in an earlier one
// or not, and one long request has as many of them as hundreds of short ones.  A page's place on the list follows from the
// sums over all warps before its own.  With the requests dealt out instead, 64 of them at 131,072 tokens took 64 us, and one 58 (now 3.9).
// Eight pages of a lane under way take 8.0 where four take 8.5, but 0.1 to 0.4 more in small batches.
__global__ void __cluster_dims__(kReleaseCtas, 1, 1) __launch_bounds__(kTableThreads, 1)
    batch_release_kernel(const __grid_constant__ BatchReleaseArgs a) {
    constexpr int NT = kTableThreads, U = 4;       // pages of a lane under way
    __shared__ int start[NT + 1], lo0[NT], n0[NT], lo1[NT];
    __shared__ int2 scratch[kWarps];
    __shared__ int counts[kReleaseCtas];           // every CTA's pages, in each CTA
    __shared__ int warps[kWarps];
    cluster_sync();                                // every CTA of the cluster has begun: its memory may be written
    pdl_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = int(cluster_rank());
    const int top = min(max(*a.free_count, 0), a.num_pages);
    int keep = 0;                                  // of the thread's request in the last pass
    // the requests [b0, b0 + NT): their pages' places in the order, counted from b0's first; returns how many pages
    auto pass = [&](int b0) {
        const Gone g = gone_of(a, b0 + tid);
        keep = g.keep;
        int x = g.n0 + g.n1, y = 0;
        __syncthreads();                           // nothing reads the pass before any more
        block_sums(x, y, scratch);
        start[tid + 1] = x;
        if (tid == 0) start[0] = 0;
        lo0[tid] = g.lo0;
        n0[tid] = g.n0;
        lo1[tid] = g.lo1;
        __syncthreads();
        return start[NT];
    };
    int all = pass(0);                             // (num_reqs * max_pages_per_req < 2^31)
    const int in_first = all;
#pragma unroll 1
    for (int b0 = NT; b0 < a.B; b0 += NT) all += pass(b0);
    const uint32_t run = (uint32_t(all) + kReleaseCtas * kWarps * 32 - 1) / (kReleaseCtas * kWarps * 32) * 32;
    const uint32_t first = min(run * uint32_t(rank * kWarps + warp), uint32_t(all)), last = min(first + run, uint32_t(all));

    int id[U], at[U];
    // groups of 32 U pages: each(g) for the warp's g-th, after fetch(g) unless that says that it may be skipped
    auto sweep = [&](auto skip, auto each) {
        int g = 0;
        uint32_t base = 0;
#pragma unroll 1
        for (int b0 = 0; b0 < a.B; b0 += NT) {
            const uint32_t here = uint32_t(a.B > NT ? pass(b0) : in_first);
            const uint32_t end = min(last, base + here);
            int j = 0;
#pragma unroll 1
            for (uint32_t i0 = max(first, base); i0 < end; i0 += 32 * U, ++g) {
                if (!skip(g)) {
#pragma unroll
                    for (int e = 0; e < U; ++e) {
                        const uint32_t i = i0 + e * 32 + lane;
                        id[e] = at[e] = -1;
                        if (i < end) {
                            const int k = int(i - base);
                            if (k >= start[j + 1]) j = owner(start, min(NT, a.B - b0), k);
                            const int n = k - start[j], page = n < n0[j] ? lo0[j] + n : lo1[j] + n - n0[j];
                            at[e] = (b0 + j) * a.max_pages + page;
                            id[e] = a.table[at[e]];
                        }
                    }
                }
                each(g);
            }
            base += here;
        }
    };
    // Nothing to do for group g (bit g; the last bit is that of all groups behind the 63rd too): neither a page to give back
    // nor an entry to clear.
    uint64_t busy = 0;
    int mine = 0;
    sweep([](int) { return false; },
          [&](int g) {
              bool any = false;
#pragma unroll
              for (int e = 0; e < U; ++e) {
                  any = any || id[e] != -1;
                  mine += __popc(__ballot_sync(0xffffffffu, uint32_t(id[e]) < uint32_t(a.num_pages)));
              }
              if (__any_sync(0xffffffffu, any)) busy |= uint64_t(1) << min(g, 63);
          });
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
    const bool held = run <= 32 * U && a.B <= NT;  // the warp's only group is in its registers still
    auto idle = [&](int g) { return !((busy >> min(g, 63)) & 1); };
    sweep([&](int g) { return held || idle(g); },
          [&](int g) {
              if (idle(g)) return;
#pragma unroll
              for (int e = 0; e < U; ++e) {
                  const bool valid = uint32_t(id[e]) < uint32_t(a.num_pages);
                  const uint32_t m = __ballot_sync(0xffffffffu, valid);
                  const int to = place - __popc(m & ((1u << lane) - 1));
                  if (valid && to < a.num_pages) a.free_pages[to] = id[e];
                  if (id[e] != -1) a.table[at[e]] = -1;
                  place -= __popc(m);
              }
          });
    if (a.B > NT) cluster_sync();                  // no CTA reads the lengths any more
#pragma unroll 1
    for (int r = rank * NT + tid; r < a.B; r += kReleaseCtas * NT) {
        if (a.B > NT) keep = gone_of(a, r).keep;
        a.ctx[r] = keep;
    }
    if (rank == 0 && tid == 0) *a.free_count = min(top + total, a.num_pages);
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
