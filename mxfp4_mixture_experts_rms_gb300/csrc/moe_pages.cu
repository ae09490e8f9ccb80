// moe_pages.cu -- block tables and slot maps of a paged cache, built on the
// GPU from request lengths: finished requests' pages go back to the free
// list, the others take what their new tokens need, and every new token gets
// its slot and position.
//
// Three prefix sums over the requests (entries that finished ones give back,
// pages that the others take, new tokens) make everything flat: entry e,
// page p and token t each find their request by binary search, and the page
// of a token is either in the table or at a known place of the free list, so
// that tables and slots are written side by side.  What remains in order is
// the free list: entries are compacted (those below 0 are none) and pushed
// before any is popped.
//
// A small step is one kernel of one CTA, bound by its chain of dependent
// loads; a large one is a cluster that pushes, then a grid that writes tables
// and slots, whose CTAs each repeat the prefix sums (two loads a request from
// L2) rather than wait for them through memory.  Neighbouring entries rarely
// leave a request; one that does looks for the next by a step and then by
// search (steps alone, over the running requests between two finished ones:
// 25 us instead of 15 for 2048 requests with 586 thousand new tokens).  64
// requests of a decode step: 7.2 us.
#include "moe_common.cuh"
#include "../../include/moe.h"

#include <cooperative_groups.h>

#include <algorithm>
#include <climits>

namespace cg = cooperative_groups;

namespace {

constexpr int kMaxSeqs = 4096;
constexpr int kPushThreads = 512, kSmallThreads = 256;
constexpr int kFillThreads = 256;
constexpr int kCluster = 8;
// One CTA does it all up to so many requests, tokens that there is room for and
// table entries; above, the second kernel's parallel writes gain more than its
// launch costs.  One CTA and two kernels, us: 64 requests with 899, 2022, 2891,
// 5785 new tokens 6.7 and 9.5, 8.0 and 9.1, 10.5 and 9.3, 15.3 and 9.2 (room for
// 4096 and 8192 with 60 there: 7.2 and 9.6, 8.1 and 9.4); 512, 1024, 2048
// requests of one token 9.3 and 10.6, 11.4 and 11.3, 19.1 and 12.4; 256 requests
// with tables of 16 K and 128 K entries 7.3 and 10.4, 11.3 and 10.3, 1024 with
// 513 K (many finished) 30.9 and 11.9.
constexpr int kSmallSeqs = 1024, kSmallTokens = 2048, kSmallTable = 65536;

struct PagesArgs {
    int P, shift, n, width, cap, max_tokens;   // shift: log2 P where P is a power of two, else -1
    const int32_t *cached, *fresh;
    int32_t *table, *free_pages;
    const int32_t *counts;
    int32_t *counts_out, *starts, *lens, *slots, *positions;
};

// Exclusive sums over requests: entries given back (those below 0 among them),
// pages wanted, new tokens.
struct Sums {
    int back, want;
    long long tok;
};
__device__ __forceinline__ Sums operator+(Sums a, Sums b) { return {a.back + b.back, a.want + b.want, a.tok + b.tok}; }
__device__ __forceinline__ Sums operator-(Sums a, Sums b) { return {a.back - b.back, a.want - b.want, a.tok - b.tok}; }
__device__ __forceinline__ Sums warp_inclusive(Sums v) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const Sums o = {__shfl_up_sync(0xffffffffu, v.back, d), __shfl_up_sync(0xffffffffu, v.want, d), __shfl_up_sync(0xffffffffu, v.tok, d)};
        if (lane >= d) v = v + o;
    }
    return v;
}

// x / P for x below 2^32: lengths and their sums are
__device__ __forceinline__ unsigned page_of(unsigned x, const PagesArgs &a) { return a.shift >= 0 ? x >> a.shift : x / (unsigned)a.P; }
// pages of so many tokens, at most a row of the table
__device__ __forceinline__ int pages_of(unsigned tokens, const PagesArgs &a) {
    return tokens ? (int)min(page_of(tokens - 1, a) + 1, (unsigned)a.width) : 0;
}
__device__ __forceinline__ int clamp_int(long long v) { return (int)min(v, (long long)INT_MAX); }

// Shared memory: [n] each, exclusive sums over the requests before.
struct Requests {
    int *have, *fresh, *back, *want, *start;
    __device__ Requests(int *s, int n) : have(s), fresh(s + n), back(s + 2 * n), want(s + 3 * n), start(s + 4 * n) {}
};

template <int T>
__device__ Sums scan_requests(const PagesArgs &a, const Requests &q, Sums *part) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (int b = tid; b < a.n; b += T) q.have[b] = max(a.cached[b], 0), q.fresh[b] = a.fresh[b];
    __syncthreads();
    const int per = (a.n + T - 1) / T, b0 = min(tid * per, a.n), b1 = min(b0 + per, a.n);
    auto of = [&](int b) {
        const int f = q.fresh[b], held = pages_of(q.have[b], a);
        return f < 0 ? Sums{held, 0, 0} : Sums{0, pages_of((unsigned)q.have[b] + (unsigned)f, a) - held, f};
    };
    Sums v = {0, 0, 0};
    for (int b = b0; b < b1; b++) v = v + of(b);
    const Sums inc = warp_inclusive(v);
    if (lane == 31) part[warp] = inc;
    __syncthreads();
    const Sums mine = lane < T / 32 ? part[lane] : Sums{0, 0, 0}, upto = warp_inclusive(mine), before = upto - mine;
    const Sums total = {__shfl_sync(0xffffffffu, upto.back, 31), __shfl_sync(0xffffffffu, upto.want, 31), __shfl_sync(0xffffffffu, upto.tok, 31)};
    Sums at = inc - v;
    at = at + Sums{__shfl_sync(0xffffffffu, before.back, warp), __shfl_sync(0xffffffffu, before.want, warp), __shfl_sync(0xffffffffu, before.tok, warp)};
    for (int b = b0; b < b1; b++) {
        q.back[b] = at.back, q.want[b] = at.want, q.start[b] = clamp_int(at.tok);
        at = at + of(b);
    }
    __syncthreads();
    return total;
}

// The last request whose sum is at most x (the one that x lies in).
__device__ __forceinline__ int request_of(const int *sum, int n, int x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (sum[mid] <= x) lo = mid;
        else hi = mid;
    }
    return lo;
}

// The same for the next x, from b on: the request itself, the next or any.
__device__ __forceinline__ int request_from(const int *sum, int n, int x, int b) {
    if (b + 1 < n && sum[b + 1] <= x && ++b + 1 < n && sum[b + 1] <= x) b = request_of(sum, n, x);
    return b;
}

// Tables of wanted pages first, first + step, .. and slots and positions of
// tokens likewise, four neighbours at a time.  n1: free pages before the pops.
__device__ __forceinline__ void fill(const PagesArgs &a, const Requests &q, const Sums &total, int n1, int first, int step) {
    for (unsigned at = first; at < (unsigned)total.want; at += step) {   // (at + step may pass 2^31)
        const int p = (int)at, b = request_of(q.want, a.n, p), src = n1 - 1 - p;
        a.table[(size_t)b * a.width + pages_of(q.have[b], a) + (p - q.want[b])] = src >= 0 ? a.free_pages[src] : -1;
    }
    const int tokens = clamp_int(total.tok), most = INT_MAX / a.P;   // pages whose slots are 32-bit
    const bool wide = (((uintptr_t)a.slots | (uintptr_t)a.positions) & 15u) == 0;
    for (long long t0 = 4ll * first; t0 < a.max_tokens; t0 += 4ll * step) {
        int slot[4], pos[4], b = t0 < tokens ? request_of(q.start, a.n, (int)t0) : 0;
#pragma unroll
        for (int e = 0; e < 4; e++) {
            const int t = (int)min(t0 + e, (long long)INT_MAX);
            slot[e] = pos[e] = -1;
            if (t >= tokens || t >= a.max_tokens) continue;
            b = request_from(q.start, a.n, t, b);
            const unsigned x = (unsigned)q.have[b] + (unsigned)(t - q.start[b]), j = page_of(x, a);
            pos[e] = (int)min(x, (unsigned)INT_MAX);
            if (j >= (unsigned)a.width) continue;
            const int held = pages_of(q.have[b], a);
            int page = -1;
            if ((int)j < held) {
                page = a.table[(size_t)b * a.width + j];
            } else {
                const int src = n1 - 1 - (q.want[b] + (int)j - held);
                if (src >= 0) page = a.free_pages[src];
            }
            if (page >= 0 && page < most) slot[e] = page * a.P + (int)(x - j * a.P);
        }
        if (wide && t0 + 4 <= a.max_tokens) {
            *reinterpret_cast<int4 *>(a.slots + t0) = make_int4(slot[0], slot[1], slot[2], slot[3]);
            if (a.positions) *reinterpret_cast<int4 *>(a.positions + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
        } else {
            for (int e = 0; e < 4 && t0 + e < a.max_tokens; e++) {
                a.slots[t0 + e] = slot[e];
                if (a.positions) a.positions[t0 + e] = pos[e];
            }
        }
    }
}

// The pushes, and what there is one of; SMALL (one CTA): all of it.
template <bool SMALL, int T>
__global__ void __launch_bounds__(T) moe_pages_push_kernel(const PagesArgs a) {
    extern __shared__ int smem[];
    __shared__ Sums part[T / 32];
    __shared__ int wsum[T / 32], told[kCluster];
    __shared__ unsigned s_base;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int rank = 0, C = 1;
    if (!SMALL) {
        rank = (int)cg::this_cluster().block_rank(), C = (int)cg::this_cluster().num_blocks();
        asm volatile("barrier.cluster.arrive.relaxed.aligned;");   // waited for before the first write to another CTA
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // (after the wait: the second kernel reads the request lengths before its own)
    asm volatile("griddepcontrol.launch_dependents;");
    const Requests q(smem, a.n);
    const int n_free = min(max(a.counts[0], 0), a.cap);
    const Sums total = scan_requests<T>(a, q, part);
    // this CTA's entries, in order; kPer neighbours a thread at a time
    constexpr int kPer = SMALL ? 4 : 8;
    const int e0 = (int)((long long)total.back * rank / C), e1 = (int)((long long)total.back * (rank + 1) / C);
    auto load = [&](int x0, int (&id)[kPer]) {   // and how many are there
        int c = 0, b = x0 < e1 ? request_of(q.back, a.n, x0) : 0;
#pragma unroll
        for (int i = 0; i < kPer; i++) {
            id[i] = -1;
            if (i >= e1 - x0) continue;
            b = request_from(q.back, a.n, x0 + i, b);
            id[i] = a.table[(size_t)b * a.width + (x0 + i - q.back[b])];
            c += id[i] >= 0;
        }
        return c;
    };
    int id[kPer], got = 0;
    unsigned base = n_free, all = 0;   // places in the free list, with those past its end: up to 2^32 - 2
    const bool once = C > 1 && e1 - e0 <= kPer * T;   // what the first look loads is kept
    if (C > 1) {
        // entries that are there in each CTA's share
        int c = 0;
#pragma unroll
        for (int i = 0; i < kPer; i++) id[i] = -1;
        for (unsigned x = e0 + kPer * tid; x < (unsigned)e1; x += kPer * T) c += got = load((int)x, id);
        c = __reduce_add_sync(0xffffffffu, c);
        if (lane == 0) wsum[warp] = c;
        __syncthreads();
        c = __reduce_add_sync(0xffffffffu, lane < T / 32 ? wsum[lane] : 0);
        asm volatile("barrier.cluster.wait.aligned;" ::: "memory");   // every CTA runs
        if (tid < C) cg::this_cluster().map_shared_rank(told, tid)[rank] = c;
        cg::this_cluster().sync();
        for (int x = 0; x < C; x++) {
            if (x < rank) base += told[x];
            all += told[x];
        }
    }
    if (tid == 0) s_base = base;
    __syncthreads();
    for (unsigned x = e0; x < (unsigned)e1; x += kPer * T) {
        const int c = once ? got : load((int)min(x + kPer * tid, (unsigned)e1), id);
        int inc = c;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, inc, d);
            if (lane >= d) inc += o;
        }
        if (lane == 31) wsum[warp] = inc;
        __syncthreads();
        const int ws = lane < T / 32 ? wsum[lane] : 0;
        const int sum = __reduce_add_sync(0xffffffffu, ws);
        unsigned at = s_base + inc - c + __reduce_add_sync(0xffffffffu, lane < warp ? ws : 0);
#pragma unroll
        for (int i = 0; i < kPer; i++)
            if (id[i] >= 0) {
                if (at < (unsigned)a.cap) a.free_pages[at] = id[i];
                at++;
            }
        __syncthreads();
        if (tid == 0) s_base += sum;
        __syncthreads();
    }
    const int n1 = (int)min(C > 1 ? n_free + all : s_base, (unsigned)a.cap);
    if (rank == 0) {
        for (int b = tid; b < a.n; b += T) {
            a.starts[b] = q.start[b];
            a.lens[b] = q.fresh[b] < 0 ? 0 : clamp_int((long long)q.have[b] + q.fresh[b]);
        }
        if (tid == 0) {
            a.starts[a.n] = clamp_int(total.tok);
            const int left = n1 - total.want;
            a.counts_out[0] = max(left, 0);
            a.counts_out[1] = max(-left, 0);
        }
    }
    if (SMALL) fill(a, q, total, n1, tid, T);
}

__global__ void __launch_bounds__(kFillThreads) moe_pages_fill_kernel(const PagesArgs a) {
    extern __shared__ int smem[];
    __shared__ Sums part[kFillThreads / 32];
    const Requests q(smem, a.n);
    const Sums total = scan_requests<kFillThreads>(a, q, part);   // (the first kernel has waited for what this reads)
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    // the first kernel left counts_out = (free pages left, or 0; pages missing, or 0)
    const int n1 = a.counts_out[0] - a.counts_out[1] + total.want;
    fill(a, q, total, n1, blockIdx.x * kFillThreads + threadIdx.x, gridDim.x * kFillThreads);
}

cudaError_t pages_launch(const PagesArgs &a, cudaStream_t st) {
    const size_t smem = (size_t)a.n * 20;
    if (a.n <= kSmallSeqs && a.max_tokens <= kSmallTokens && (long long)a.n * a.width <= kSmallTable)
        return launch_pdl(moe_pages_push_kernel<true, kSmallThreads>, dim3(1), dim3(kSmallThreads), smem, st, a);
    static PerDevice<bool> push_opted, fill_opted;
    MOE_CUDA_TRY(smem_optin_once(moe_pages_push_kernel<false, kPushThreads>, push_opted));
    MOE_CUDA_TRY(smem_optin_once(moe_pages_fill_kernel, fill_opted));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kCluster);
    cfg.blockDim = dim3(kPushThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = kCluster, attr[1].val.clusterDim.y = 1, attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    MOE_CUDA_TRY(cudaLaunchKernelEx(&cfg, moe_pages_push_kernel<false, kPushThreads>, a));
    // four tokens a thread, at most four CTAs an SM of a 152-SM GPU
    const long long want = (a.max_tokens + 4ll * kFillThreads - 1) / (4ll * kFillThreads);
    const int grid = (int)std::min(std::max(want, 32ll), 608ll);
    return launch_pdl(moe_pages_fill_kernel, dim3(grid), dim3(kFillThreads), smem, st, a);
}

}  // namespace

extern "C" int moe_pages_assign(int page_size, int n_seqs, const int32_t *cached, const int32_t *fresh, int32_t *free_pages,
                                int capacity, const int32_t *counts, int32_t *counts_out, int32_t *table, int table_width,
                                int32_t *starts, int32_t *lens, int32_t *slots, int32_t *positions, int max_tokens,
                                void *stream) {
    if (page_size < 1 || page_size > 65536) return moe_fail_status(MOE_EINVAL, "page_size must be 1..65536");
    if (n_seqs < 0 || n_seqs > kMaxSeqs) return moe_fail_status(MOE_EINVAL, "n_seqs must be 0..%d", kMaxSeqs);
    if (capacity < 0 || table_width < 0 || max_tokens < 0)
        return moe_fail_status(MOE_EINVAL, "capacity, table_width and max_tokens must be >= 0");
    if ((long long)n_seqs * table_width > INT_MAX)
        return moe_fail_status(MOE_EINVAL, "a table of more than 2^31 - 1 entries");
    if (!counts || !counts_out || !starts || (n_seqs && (!cached || !fresh || !lens)) || (capacity && !free_pages) ||
        ((long long)n_seqs * table_width && !table) || (max_tokens && !slots))
        return moe_fail_status(MOE_EINVAL, "NULL argument");
    if (((uintptr_t)cached | (uintptr_t)fresh | (uintptr_t)free_pages | (uintptr_t)counts | (uintptr_t)counts_out |
         (uintptr_t)table | (uintptr_t)starts | (uintptr_t)lens | (uintptr_t)slots | (uintptr_t)positions) & 3u)
        return moe_fail_status(MOE_EINVAL, "pointers must be 4-byte aligned");
    for (const int32_t *in : {cached, fresh})
        if (n_seqs && ((in < lens + n_seqs && lens < in + n_seqs) || (in < starts + n_seqs + 1 && starts < in + n_seqs)))
            return moe_fail_status(MOE_EINVAL, "starts and lens must not overlap cached or fresh");
    int shift = -1;
    if ((page_size & (page_size - 1)) == 0)
        for (shift = 0; (1 << shift) < page_size; shift++) {
        }
    PagesArgs a{page_size, shift, n_seqs, table_width, capacity, max_tokens, cached, fresh, table, free_pages, counts, counts_out,
                starts, lens, slots, positions};
    const cudaError_t e = pages_launch(a, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? MOE_OK : moe_fail_status(MOE_ECUDA, "moe_pages_assign: %s", cudaGetErrorString(e));
}
