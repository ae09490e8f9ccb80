// moe_pages.cu -- block tables and slot maps of a paged cache, built on the
// GPU from request lengths: finished requests' pages go back to the free
// list, the others take what their new tokens need, and every new token gets
// its slot and position.
#include "moe_common.cuh"
#include "../../include/moe.h"

#include <climits>

namespace {

constexpr int kMaxSeqs = 4096;
constexpr int kThreads = 1024;
constexpr int kPer = kMaxSeqs / kThreads;  // requests a thread scans

struct PagesArgs {
    int P, n, width, cap, max_tokens;
    const int32_t *cached, *fresh;
    int32_t *table, *free_pages;
    const int32_t *counts;
    int32_t *counts_out, *starts, *lens, *slots, *positions;
};

// Exclusive block scan of three values a thread, and their sums.
struct Sum3 {
    int back, want;
    long long tok;
};
__device__ __forceinline__ Sum3 operator+(Sum3 a, Sum3 b) { return {a.back + b.back, a.want + b.want, a.tok + b.tok}; }
__device__ __forceinline__ Sum3 shfl_up(Sum3 v, int d) {
    return {__shfl_up_sync(0xffffffffu, v.back, d), __shfl_up_sync(0xffffffffu, v.want, d),
            __shfl_up_sync(0xffffffffu, v.tok, d)};
}
__device__ Sum3 block_scan(Sum3 v, Sum3 *part, Sum3 &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    Sum3 inc = v;
    for (int d = 1; d < 32; d <<= 1) {
        const Sum3 o = shfl_up(inc, d);
        if (lane >= d) inc = inc + o;
    }
    if (lane == 31) part[warp] = inc;
    __syncthreads();
    if (warp == 0) {
        Sum3 w = part[lane], own = w;
        for (int d = 1; d < 32; d <<= 1) {
            const Sum3 o = shfl_up(w, d);
            if (lane >= d) w = w + o;
        }
        part[lane] = {w.back - own.back, w.want - own.want, w.tok - own.tok};
        if (lane == 31) part[32] = w;
    }
    __syncthreads();
    total = part[32];
    const Sum3 base = part[warp];
    return {base.back + inc.back - v.back, base.want + inc.want - v.want, base.tok + inc.tok - v.tok};
}

__device__ __forceinline__ int pages_of(long long tokens, const PagesArgs &a) {
    return (int)min((tokens + a.P - 1) / a.P, (long long)a.width);
}
__device__ __forceinline__ int clamp_int(long long v) { return (int)min(v, (long long)INT_MAX); }

__global__ void __launch_bounds__(kThreads) moe_pages_kernel(const PagesArgs a) {
    __shared__ Sum3 part[33];
    // off: a finished request's page count, then the index of its first page
    // among those given back; of another request, among those taken
    __shared__ int off[kMaxSeqs];
    __shared__ int start[kMaxSeqs + 1];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int n_free = min(max(a.counts[0], 0), a.cap);
    // pages that finished requests give back (a warp a request; entries < 0 are none)
    for (int b = warp; b < a.n; b += kThreads / 32) {
        int c = 0;
        if (a.fresh[b] < 0) {
            const int held = pages_of(max(a.cached[b], 0), a);
            for (int j0 = 0; j0 < held; j0 += 32)
                c += __popc(__ballot_sync(0xffffffffu, j0 + lane < held && a.table[(size_t)b * a.width + j0 + lane] >= 0));
        }
        if (lane == 0) off[b] = c;
    }
    __syncthreads();
    auto counts_of = [&](int b) {
        const int have = max(a.cached[b], 0), f = a.fresh[b];
        Sum3 v = {0, 0, 0};
        if (f < 0) v.back = off[b];
        else v.want = pages_of((long long)have + f, a) - pages_of(have, a), v.tok = f;
        return v;
    };
    Sum3 sum = {0, 0, 0};
    const int b0 = tid * kPer, b1 = min(b0 + kPer, a.n);
    for (int b = b0; b < b1; b++) sum = sum + counts_of(b);
    Sum3 total, at = block_scan(sum, part, total);
    for (int b = b0; b < b1; b++) {
        const Sum3 v = counts_of(b);
        const int f = a.fresh[b];
        off[b] = f < 0 ? at.back : at.want, start[b] = clamp_int(at.tok);
        a.starts[b] = start[b];
        a.lens[b] = f < 0 ? 0 : clamp_int((long long)max(a.cached[b], 0) + f);
        at = at + v;
    }
    if (tid == 0) start[a.n] = a.starts[a.n] = clamp_int(total.tok);
    __syncthreads();
    for (int b = warp; b < a.n; b += kThreads / 32) {
        if (a.fresh[b] >= 0) continue;
        const int held = pages_of(max(a.cached[b], 0), a);
        int to = n_free + off[b];
        for (int j0 = 0; j0 < held; j0 += 32) {
            const int id = j0 + lane < held ? a.table[(size_t)b * a.width + j0 + lane] : -1;
            const unsigned m = __ballot_sync(0xffffffffu, id >= 0);
            const int k = to + __popc(m & ((1u << lane) - 1));
            if (id >= 0 && k < a.cap) a.free_pages[k] = id;
            to += __popc(m);
        }
    }
    __syncthreads();
    const int n1 = min(n_free + total.back, a.cap);
    for (int b = warp; b < a.n; b += kThreads / 32) {
        const int f = a.fresh[b], have = max(a.cached[b], 0);
        if (f <= 0) continue;
        const int held = pages_of(have, a), w = pages_of((long long)have + f, a) - held;
        for (int j = lane; j < w; j += 32) {
            const int src = n1 - 1 - (off[b] + j);
            a.table[(size_t)b * a.width + held + j] = src >= 0 ? a.free_pages[src] : -1;
        }
    }
    __syncthreads();
    if (tid == 0) {
        const int left = n1 - total.want;
        a.counts_out[0] = max(left, 0);
        a.counts_out[1] = max(-left, 0);
    }
    for (int t = tid; t < a.max_tokens; t += kThreads) {
        int slot = -1, pos = -1;
        if (t < start[a.n]) {
            int lo = 0, hi = a.n;  // the last request that starts at or before t
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (start[mid] <= t) lo = mid;
                else hi = mid;
            }
            const long long p = (long long)max(a.cached[lo], 0) + (t - start[lo]);
            pos = clamp_int(p);
            if (p / a.P < a.width) {
                const int page = a.table[(size_t)lo * a.width + p / a.P];
                if (page >= 0 && page < INT_MAX / a.P) slot = page * a.P + (int)(p % a.P);
            }
        }
        a.slots[t] = slot;
        if (a.positions) a.positions[t] = pos;
    }
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
    if (n_seqs && cached < lens + n_seqs && lens < cached + n_seqs)
        return moe_fail_status(MOE_EINVAL, "lens must not overlap cached");
    PagesArgs a{page_size, n_seqs, table_width, capacity, max_tokens, cached, fresh, table, free_pages, counts, counts_out,
                starts, lens, slots, positions};
    const cudaError_t e = launch_pdl(moe_pages_kernel, dim3(1), dim3(kThreads), 0, static_cast<cudaStream_t>(stream), a);
    return e == cudaSuccess ? MOE_OK : moe_fail_status(MOE_ECUDA, "moe_pages_assign: %s", cudaGetErrorString(e));
}
