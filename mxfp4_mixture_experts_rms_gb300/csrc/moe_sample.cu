// moe_sample.cu -- the next token of each row of logits: temperature, top-k,
// top-p and min-p, then the inverse of the cumulative distribution (in index
// order) at a given random number.
//
// With M the row's largest logit, a token's weight is w = e^((l - M) / t),
// 1 for l = M.  top-k keeps the k first in descending order (equal logits: the
// lower index first), top-p of those the shortest prefix whose weights reach p
// of theirs, min-p of those the ones with w >= min_p.  No sort is needed: the
// kept set is "key above T, and the first r with key T", and T comes from
// radix selection over the logits' order-preserving 32-bit keys, by count for
// top-k and by weight for top-p.  Weights are summed as whole multiples of
// 2^-40, so that sums do not depend on their order.
#include "moe_common.cuh"
#include "../../include/moe.h"

#include <climits>

namespace {

typedef unsigned long long u64;
constexpr int kThreads = 1024;

struct SampleArgs {
    const void *x;
    int bf16, rows, V;
    long long stride;
    const float *temperature;
    const int32_t *top_k;
    const float *top_p, *min_p, *u;
    int32_t *ids;
};

// Larger logit, larger key; NaN and -inf (never chosen): 0.
__device__ __forceinline__ uint32_t order_key(float l) {
    if (!(l > -INFINITY)) return 0;
    const uint32_t b = __float_as_uint(l + 0.f);  // -0 becomes +0
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float key_logit(uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k);
}
__device__ __forceinline__ float load_logit(const SampleArgs &a, int row, int i) {
    return a.bf16 ? bf16_to_f32(static_cast<const uint16_t *>(a.x)[row * a.stride + i])
                  : static_cast<const float *>(a.x)[row * a.stride + i];
}
__device__ __forceinline__ float weight(float l, float top, float t) {
    return l == top ? 1.f : (t > 0.f ? expf((l - top) / t) : 0.f);
}
__device__ __forceinline__ u64 fixed(float w) { return (u64)((double)w * 0x1p40 + 0.5); }

// The largest T such that what lies above T is less than `goal`: by count, or
// by weight (among keys above `floor_key`, `ties` of those equal to it).
// above: count / weight of the keys above T.
__device__ uint32_t radix_select(const SampleArgs &a, int row, float top, float t, bool by_weight, u64 goal,
                                 uint32_t floor_key, u64 *hist, u64 &above) {
    uint32_t prefix = 0;
    above = 0;
    __shared__ u64 s_above;
    __shared__ int s_digit;
    for (int shift = 24; shift >= 0; shift -= 8) {
        for (int i = threadIdx.x; i < 256; i += kThreads) hist[i] = 0;
        __syncthreads();
        for (int i = threadIdx.x; i < a.V; i += kThreads) {
            const float l = load_logit(a, row, i);
            const uint32_t k = order_key(l);
            if (k == 0 || k <= floor_key || (shift < 24 && (k >> (shift + 8)) != (prefix >> (shift + 8)))) continue;
            atomicAdd(&hist[(k >> shift) & 255], by_weight ? fixed(weight(l, top, t)) : 1ull);
        }
        __syncthreads();
        if (threadIdx.x == 0) {
            u64 s = above;
            int d = 255;
            for (; d > 0 && s + hist[d] < goal; d--) s += hist[d];
            s_above = s, s_digit = d;
        }
        __syncthreads();
        above = s_above;
        prefix |= (uint32_t)s_digit << shift;
        __syncthreads();
    }
    return prefix;
}

__global__ void __launch_bounds__(kThreads) moe_sample_kernel(const SampleArgs a) {
    __shared__ u64 hist[256];
    __shared__ u64 part[kThreads / 32], s_total, s_base;
    __shared__ uint32_t kmax[kThreads / 32];
    __shared__ int ties[kThreads / 32], s_ties, s_id, s_last;
    const int row = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    uint32_t km = 0;
    for (int i = tid; i < a.V; i += kThreads) km = max(km, order_key(load_logit(a, row, i)));
    km = __reduce_max_sync(0xffffffffu, km);
    if (lane == 0) kmax[warp] = km;
    __syncthreads();
    for (int w = 0; w < kThreads / 32; w++) km = max(km, kmax[w]);
    if (km == 0) {
        if (tid == 0) a.ids[row] = -1;
        return;
    }
    const float top = key_logit(km), t = a.temperature ? fminf(a.temperature[row], 3.402823466e38f) : 1.f;
    const bool greedy = !(t > 0.f);
    long long k = a.top_k ? a.top_k[row] : 0;
    const float p = a.top_p ? a.top_p[row] : 1.f, mp = a.min_p ? fminf(a.min_p[row], 1.f) : 0.f;
    // kept: keys above T, and the first r tokens whose key is T
    uint32_t T = 0;
    u64 r = 0, above;
    if (greedy) {
        T = km, r = 1;
    } else {
        if (k > 0 && k < a.V) {
            T = radix_select(a, row, top, t, false, (u64)k, 0, hist, above);
            r = T ? (u64)k - above : 0;
            if (T == 0) r = 0;
        }
        if (p < 1.f) {
            // weight of what top-k left
            u64 sum = 0;
            for (int i = tid; i < a.V; i += kThreads) {
                const float l = load_logit(a, row, i);
                if (order_key(l) > T) sum += fixed(weight(l, top, t));
            }
            for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
            if (lane == 0) part[warp] = sum;
            __syncthreads();
            sum = 0;
            for (int w = 0; w < kThreads / 32; w++) sum += part[w];
            __syncthreads();
            const u64 wt = T ? fixed(weight(key_logit(T), top, t)) : 0;
            // a token stays while the weight before it is less than p of the
            // whole: the prefix that reaches goal (at least one token)
            const u64 goal = max((u64)ceil((double)fmaxf(p, 0.f) * (double)(sum + r * wt)), 1ull);
            if (sum >= goal) {
                T = radix_select(a, row, top, t, true, goal, T, hist, above);
                const u64 w = fixed(weight(key_logit(T), top, t));
                r = w ? (goal - above + w - 1) / w : 1;
            } else if (T && wt) {
                r = min(r, (goal - sum + wt - 1) / wt);  // among the tokens at T
            }
        }
    }
    // total of the kept, then the token where the running sum passes u * total
    for (int pass = 0; pass < 2; pass++) {
        if (tid == 0) s_base = 0, s_ties = 0, s_id = INT_MAX, s_last = -1;
        __syncthreads();
        const u64 target = pass ? (u64)((double)a.u[row] * (double)s_total) : 0;
        for (int i0 = 0; i0 < a.V; i0 += kThreads) {
            const int i = i0 + tid;
            const float l = i < a.V ? load_logit(a, row, i) : -INFINITY;
            const uint32_t key = order_key(l);
            const unsigned tm = __ballot_sync(0xffffffffu, key != 0 && key == T);
            if (lane == 0) ties[warp] = __popc(tm);
            __syncthreads();
            int tb = s_ties, all = 0;
            for (int w = 0; w < kThreads / 32; w++) {
                if (w < warp) tb += ties[w];
                all += ties[w];
            }
            bool keep = key > T || (key != 0 && key == T && (u64)(tb + __popc(tm & ((1u << lane) - 1))) < r);
            const float w = weight(l, top, t);
            keep = keep && w >= mp;
            u64 m = keep ? fixed(w) : 0, inc = m;
            for (int d = 1; d < 32; d <<= 1) {
                const u64 o = __shfl_up_sync(0xffffffffu, inc, d);
                if (lane >= d) inc += o;
            }
            if (lane == 31) part[warp] = inc;
            __syncthreads();
            u64 base = s_base, sum = 0;
            for (int w2 = 0; w2 < kThreads / 32; w2++) {
                if (w2 < warp) base += part[w2];
                sum += part[w2];
            }
            if (pass && m && base + inc > target) atomicMin(&s_id, i);
            if (pass && m) atomicMax(&s_last, i);
            __syncthreads();
            if (tid == 0) s_base += sum, s_ties += all;
            __syncthreads();
            if (pass && s_id != INT_MAX) break;
        }
        if (tid == 0 && !pass) s_total = s_base;
        __syncthreads();
    }
    if (tid == 0) a.ids[row] = s_id != INT_MAX ? s_id : s_last;
}

}  // namespace

extern "C" int moe_sample(const void *logits, int is_bf16, int n_rows, int vocab, long long row_stride,
                          const float *temperature, const int32_t *top_k, const float *top_p, const float *min_p,
                          const float *u, int32_t *ids, void *stream) {
    if (n_rows < 0 || vocab < 1 || vocab > (1 << 24))
        return moe_fail_status(MOE_EINVAL, "n_rows must be >= 0 and vocab 1..2^24");
    if (is_bf16 != 0 && is_bf16 != 1) return moe_fail_status(MOE_EINVAL, "is_bf16 must be 0 or 1");
    if (n_rows == 0) return MOE_OK;
    if (!logits || !u || !ids) return moe_fail_status(MOE_EINVAL, "NULL logits, u or ids");
    if (row_stride < vocab) return moe_fail_status(MOE_EINVAL, "row_stride must be at least vocab");
    if ((uintptr_t)logits & (is_bf16 ? 1u : 3u)) return moe_fail_status(MOE_EINVAL, "misaligned logits");
    if (((uintptr_t)temperature | (uintptr_t)top_k | (uintptr_t)top_p | (uintptr_t)min_p | (uintptr_t)u | (uintptr_t)ids) & 3u)
        return moe_fail_status(MOE_EINVAL, "pointers must be 4-byte aligned");
    SampleArgs a{logits, is_bf16, n_rows, vocab, row_stride, temperature, top_k, top_p, min_p, u, ids};
    const cudaError_t e = launch_pdl(moe_sample_kernel, dim3(n_rows), dim3(kThreads), 0, static_cast<cudaStream_t>(stream), a);
    return e == cudaSuccess ? MOE_OK : moe_fail_status(MOE_ECUDA, "moe_sample: %s", cudaGetErrorString(e));
}
