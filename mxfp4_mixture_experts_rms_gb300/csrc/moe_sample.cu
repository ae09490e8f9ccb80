// moe_sample.cu -- the next token of each row of logits: temperature, top-k,
// top-p and min-p, then the inverse of the cumulative distribution (in index
// order) at a given random number.
//
// With M the row's largest logit, a token's weight is w = e^((l - M) / t),
// 1 for l = M.  top-k keeps the k first in descending order (equal logits: the
// lower index first), top-p of those the shortest prefix whose weights reach p
// of theirs, min-p of those the ones with w >= min_p.  Nothing is sorted: the
// kept set is "logit above T, and the first r tokens with logit T", so T and r
// are looked for, by count for top-k and by weight for top-p:
//  1. a histogram of 512 bins of equal width in log2 w (24 powers of two; what
//     is below is not counted) finds the bin that holds T; counts are exact,
//     weights here 32-bit fixed point relative to the bin's upper edge;
//  2. one more pass sums what lies above that bin exactly and lists the bin's
//     logits;
//  3. the list is cut by histograms over the logits' order-preserving 32-bit
//     keys until one key is left.
// Where a bin's list does not fit, where T lies below the 24 powers of two, or
// where step 1's rounding named a neighbour of T's bin, step 3 runs over the
// row instead.  Weights are summed as whole multiples of 2^-40, so sums do not
// depend on their order.
//
// A row is a cluster's: each CTA keeps its part in shared memory (read from
// memory once) where it fits, and meets the others through distributed shared
// memory.  Bound by HBM for large batches in principle (2 or 4 bytes a
// logit); what it spends its time on is the instructions of the passes.
#include "moe_common.cuh"
#include "../../include/moe.h"

#include <cooperative_groups.h>

#include <algorithm>
#include <climits>

namespace cg = cooperative_groups;

namespace {

typedef unsigned long long u64;
constexpr int kBins = 512;
constexpr int kMaxCluster = 8;
constexpr int kList = 2048;           // keys listed by a CTA
constexpr float kSpan = 24.f;         // powers of two that the first histogram covers
constexpr float kLog2e = 1.4426950408889634f;

struct SampleArgs {
    const void *x;
    int rows, V;
    long long stride;
    const float *temperature;
    const int32_t *top_k;
    const float *top_p, *min_p, *u;
    int32_t *ids;
    int seg;         // 16-byte vectors of a row's part
    float bin_unit;  // weight units of the first histogram: 2^30 / (the power of two <= V)
};

// Larger logit, larger key; NaN and -inf (never chosen): 0.
__device__ __forceinline__ uint32_t order_key(float l) {
    const uint32_t b = __float_as_uint(l + 0.f);  // -0 becomes +0
    return l > -INFINITY ? (b & 0x80000000u ? ~b : b | 0x80000000u) : 0u;
}
__device__ __forceinline__ float key_logit(uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k);
}
// A weight (0 .. 1) in units of 2^-40, by its bits.
__device__ __forceinline__ u64 fixed40(float w) {
    const uint32_t b = __float_as_uint(w);
    const int s = (int)(b >> 23) - 110;   // mantissa times 2^(exponent - 150) = units of 2^-40 times 2^s
    const uint32_t m = (b & 0x7FFFFFu) | 0x800000u;
    return s >= 0 ? (u64)m << s : (u64)(m >> min(-s, 31));
}

// What the CTAs of a row tell one another, each its slot.
struct Told {
    uint32_t key;
    int n, ties;
    u64 sum;
};

template <bool BF16, bool RES, int NT>
struct Row {
    static constexpr int VE = BF16 ? 8 : 4;   // logits of a 16-byte vector
    const uint4 *g;       // the row's vectors in memory, from the one that holds its first logit
    const uint4 *s;       // this CTA's in shared memory (RES)
    int off, V;           // logits of the first vector that are not the row's; the row's logits
    int v0, v1;           // this warp's vectors
    int c0;               // the CTA's first vector

    __device__ __forceinline__ uint4 fetch(int v) const {   // from memory, -inf outside the row
        const int i = v * VE - off;
        if (i >= 0 && i + VE <= V) return __ldg(g + v);
        uint32_t w[4];
#pragma unroll
        for (int q = 0; q < 4; q++) {
            if (BF16) {
                const uint16_t *p = reinterpret_cast<const uint16_t *>(g) + (size_t)v * VE + 2 * q;
                const uint32_t lo = i + 2 * q >= 0 && i + 2 * q < V ? p[0] : 0xFF80u;
                const uint32_t hi = i + 2 * q + 1 >= 0 && i + 2 * q + 1 < V ? p[1] : 0xFF80u;
                w[q] = lo | hi << 16;
            } else {
                w[q] = i + q >= 0 && i + q < V ? reinterpret_cast<const uint32_t *>(g)[(size_t)v * VE + q] : 0xFF800000u;
            }
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    static __device__ __forceinline__ void values(uint4 w, float (&x)[VE]) {
        const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int q = 0; q < 4; q++) {
            if (BF16) {
                x[2 * q] = __uint_as_float(a[q] << 16), x[2 * q + 1] = __uint_as_float(a[q] & 0xFFFF0000u);
            } else {
                x[q] = __uint_as_float(a[q]);
            }
        }
    }
    __device__ __forceinline__ uint4 vec(int v) const { return RES ? s[v - c0] : fetch(v); }
    // f(logits, first one's index) for the warp's vectors, a lane a vector; in order of index
    template <class F>
    __device__ __forceinline__ void each(F f) const {
        for (int v = v0 + (threadIdx.x & 31); v < v1; v += 32) {
            float x[VE];
            values(vec(v), x);
            f(x, v * VE - off);
        }
    }
};

template <bool BF16, bool RES, int NT>
__global__ void __launch_bounds__(NT, 1024 / NT) moe_sample_kernel(const SampleArgs a) {
    typedef Row<BF16, RES, NT> R;
    constexpr int VE = R::VE, NW = NT / 32;
    extern __shared__ __align__(16) uint4 data[];
    __shared__ u64 hist[kBins];
    __shared__ uint32_t hist32[kBins];
    __shared__ uint32_t list[kList];
    __shared__ Told told[2][kMaxCluster];
    __shared__ u64 part[NW], s_above, wmass[NW];
    __shared__ uint32_t red[NW], s_lo, s_hi;
    __shared__ int s_bin, s_n, wties[NW];
    cg::cluster_group cl = cg::this_cluster();
    const int rank = (int)cl.block_rank(), C = (int)cl.num_blocks();
    const int row = blockIdx.x / C, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");

    R d;
    {
        const uintptr_t at = (uintptr_t)a.x + (size_t)row * a.stride * (BF16 ? 2 : 4);
        d.g = reinterpret_cast<const uint4 *>(at & ~(uintptr_t)15);
        d.off = (int)(at & 15) / (BF16 ? 2 : 4);
        d.V = a.V;
        d.s = data;
        const int all = (d.off + a.V + VE - 1) / VE;
        d.c0 = min(rank * a.seg, all);
        const int c1 = min(d.c0 + a.seg, all), per = (c1 - d.c0 + NW - 1) / NW;
        d.v0 = min(d.c0 + warp * per, c1), d.v1 = min(d.v0 + per, c1);
    }
    const float t = a.temperature ? fminf(a.temperature[row], 3.402823466e38f) : 1.f;
    const int k = a.top_k ? a.top_k[row] : 0;
    const float p = a.top_p ? a.top_p[row] : 1.f, mp = a.min_p ? fminf(a.min_p[row], 1.f) : 0.f;
    const float u = a.u[row];
    int turn = 0;
    // every CTA's value to every CTA; all of them are there after it
    auto tell = [&](Told mine) {
        turn ^= 1;
        if (tid < C) *cl.map_shared_rank(&told[turn][rank], tid) = mine;
        cl.sync();
    };

    // the row's largest logit, while its part comes in
    uint32_t km = 0;
    for (int v = d.v0 + lane; v < d.v1; v += 128) {   // four vectors a lane on their way
        uint4 w[4];
#pragma unroll
        for (int q = 0; q < 4; q++)
            if (v + 32 * q < d.v1) w[q] = d.fetch(v + 32 * q);
#pragma unroll
        for (int q = 0; q < 4; q++)
            if (v + 32 * q < d.v1) {
                if (RES) data[v + 32 * q - d.c0] = w[q];
                float x[VE], m = -INFINITY;
                R::values(w[q], x);
#pragma unroll
                for (int e = 0; e < VE; e++) m = fmaxf(m, x[e]);   // NaN passes over
                km = max(km, order_key(m));
            }
    }
    km = __reduce_max_sync(0xffffffffu, km);
    if (lane == 0) red[warp] = km;
    __syncthreads();
    km = __reduce_max_sync(0xffffffffu, red[lane % NW]);
    tell({km, 0, 0, 0});
    for (int c = 0; c < C; c++) km = max(km, told[turn][c].key);
    if (km == 0) {   // nothing to choose
        if (rank == 0 && tid == 0) a.ids[row] = -1;
        return;
    }
    const float top = key_logit(km), scale = kLog2e / t;
    // kept: keys above T, and the first r tokens whose key is T
    uint32_t T = 0;
    u64 r = 0;
    if (!(t > 0.f)) {
        T = km, r = 1;
    } else {
        auto log2w = [&](float x) { return x == top ? 0.f : (x - top) * scale; };
        auto weight = [&](float x) {
            float w;
            asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(w) : "f"(log2w(x)));
            return w;
        };
        constexpr float kPerBin = kSpan / kBins;
        auto bin_of = [&](float x) { return log2w(x) * (-1.f / kPerBin); };   // truncated: 0 holds the largest
        // block-wide: the first bin whose inclusive sum of h (one a thread, kBins of them) reaches goal
        auto find = [&](u64 h, u64 goal) {
            u64 inc = h;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const u64 y = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += y;
            }
            if (lane == 31 && warp < kBins / 32) part[warp] = inc;
            if (tid == 0) s_bin = -1;
            __syncthreads();
            if (tid < kBins) {
                for (int w = 0; w < warp; w++) inc += part[w];
                if (inc >= goal && inc - h < goal) s_bin = tid, s_above = inc - h;
            }
            __syncthreads();
            return s_bin;
        };
        // block-wide sum
        auto total = [&](u64 v) {
#pragma unroll
            for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
            __syncthreads();
            if (lane == 0) part[warp] = v;
            __syncthreads();
            v = 0;
            for (int w = 0; w < NW; w++) v += part[w];
            return v;
        };
        for (int stage = 0; stage < 2; stage++) {
            const bool by_weight = stage == 1;
            if (by_weight ? !(p < 1.f) : !(k > 0 && k < a.V)) continue;
            const float over = T ? key_logit(T) : -INFINITY;   // what top-k left lies above, and r tokens at it
            // 1. the histogram, and the weight of all
            __syncthreads();
            for (int b = tid; b < kBins; b += NT) hist32[b] = 0;
            __syncthreads();
            float sum = 0.f;
            d.each([&](float (&x)[VE], int) {
#pragma unroll
                for (int e = 0; e < VE; e++) {
                    if (!(x[e] > over)) continue;
                    const float f = bin_of(x[e]);
                    float w = 1.f;
                    if (by_weight) {
                        w = weight(x[e]);
                        sum += w;
                    }
                    if (f < (float)(kBins - 1)) {
                        const int b = (int)f;
                        uint32_t add = 1;
                        if (by_weight) {
                            asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(w) : "f"(fmaf((float)b, kPerBin, log2w(x[e]))));
                            add = (uint32_t)fmaf(w, a.bin_unit, 0.5f);
                        }
                        atomicAdd(&hist32[b], add);
                    }
                }
            });
            u64 goal = (u64)k, all = 0;
            u64 mine = 0;
            if (by_weight) {
                // fp32 over a lane's logits, then whole multiples of 2^-40
                mine = total((u64)(sum * 0x1p40f));
            }
            tell({0, 0, 0, mine});   // and the histograms are there
            const u64 at_T = T ? fixed40(weight(key_logit(T))) : 0;
            if (by_weight) {
                for (int c = 0; c < C; c++) all += told[turn][c].sum;
                goal = max((u64)ceil((double)fmaxf(p, 0.f) * (double)(all + r * at_T)), (u64)1);
                if (goal > all && T) {   // among the tokens at T
                    if (at_T) r = min(r, (goal - all + at_T - 1) / at_T);
                    cl.sync();           // the histograms are read no more
                    continue;
                }
            }
            u64 h = 0;
            if (tid < kBins) {
                for (int c = 0; c < C; c++) h += cl.map_shared_rank(hist32, c)[tid];
                if (by_weight) {
                    float w;
                    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(w) : "f"(-(float)tid * kPerBin));
                    h = (u64)((float)h / a.bin_unit * w * 0x1p40f);
                }
            }
            int bin = find(h, goal);
            // 2. what lies above the bin, exactly, and the bin's keys
            u64 above = 0;
            uint32_t lo = 1, hi = km;   // T is among these keys
            bool listed = false;
            if (bin >= 0) {
                if (tid == 0) s_n = 0;
                __syncthreads();
                u64 before = 0;
                d.each([&](float (&x)[VE], int) {
#pragma unroll
                    for (int e = 0; e < VE; e++) {
                        const float f = bin_of(x[e]);
                        if (!(x[e] > over) || !(f < (float)(bin + 1))) continue;
                        if (f < (float)bin) {
                            before += by_weight ? fixed40(weight(x[e])) : 1;
                        } else {
                            const int at = atomicAdd(&s_n, 1);
                            if (at < kList) list[at] = order_key(x[e]);
                        }
                    }
                });
                before = total(before);
                tell({0, s_n, 0, before});
                listed = true;
                for (int c = 0; c < C; c++) above += told[turn][c].sum, listed = listed && told[turn][c].n <= kList;
                listed = listed && above < goal;
                if (!listed) above = 0;   // the whole row decides, from its first key on
            } else {
                cl.sync();   // the histograms are read no more
            }
            // 3. by keys: of the lists (all of them read by every CTA), else of the row
            if (listed) {
                if (tid == 0) s_lo = 0xFFFFFFFFu, s_hi = 0;
                __syncthreads();
                uint32_t l = 0xFFFFFFFFu, m = 0;
                for (int c = 0; c < C; c++) {
                    const uint32_t *q = cl.map_shared_rank(list, c);
                    for (int i = tid; i < told[turn][c].n; i += NT) l = min(l, q[i]), m = max(m, q[i]);
                }
                l = __reduce_min_sync(0xffffffffu, l), m = __reduce_max_sync(0xffffffffu, m);
                if (lane == 0) atomicMin(&s_lo, l), atomicMax(&s_hi, m);
                __syncthreads();
                lo = s_lo, hi = s_hi;
            }
            const int listed_turn = turn;
            for (bool again = true; again;) {
                u64 base = above;
                again = false;
                for (;;) {
                    const int shift = max(0, 32 - __clz((hi - lo) | 1) - 9);
                    __syncthreads();
                    for (int b = tid; b < kBins; b += NT) hist[b] = 0;
                    __syncthreads();
                    auto count = [&](uint32_t key) {
                        if (key >= lo && key <= hi)
                            atomicAdd(&hist[(hi - key) >> shift], by_weight ? fixed40(weight(key_logit(key))) : 1ull);
                    };
                    if (listed) {
                        for (int c = 0; c < C; c++) {
                            const uint32_t *q = cl.map_shared_rank(list, c);
                            for (int i = tid; i < told[listed_turn][c].n; i += NT) count(q[i]);
                        }
                        __syncthreads();
                        h = tid < kBins ? hist[tid] : 0;
                    } else {
                        d.each([&](float (&x)[VE], int) {
#pragma unroll
                            for (int e = 0; e < VE; e++)
                                if (x[e] > over) count(order_key(x[e]));
                        });
                        cl.sync();
                        h = 0;
                        if (tid < kBins)
                            for (int c = 0; c < C; c++) h += cl.map_shared_rank(hist, c)[tid];
                    }
                    bin = find(h, goal - base);
                    if (!listed) cl.sync();
                    if (bin < 0) break;
                    base += s_above;
                    const uint32_t width = (1u << shift) - 1, top_key = hi - ((uint32_t)bin << shift);
                    lo = max(lo, top_key - min(width, top_key)), hi = top_key;
                    if (shift == 0) break;
                }
                if (bin >= 0) {
                    T = hi;
                    const u64 w = by_weight ? fixed40(weight(key_logit(T))) : 1;
                    r = w ? (goal - base + w - 1) / w : 1;
                } else if (listed) {   // the bin falls short: a neighbour of it was named; the whole row decides
                    listed = false, again = true, above = 0, lo = 1, hi = km;
                    cl.sync();
                } else {
                    if (!by_weight) T = 0, r = 0;   // fewer than k tokens; or a goal beyond the rounding of the sum: all
                }
            }
            cl.sync();   // lists and histograms are read no more
        }
    }

    // the kept weight of each warp's part, and its tokens at T
    const float xT = T ? key_logit(T) : -INFINITY;
    const float sc = t > 0.f ? scale : 0.f;
    auto weight = [&](float x) {
        float w;
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(w) : "f"(x == top ? 0.f : (x - top) * sc));
        return w;
    };
    const float wT = T ? weight(xT) : 0.f;
    const u64 fT = wT >= mp ? fixed40(wT) : 0;
    u64 mass = 0;
    int ties = 0;
    d.each([&](float (&x)[VE], int) {
#pragma unroll
        for (int e = 0; e < VE; e++) {
            if (x[e] > xT) {
                const float w = weight(x[e]);
                if (w >= mp) mass += fixed40(w);
            } else if (T && x[e] == xT) {
                ties++;
            }
        }
    });
#pragma unroll
    for (int o = 16; o; o >>= 1) mass += __shfl_xor_sync(0xffffffffu, mass, o);
    ties = __reduce_add_sync(0xffffffffu, ties);
    if (lane == 0) wmass[warp] = mass, wties[warp] = ties;
    __syncthreads();
    mass = 0, ties = 0;
    for (int w = 0; w < NW; w++) mass += wmass[w], ties += wties[w];
    tell({0, 0, ties, mass});
    // in order of index: kept weight before each CTA, warp, vector, logit
    u64 sum = 0, base = 0, tb = 0, tsum = 0, own = 0;
    for (int c = 0; c < C; c++) {
        const u64 ct = told[turn][c].ties, keep_t = tsum < r ? min(r - tsum, ct) : 0;
        const u64 m = told[turn][c].sum + keep_t * fT;
        if (c == rank) base = sum, tb = tsum, own = m;
        sum += m, tsum += ct;
    }
    u64 target = (u64)((double)u * (double)sum);   // the first token whose running sum exceeds u times the total
    if (target >= sum) target = sum - 1;           // (u = 1 - 2^-24 rounds up to the total at most)
    if (target < base || target >= base + own) return;
    for (int w = 0; w < NW; w++) {
        const u64 ct = wties[w], keep_t = tb < r ? min(r - tb, ct) : 0, m = wmass[w] + keep_t * fT;
        if (target < base + m) {
            if (w != warp) return;
            break;
        }
        base += m, tb += ct;
    }
    // this warp's: 32 vectors at a time
    for (int v = d.v0; v < d.v1; v += 32) {
        float x[VE];
        int mt = 0;
        u64 m = 0;
        if (v + lane < d.v1) {
            R::values(d.vec(v + lane), x);
        } else {
#pragma unroll
            for (int e = 0; e < VE; e++) x[e] = -INFINITY;
        }
#pragma unroll
        for (int e = 0; e < VE; e++) mt += T && x[e] == xT;
        int it = mt;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, it, o);
            if (lane >= o) it += y;
        }
        u64 rt = tb + it - mt;   // tokens at T before this lane's
        u64 we[VE];
#pragma unroll
        for (int e = 0; e < VE; e++) {
            we[e] = 0;
            if (x[e] > xT) {
                const float w = weight(x[e]);
                we[e] = w >= mp ? fixed40(w) : 0;
            } else if (T && x[e] == xT) {
                we[e] = rt++ < r ? fT : 0;
            }
            m += we[e];
        }
        u64 inc = m;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const u64 y = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += y;
        }
        u64 run = base + inc - m;
        if (target >= run && target < run + m) {
            int id = 0;
#pragma unroll
            for (int e = 0; e < VE; e++) {
                if (target >= run && target < run + we[e]) id = (v + lane) * VE - d.off + e;
                run += we[e];
            }
            a.ids[row] = id;
        }
        base += __shfl_sync(0xffffffffu, inc, 31);
        tb += __shfl_sync(0xffffffffu, it, 31);
        if (target < base) break;
    }
}

template <bool BF16, bool RES, int NT>
cudaError_t sample_launch(const SampleArgs &a, int C, size_t smem, cudaStream_t st) {
    static PerDevice<bool> opted;
    cudaError_t e = smem_optin_once(moe_sample_kernel<BF16, RES, NT>, opted);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)a.rows * C);
    cfg.blockDim = dim3(NT);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = C, attr[1].val.clusterDim.y = 1, attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, moe_sample_kernel<BF16, RES, NT>, a);
}

template <bool BF16>
cudaError_t sample_plan(SampleArgs a, cudaStream_t st) {
    const int VE = BF16 ? 8 : 4;
    const long long vecs = ((long long)a.V + VE - 1) / VE + 1;   // one more where the first is cut
    // CTAs of a row: as many as give a large GPU two a multiprocessor, each
    // with at least 256 vectors; more where a part must fit shared memory
    int C = 1;
    while (C < kMaxCluster && ((long long)a.rows * C < 152 && vecs / C > 256 || vecs * 16 / C > 100000)) C *= 2;
    a.seg = (int)((vecs + C - 1) / C);
    const size_t smem = (size_t)a.seg * 16;
    float unit = 256.f;   // 2^30 / 2^22
    for (int b = 1 << 22; b > a.V && b > 2; b >>= 1) unit *= 2.f;
    a.bin_unit = unit;
    const bool wide = (long long)a.rows * C <= 152;
    if (smem > 190000) return sample_launch<BF16, false, 1024>(a, C, 0, st);
    return wide ? sample_launch<BF16, true, 1024>(a, C, smem, st) : sample_launch<BF16, true, 512>(a, C, smem, st);
}

}  // namespace

extern "C" int moe_sample(const void *logits, int is_bf16, int n_rows, int vocab, long long row_stride,
                          const float *temperature, const int32_t *top_k, const float *top_p, const float *min_p,
                          const float *u, int32_t *ids, void *stream) {
    if (n_rows < 0 || n_rows > (1 << 24) || vocab < 1 || vocab > (1 << 22))
        return moe_fail_status(MOE_EINVAL, "n_rows must be 0..2^24 and vocab 1..2^22");
    if (is_bf16 != 0 && is_bf16 != 1) return moe_fail_status(MOE_EINVAL, "is_bf16 must be 0 or 1");
    if (n_rows == 0) return MOE_OK;
    if (!logits || !u || !ids) return moe_fail_status(MOE_EINVAL, "NULL logits, u or ids");
    if (row_stride < vocab) return moe_fail_status(MOE_EINVAL, "row_stride must be at least vocab");
    if ((uintptr_t)logits & (is_bf16 ? 1u : 3u)) return moe_fail_status(MOE_EINVAL, "misaligned logits");
    if (((uintptr_t)temperature | (uintptr_t)top_k | (uintptr_t)top_p | (uintptr_t)min_p | (uintptr_t)u | (uintptr_t)ids) & 3u)
        return moe_fail_status(MOE_EINVAL, "pointers must be 4-byte aligned");
    SampleArgs a{};
    a.x = logits, a.rows = n_rows, a.V = vocab, a.stride = row_stride;
    a.temperature = temperature, a.top_k = top_k, a.top_p = top_p, a.min_p = min_p, a.u = u, a.ids = ids;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = is_bf16 ? sample_plan<true>(a, st) : sample_plan<false>(a, st);
    return e == cudaSuccess ? MOE_OK : moe_fail_status(MOE_ECUDA, "moe_sample: %s", cudaGetErrorString(e));
}
