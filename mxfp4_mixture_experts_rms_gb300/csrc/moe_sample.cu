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
//  1. a histogram over the weights' leading bits (16 bins an octave, 32
//     octaves; what is below is not counted) finds the bin that holds T; a
//     weight adds its mantissa, so bins hold their weights in units of their
//     octave;
//  2. one more pass sums what lies above that bin and lists the bin's logits;
//  3. the list is cut by histograms over the logits' order-preserving 32-bit
//     keys until one key is left.
// A top-k of few tokens lists all of them in step 2 instead, and a CTA ranks
// the list by comparing each with each: top-k, top-p and the choice itself
// need nothing more of the row.  A bin with more tokens than a list holds is cut
// into 512 by its weights' further bits, and listed then; only where a sub-bin
// holds too many again, or T lies below the 32 octaves, the row is searched by
// its keys (16 x 200 K logits within 0.1 of one another: 59 us).  Where step
// 1's rounding named a neighbour of T's bin, that one is looked at next.
//
// Weights are fp32: those below 2^-126 are 0.  Sums are fp32 over a lane's logits
// and whole multiples of 2^-40 above that, so they do not depend on their order;
// below the octaves, and in the part of a row that holds the chosen token, units
// are as small as the weights there.
//
// A row is a cluster's: each CTA keeps its part in shared memory (read from
// memory once) where it fits, and meets the others through distributed shared
// memory.  Large batches are bound by the passes' instructions (about eleven a
// logit in step 1, three where a pass skips it), single rows by the cluster's
// meetings, about half a microsecond each.
#include "moe_sample.cuh"
#include "../../include/moe.h"

#include <cooperative_groups.h>

#include <algorithm>
#include <climits>

namespace cg = cooperative_groups;

namespace {

typedef unsigned long long u64;
// Another CTA's shared memory, by 32-bit addresses.
__device__ __forceinline__ uint32_t remote(const void *p, int rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
    return r;
}
__device__ __forceinline__ uint32_t remote_u32(uint32_t at) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ u64 remote_u64(uint32_t at) {
    u64 v;
    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(at) : "memory");
    return v;
}
constexpr int kBins = 512;
constexpr int kMaxCluster = 8;
constexpr int kList = 2048;           // keys listed by a CTA
constexpr int kKeys = 2048;           // listed keys of a row that a CTA has room for
constexpr int kRank = 512;            // tokens that are ranked by comparing each with each
constexpr int kAloneBytes = 170000, kSharedBytes = 80000;   // of a row's part in shared memory: one CTA an SM, two
constexpr int kBinShift = 19;         // a weight's bits above: exponent and four bits of mantissa

// n tokens of weight w (0 .. 1; n at most 2^22) in units of 2^-(40 + up), up at
// least 0, rounded up: what can be chosen has a unit.  The caller sees to it
// that the result fits.
__device__ __forceinline__ u64 units(u64 n, float w, int up = 0) {
    const uint32_t b = __float_as_uint(w);
    if (b < 0x800000u || n == 0) return 0;   // 0, and below 2^-126 (which ex2 makes 0)
    const int s = (int)(b >> 23) - 110 + up;   // mantissa times 2^(exponent - 150) = units times 2^s
    const u64 m = n * ((b & 0x7FFFFFu) | 0x800000u);
    return s >= 0 ? m << s : (m + (1ull << min(-s, 47)) - 1) >> min(-s, 47);   // (m is below 2^47)
}
// A weight (0 .. 1) in units of 2^-40, by its bits, the nearest.
__device__ __forceinline__ u64 fixed40(float w) {
    const uint32_t b = __float_as_uint(w);
    const int s = (int)(b >> 23) - 110;   // as above
    const uint32_t m = (b & 0x7FFFFFu) | 0x800000u, down = min(max(-s, 0), 31);
    return s >= 0 ? (u64)m << s : (u64)((m + (1u << down >> 1)) >> down);
}

// p or u (0 .. 1 - 2^-24; NaN: 0) in units of 2^-64, and a part of a sum: all
// threads need it, and 64-bit floats are the GPU's slowest numbers.
__device__ __forceinline__ u64 fraction(float p) {
    const uint32_t b = __float_as_uint(fminf(fmaxf(p, 0.f), 0.99999994f));
    const int s = (int)(b >> 23) - 86;
    const uint32_t m = (b & 0x7FFFFFu) | 0x800000u;
    return s >= 0 ? (u64)m << s : (u64)(m >> min(-s, 31));
}
__device__ __forceinline__ u64 part_up(u64 sum, u64 f) { return __umul64hi(sum, f) + (sum * f != 0); }

// A lane's weights, a vector's at a time.  Limits are told of sums in two parts:
// 2^10 weights in one fp32 sum are off by up to 2^-16 where they are equal, as each
// addition rounds the same way.  (lo is what hi's additions lost, but where one
// added more than hi had, which is at most 2^-23 of the sum in all.  64 x up to 5
// rows of 128 K bf16 take 146 us with it, 144 without.)
template <bool LIMITS>
struct LaneSum {
    float hi = 0.f, lo = 0.f;
    // a vector's weights are added to what this gives, and that is put back
    __device__ __forceinline__ float take() const { return LIMITS ? 0.f : hi; }
    __device__ __forceinline__ void put(float w) {
        const float s = LIMITS ? hi + w : w;
        if (LIMITS) lo += w - (s - hi);
        hi = s;
    }
    __device__ __forceinline__ u64 fixed() const {   // in units of 2^-40
        const u64 sum = __float2ull_rn(hi * 0x1p40f);
        return LIMITS ? sum + (u64)__float2ll_rn(lo * 0x1p40f) : sum;
    }
};

// What the CTAs of a row tell one another, each its slot.
struct Told {
    uint32_t key;
    int n, ties;
    u64 sum;
};

// LIMITS: tells what the row's token would be chosen from (SampleLimits) instead of choosing it.
template <bool BF16, bool RES, int NT, bool LIMITS>
__global__ void __launch_bounds__(NT, 1024 / NT) moe_sample_kernel(const SampleArgs a) {
    typedef Row<BF16, RES, NT> R;
    constexpr int VE = R::VE, NW = NT / 32;
    extern __shared__ __align__(16) uint4 data[];
    __shared__ u64 hist[kBins];         // (also: weights of the ranked tokens)
    __shared__ uint32_t hist32[kBins];
    __shared__ uint2 list[kList];       // key, index
    __shared__ uint32_t keys[kKeys];    // all CTAs' listed keys (or the ranked tokens' keys and indices)
    uint2 *const all = reinterpret_cast<uint2 *>(keys);
    __shared__ int ranks[kRank];
    __shared__ Told told[2][kMaxCluster];
    __shared__ u64 part[NW], sums[2][NW], s_above, wmass[NW];
    __shared__ uint32_t red[NW], s_lo, s_hi;
    __shared__ int s_bin, s_n, wties[NW];
    cg::cluster_group cl = cg::this_cluster();
    const int rank = (int)cl.block_rank(), C = (int)cl.num_blocks();
    const int row = blockIdx.x / C, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    asm volatile("barrier.cluster.arrive.relaxed.aligned;");   // waited for before the first write to another CTA
    if (!LIMITS) asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (LIMITS) asm volatile("griddepcontrol.launch_dependents;");   // the dependent reads what earlier kernels wrote before it waits

    R d;
    {
        const uintptr_t at = (uintptr_t)a.x + (size_t)row * a.stride * (BF16 ? 2 : 4);
        d.g = reinterpret_cast<const uint4 *>(at & ~(uintptr_t)15);
        d.off = (int)(at & 15) / (BF16 ? 2 : 4);
        d.V = a.V;
        d.s = data;
        const int vecs = (d.off + a.V + VE - 1) / VE;
        d.c0 = min(rank * a.seg, vecs);
        const int c1 = min(d.c0 + a.seg, vecs), per = (c1 - d.c0 + NW - 1) / NW;
        d.v0 = min(d.c0 + warp * per, c1), d.v1 = min(d.v0 + per, c1);
    }
    float t, p, mp, u;
    int k, of = row;
    auto settings = [&](int of) {
        t = used_temperature(a.temperature ? a.temperature[of] : 1.f);
        k = a.top_k ? a.top_k[of] : 0;
        p = a.top_p ? a.top_p[of] : 1.f, mp = a.min_p ? used_min_p(a.min_p[of]) : 0.f;
        u = LIMITS ? 0.f : a.u[of];
    };
    if (!LIMITS) settings(row);
    int turn = 0;
    // every CTA's value to every CTA; all of them are there after it
    auto tell = [&](Told mine) {
        turn ^= 1;
        if (tid < C) *cl.map_shared_rank(&told[turn][rank], tid) = mine;
        cl.sync();
    };

    // the row's largest logit, while its part comes in
    uint32_t km = 0;
    {
        float m = -INFINITY;
        for (int v = d.v0 + lane; v < d.v1; v += 128) {   // four vectors a lane on their way
            uint4 w[4];
#pragma unroll
            for (int q = 0; q < 4; q++)
                if (v + 32 * q < d.v1) w[q] = d.fetch(v + 32 * q);
#pragma unroll
            for (int q = 0; q < 4; q++)
                if (v + 32 * q < d.v1) {
                    if (RES) data[v + 32 * q - d.c0] = w[q];
                    float x[VE];
                    R::values(w[q], x);
#pragma unroll
                    for (int e = 0; e < VE; e++) m = fmaxf(m, x[e]);   // NaN passes over
                }
        }
        km = order_key(m);
    }
    km = __reduce_max_sync(0xffffffffu, km);
    if (lane == 0) red[warp] = km;
    if (LIMITS) {
        of = sequence_of(a.starts, a.n_seqs, row);
        settings(max(of, 0));
    }
    __syncthreads();
    km = __reduce_max_sync(0xffffffffu, red[lane % NW]);
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");   // every CTA of the row runs
    tell({km, 0, 0, 0});
    for (int c = 0; c < C; c++) km = max(km, told[turn][c].key);
    if (km == 0 || of < 0) {   // nothing to choose
        if (rank == 0 && tid == 0) {
            if (LIMITS) a.limits[row] = {0u, 0u, 0, 0.f, 0.f, 0.f};
            else a.ids[row] = -1;
        }
        return;
    }
    const Weight<LIMITS> weight(key_logit(km), t);
    const float top = weight.top, scale = weight.scale, shift_w = weight.shift;
    const bool endless = weight.endless, steep = weight.steep;
    auto weights = [&](const float (&x)[VE], float (&w)[VE]) {
        if (endless || steep) {
#pragma unroll
            for (int e = 0; e < VE; e++) w[e] = weight(x[e]);
            return;
        }
#pragma unroll
        for (int e = 0; e < VE; e += 2) {
            asm("{ .reg .b64 a, b, c; mov.b64 a, {%2, %3}; mov.b64 b, {%4, %4}; mov.b64 c, {%5, %5}; fma.rn.f32x2 a, a, b, c; "
                "mov.b64 {%0, %1}, a; }" : "=f"(w[e]), "=f"(w[e + 1]) : "f"(x[e]), "f"(x[e + 1]), "f"(scale), "f"(shift_w));
            if (LIMITS)   // (x lo - top lo)
                asm("{ .reg .b64 a, b, c, d; mov.b64 a, {%2, %3}; mov.b64 b, {%4, %4}; mov.b64 c, {%5, %5}; mov.b64 d, {%0, %1}; fma.rn.f32x2 a, a, b, c; "
                    "add.rn.f32x2 d, d, a; mov.b64 {%0, %1}, d; }" : "+f"(w[e]), "+f"(w[e + 1]) : "f"(x[e]), "f"(x[e + 1]), "f"(weight.lo), "f"(-top * weight.lo));
            asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(w[e]));
            asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(w[e + 1]));
        }
    };
    const float least = mp * weight(top);   // min-p is relative to the largest weight
    auto tell_limits = [&](uint32_t T, int cut, double sum) {   // by one thread
        const double inv = 1. / sum;
        a.limits[row] = {km, T, cut, least, (float)inv, (float)(inv - (float)inv)};
    };
    // 0 - the bin of weight 1 - downwards; NaN is never asked for
    auto bin_of = [](float w) { return max((0x3F800000 >> kBinShift) - (int)(__float_as_uint(w) >> kBinShift), 0); };
    auto warp_sum = [](u64 v) {
#pragma unroll
        for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        return v;
    };
    auto scan = [&](u64 v) {   // inclusive, over the warp
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const u64 y = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += y;
        }
        return v;
    };
    // block-wide sum; the buffers take turns, so that one barrier does
    int buffer = 0;
    auto total = [&](u64 v) {
        v = warp_sum(v);
        buffer ^= 1;
        if (lane == 0) sums[buffer][warp] = v;
        __syncthreads();
        return warp_sum(lane < NW ? sums[buffer][lane] : 0);
    };
    // block-wide: the first bin whose inclusive sum of h (one a thread, kBins of them) reaches goal
    auto find = [&](u64 h, u64 goal) {
        u64 inc = scan(h);
        if (lane == 31 && warp < kBins / 32) part[warp] = inc;
        if (tid == 0) s_bin = -1;
        __syncthreads();
        if (tid < kBins) {
            inc += warp_sum(lane < warp ? part[lane] : 0);
            if (inc >= goal && inc - h < goal) s_bin = tid, s_above = inc - h;
        }
        __syncthreads();
        return s_bin;
    };
    // kept: keys above T, and the first r tokens whose key is T
    uint32_t T = 0;
    u64 r = 0;
    if (!(t > 0.f)) T = km, r = 1;
#pragma unroll
    for (int stage = 0; stage < 2 && t > 0.f; stage++) {   // (each its own code)
        const bool by_weight = stage == 1;
        if (by_weight ? !(p < 1.f) : !(k > 0 && k < a.V)) continue;
        const float over = T ? key_logit(T) : -INFINITY;   // what top-k left lies above, and r tokens at it
        // 1. the histogram, and the weight of all
        __syncthreads();
        for (int b = tid; b < kBins; b += NT) hist32[b] = 0;
        __syncthreads();
        LaneSum<LIMITS> sum;
        const uint32_t half = (1u << a.drop) >> 1;
        d.each([&](float (&x)[VE], int) {
            float w[VE], here = sum.take();
            weights(x, w);
#pragma unroll
            for (int e = 0; e < VE; e++) {
                const bool in = x[e] > over;
                const int b = bin_of(w[e]);
                here += in ? w[e] : 0.f;
                if (in && b < kBins) atomicAdd(&hist32[b], by_weight ? (((__float_as_uint(w[e]) & 0x7FFFFFu) | 0x800000u) + half) >> a.drop : 1u);
            }
            sum.put(here);
        });
        u64 goal = (u64)k, everything = 0;
        u64 drop = 0;   // weight that top-p may leave out, in units of 2^-64
        tell({0, 0, 0, by_weight ? total(sum.fixed()) : 0});   // and the histograms are there
        if (by_weight) {
            for (int c = 0; c < C; c++) everything += told[turn][c].sum;
            if (T) {
                const double at_T = (double)weight(key_logit(T)) * 0x1p40, ties = (double)r * at_T, all = (double)everything + ties;
                const double out = (1. - (double)fmaxf(p, 0.f)) * all - ties;   // of the tokens above T
                if (out < 0. || everything == 0) {   // among the tokens at T
                    r -= min((u64)((out + ties) / at_T), r - 1);
                    cl.sync();     // the histograms are read no more
                    continue;
                }
                goal = (u64)ceil((double)fmaxf(p, 0.f) * all), drop = (u64)fmin(out * 0x1p24, 0x1p62);
            } else {
                goal = part_up(everything, fraction(p));
                const u64 not_p = ~fraction(p) + 1, hi = __umul64hi(everything, not_p);
                drop = hi >> 38 || !not_p ? 1ull << 62 : hi << 24 | (everything * not_p) >> 40;
            }
            goal = max(goal, (u64)1);
        }
        u64 h = 0;
        if (tid < kBins) {
#pragma unroll
            for (int c = 0; c < kMaxCluster; c++)
                if (c < C) h += remote_u32(remote(hist32 + tid, c));
            // mantissas of bins in one octave have one unit: 2^(drop - 23 - octave), here of 2^-40
            const int shift = 40 - 23 + a.drop + (int)(((0x3F800000u >> kBinShift) - (unsigned)tid) >> (23 - kBinShift)) - 127;
            if (by_weight) h = shift >= 0 ? h << shift : h >> -shift;
        }
        const int bin = find(h, goal);
        // 2. what lies above the bin, and the bin's keys; few tokens: all of them
        u64 above = 0, rest = 0;   // the goal's part that the tokens at T fill
        uint32_t T_new = 0, from = 0, span = 0;   // the bin's weights by their bits: from .. from + 2^span - 1
        bool found = false, in_bin = bin >= 0, many = false;
        if (in_bin) from = (uint32_t)((0x3F800000 >> kBinShift) - bin) << kBinShift, span = kBinShift;
        // (step 1's rounding may name a neighbour of T's bin: the next ones then, a few times)
#pragma unroll 1
        for (int look = 0; look < 6 && in_bin && !found; look++) {
            if (look == 0 && tid == bin) s_n = (int)min(s_above + h, (u64)INT_MAX);   // by count: tokens up to the bin
            __syncthreads();
            const bool few = look == 0 && !by_weight && s_n <= kRank;
            __syncthreads();
            if (tid == 0) s_n = 0, s_lo = 0xFFFFFFFFu, s_hi = 0;
            __syncthreads();
            LaneSum<LIMITS> before;
            int count = 0;
            // the bin's weights: from w_in up to w_up; listed: from w_in, up to w_end (NaN nowhere)
            const bool first = span == kBinShift && from >= 0x3F800000u;   // with all weights of 1 and (by rounding) above
            const float w_in = __uint_as_float(from), w_up = first ? INFINITY : __uint_as_float(from + (1u << span));
            const float w_end = few ? INFINITY : w_up;
            d.each([&](float (&x)[VE], int i) {
                float w[VE], here = before.take();
                weights(x, w);
                uint32_t take = 0;
#pragma unroll
                for (int e = 0; e < VE; e++) {
                    const bool in = x[e] > over, up = in && w[e] >= w_up;
                    here += up ? w[e] : 0.f;
                    count += up;
                    take |= in && w[e] >= w_in && w[e] < w_end ? 1u << e : 0u;
                }
                before.put(here);
                while (take) {
                    const int e = __ffs(take) - 1, at = atomicAdd(&s_n, 1);
                    take &= take - 1;
                    float v = x[0];
#pragma unroll
                    for (int q = 1; q < VE; q++) v = e == q ? x[q] : v;
                    if (at < kList) list[at] = make_uint2(order_key(v), i + e);
                }
            });
            const u64 mine = total(by_weight ? before.fixed() : few ? 0 : (u64)count);
            tell({0, s_n, 0, mine});
            bool listed = true;
            int n = 0, base = 0;
            u64 sum = 0;
            for (int c = 0; c < C; c++) {
                sum += told[turn][c].sum, listed = listed && told[turn][c].n <= kList;
                if (c < rank) base += told[turn][c].n;
                n += told[turn][c].n;
            }
            if (span == kBinShift) above = sum;   // (of a sub-bin it has been summed)
            if (few && n <= kRank) {
                // all that top-k can keep, in the first CTA: each token against each
                uint2 *to = cl.map_shared_rank(all, 0);
                for (int i = tid; i < s_n; i += NT) to[base + i] = list[i];
                cl.sync();
                if (rank != 0) return;
                uint2 me = make_uint2(0, 0);
                u64 w = 0;
                int mine = 0;
                if (tid < n) {
                    me = all[tid];
#pragma unroll 4
                    for (int j = 0; j < n; j++) {
                        const uint2 o = all[j];
                        mine += o.x > me.x || (o.x == me.x && o.y < me.y);
                    }
                    if (mine < k) w = units(1, weight(key_logit(me.x)), 13);   // kRank of them are below 2^63
                    ranks[tid] = mine, hist[tid] = w;
                }
                const u64 kept = total(w);
                bool keep = tid < n && mine < k;
                if (p < 1.f) {
                    const u64 g = max(part_up(kept, fraction(p)), (u64)1);
                    u64 ahead = 0;
                    if (keep)
#pragma unroll 4
                        for (int j = 0; j < n; j++) ahead += ranks[j] < mine ? hist[j] : 0;
                    keep = keep && ahead < g;
                }
                keep = keep && (mp < 1.f ? weight(key_logit(me.x)) >= least : me.x == km);
                __syncthreads();
                w = keep ? w : 0;
                if (tid < n) hist[tid] = w;
                const u64 all_kept = total(w);
                if (LIMITS) {
                    if (keep) atomicMin(&s_lo, me.x);
                    __syncthreads();
                    const uint32_t least_key = s_lo;
                    if (keep && me.x == least_key) atomicMax(&s_hi, me.y);   // the last of its tokens that is kept (all ahead of it are)
                    __syncthreads();
                    if (tid == 0) tell_limits(least_key, (int)s_hi + 1, (double)all_kept * 0x1p-53);
                    return;
                }
                const u64 target = __umul64hi(all_kept, fraction(u));
                u64 run = 0;
                if (w)
#pragma unroll 4
                    for (int j = 0; j < n; j++) run += all[j].y < me.y ? hist[j] : 0;
                if (w && target >= run && target < run + w) a.ids[row] = (int)me.y;
                return;
            }
            // 3. by keys: of the lists (every CTA all of them)
            if (above >= goal) {
                in_bin = span == kBinShift && !first;
                from += 1u << kBinShift;
            } else if (listed && n <= kKeys) {
                // into this CTA's own copy, a warp a list at a time
                uint32_t l = 0xFFFFFFFFu, m = 0;
                int to = 0;
                for (int c = 0; c < C; c++) {
                    const uint32_t q = remote(list, c);
                    const int nc = told[turn][c].n;
                    if (warp % C == c)
                        for (int i = warp / C * 32 + lane; i < nc; i += (NW + C - 1 - c) / C * 32) {
                            const uint32_t key = remote_u32(q + 8 * i);
                            keys[to + i] = key;
                            l = min(l, key), m = max(m, key);
                        }
                    to += nc;
                }
                l = __reduce_min_sync(0xffffffffu, l), m = __reduce_max_sync(0xffffffffu, m);
                if (lane == 0) atomicMin(&s_lo, l), atomicMax(&s_hi, m);
                __syncthreads();
                uint32_t lo = s_lo, hi = s_hi;
                u64 at = above;
                for (int shift = 1; shift;) {
                    shift = max(0, 32 - __clz((hi - lo) | 1) - 9);
                    __syncthreads();
                    for (int b = tid; b < kBins; b += NT) hist[b] = 0;
                    __syncthreads();
                    // exact weights in two limbs of 20 bits, at most 2^31 of 2^11 keys: 32-bit additions are the fast
                    // ones where many keys are equal
                    uint32_t *const limbs = reinterpret_cast<uint32_t *>(hist);
                    for (int i = tid; i < n; i += NT) {
                        const uint32_t key = keys[i];
                        if (key < lo || key > hi) continue;
                        const u64 w = by_weight ? fixed40(weight(key_logit(key))) : 1;
                        const int b = (int)((hi - key) >> shift);
                        atomicAdd(&limbs[2 * b], (uint32_t)(w & 0xFFFFFu));
                        if (w >> 20) atomicAdd(&limbs[2 * b + 1], (uint32_t)(w >> 20));
                    }
                    __syncthreads();
                    h = tid < kBins ? limbs[2 * tid] + ((u64)limbs[2 * tid + 1] << 20) : 0;
                    const int sub = find(h, goal - at);
                    if (sub < 0) break;
                    at += s_above;
                    const uint32_t width = (1u << shift) - 1, top_key = hi - ((uint32_t)sub << shift);
                    lo = max(lo, top_key - min(width, top_key)), hi = top_key;
                    found = !shift;
                }
                T_new = hi, rest = goal - at;
                if (found) break;
                in_bin = span == kBinShift;
                from -= 1u << kBinShift;
                cl.sync();   // the lists are read no more
            } else if (span < kBinShift) {
                many = true, in_bin = false;
            } else {
                // too many: 512 sub-bins of the weights, and the one that holds T is listed.  Their sums are exact, by
                // count and by what the bits that are left add.
                const int s = kBinShift - 9;
                uint32_t *const low = reinterpret_cast<uint32_t *>(hist);
                for (int b = tid; b < kBins; b += NT) hist32[b] = low[b] = 0;
                __syncthreads();
                d.each([&](float (&x)[VE], int) {
                    float w[VE];
                    weights(x, w);
#pragma unroll
                    for (int e = 0; e < VE; e++) {
                        const uint32_t bits = __float_as_uint(w[e]) - from;
                        if (!(x[e] > over) || bits >> kBinShift) continue;
                        atomicAdd(&hist32[(bits >> s) ^ (kBins - 1)], 1u);   // downwards
                        if (by_weight) atomicAdd(&low[(bits >> s) ^ (kBins - 1)], bits & ((1u << s) - 1));   // of at most 2^22 tokens
                    }
                });
                cl.sync();
                h = 0;
                const uint32_t w0 = from + ((uint32_t)(tid ^ (kBins - 1)) << s);   // the sub-bin's least weight
                if (tid < kBins) {
#pragma unroll
                    for (int c = 0; c < kMaxCluster; c++)
                        if (c < C) {
                            const u64 in = remote_u32(remote(hist32 + tid, c));
                            h += by_weight ? in * ((w0 & 0x7FFFFFu) | 0x800000u) + remote_u32(remote(low + tid, c)) : in;
                        }
                    const int up = (int)(w0 >> 23) - 110;   // from units of the octave to 2^-40
                    if (by_weight) h = up >= 0 ? h << up : (h + (1ull << -up >> 1)) >> -up;
                }
                const int sub = find(h, goal - above);
                cl.sync();
                if (sub >= 0) above += s_above, from += (uint32_t)(sub ^ (kBins - 1)) << s, span = s;
                else from -= 1u << kBinShift;
            }
        }
        // The row's own keys, in steps of 2^9 sub-bins that end at single keys:
        // those of the sub-bin, where even they are too many to list; where T is
        // below the octaves, or has not been found, all.  A sub-bin's weight is
        // exact: the sum of its tokens', or where it is one key their count times
        // its weight.  Tokens below the octaves are held in units of 2^-64, and
        // what is left out of them is what counts: the goal itself, next to 1, has
        // no bits for them.
        constexpr int KS = BF16 ? 16 : 0;   // a bf16 logit's key is its upper half
        auto in_span = [&](float w) { return (__float_as_uint(w) - from) >> span == 0; };
        auto full = [](uint32_t q) { return BF16 ? q << 16 | (q & 0x8000u ? 0u : 0xFFFFu) : q; };
#pragma unroll 1
        for (int whole = many ? 0 : 1; whole < 2 && !found; whole++) {
            uint32_t lo = 1 >> KS, hi = km >> KS;
            u64 at = 0, need = goal;
            const bool tail = by_weight && bin < 0;
            bool unseen = tail;   // is the sum of the tokens below the octaves still to be seen?
            auto exact = [&](float w) { return tail ? units(1, w, 24) : fixed40(w); };
            cl.sync();   // what was read of other CTAs is read no more
            if (!whole) {
                uint32_t l = 0xFFFFFFFFu, m = 0;
                d.each([&](float (&x)[VE], int) {
#pragma unroll
                    for (int e = 0; e < VE; e++)
                        if (x[e] > over && in_span(weight(x[e]))) l = min(l, order_key(x[e])), m = max(m, order_key(x[e]));
                });
                l = __reduce_min_sync(0xffffffffu, l), m = __reduce_max_sync(0xffffffffu, m);
                if (lane == 0) atomicMin(&s_lo, l), atomicMax(&s_hi, m);
                __syncthreads();
                tell({s_lo, (int)s_hi, 0, 0});
                lo = 0xFFFFFFFFu, hi = 0, at = above;
                for (int c = 0; c < C; c++) lo = min(lo, told[turn][c].key >> KS), hi = max(hi, (uint32_t)told[turn][c].n >> KS);
            }
            for (int shift = 1; shift;) {
                shift = max(0, 32 - __clz((hi - lo) | 1) - 9);
                const bool sums = by_weight && shift;
                __syncthreads();
                for (int b = tid; b < kBins; b += NT) hist[b] = 0;
                for (int b = tid; b < kBins; b += NT) hist32[b] = 0;
                __syncthreads();
                d.each([&](float (&x)[VE], int) {
#pragma unroll
                    for (int e = 0; e < VE; e++) {
                        const uint32_t key = order_key(x[e]) >> KS;
                        if (!(x[e] > over) || key < lo || key > hi) continue;
                        const float w = weight(x[e]);
                        if (tail ? bin_of(w) < kBins : !whole && !in_span(w)) continue;
                        if (sums) atomicAdd(&hist[(hi - key) >> shift], exact(w));
                        else atomicAdd(&hist32[(hi - key) >> shift], 1u);
                    }
                });
                cl.sync();
                h = 0;
                if (tid < kBins) {
#pragma unroll
                    for (int c = 0; c < kMaxCluster; c++)
                        if (c < C) h += sums ? remote_u64(remote(hist + tid, c)) : remote_u32(remote(hist32 + tid, c));
                    if (by_weight && !shift && h) h *= exact(weight(key_logit(full(hi - tid))));
                }
                if (unseen) {
                    unseen = false;
                    const u64 of_tail = total(h);
                    need = of_tail > drop ? of_tail - drop : 1;
                }
                const int sub = find(h, need - at);
                cl.sync();
                if (sub < 0) break;
                at += s_above;
                const uint32_t width = (1u << shift) - 1, top_key = hi - ((uint32_t)sub << shift);
                lo = max(lo, top_key - min(width, top_key)), hi = top_key;
                found = !shift;
            }
            T_new = full(hi), rest = need - at;
        }
        if (found) {
            const float w_T = weight(key_logit(T_new));
            const u64 w = !by_weight ? 1 : bin < 0 ? units(1, w_T, 24) : fixed40(w_T);
            T = T_new, r = (rest + w - 1) / w;
        } else if (!by_weight) {
            T = 0, r = 0;   // fewer than k tokens
        }                   // (by weight: the goal is beyond the sum's rounding, and all that top-k left is kept)
        cl.sync();   // lists, histograms and what was told are read no more
    }

    // min-p of 1: the largest logit's tokens, not those whose weight rounds to 1
    if (!(mp < 1.f) && T != km) T = km, r = a.V;
    // the kept weight of each warp's part, and its tokens at T.  A lane's sum is
    // at least one unit, the sum over the tokens at T is rounded up (the n-th of
    // them adds at_T(n) - at_T(n - 1)): a part with a token to choose is never
    // nothing.
    const float xT = T ? key_logit(T) : -INFINITY;
    const float wT = T ? weight(xT) : 0.f;
    auto at_T = [&](u64 n) { return wT >= least ? units(min(n, r), wT) : 0; };
    LaneSum<LIMITS> sum;
    int ties = 0;
    d.each([&](float (&x)[VE], int) {
        float w[VE], here = sum.take();
        weights(x, w);
#pragma unroll
        for (int e = 0; e < VE; e++) {
            here += x[e] > xT && w[e] >= least ? w[e] : 0.f;
            ties += x[e] == xT;   // (-inf where no logit is at T: not counted below, as r is 0)
        }
        sum.put(here);
    });
    u64 mass = warp_sum(max(sum.fixed(), (u64)(sum.hi > 0.f)));
    ties = __reduce_add_sync(0xffffffffu, ties);
    if (lane == 0) wmass[warp] = mass, wties[warp] = ties;
    __syncthreads();
    // (a lane a warp from here on)
    mass = lane < NW ? wmass[lane] : 0, ties = lane < NW ? wties[lane] : 0;
    tell({0, 0, (int)__reduce_add_sync(0xffffffffu, ties), warp_sum(mass)});
    // in order of index: kept weight before each CTA, warp, lane, logit
    u64 kept = 0, base = 0, tb = 0, tsum = 0, own = 0, upto = 0;   // (upto: at_T(tsum))
    for (int c = 0; c < C; c++) {
        const u64 ct = told[turn][c].ties;
        u64 m = told[turn][c].sum;
        if (c == rank) base = kept, tb = tsum;
        if (ct && tsum < r) {
            const u64 f = at_T(tsum + ct);
            m += f - upto, upto = f;
        }
        if (c == rank) own = m;
        kept += m, tsum += ct;
    }
    if (LIMITS) {
        const double sum = (double)kept * 0x1p-40;
        if (!T || tsum <= r) {
            if (rank == 0 && tid == 0) tell_limits(T, a.V, sum);
            return;
        }
        // where the r-th token at T is: one warp's part
        const u64 t0 = tb + scan((u64)ties) - ties;
        const unsigned hit = __ballot_sync(0xffffffffu, t0 < r && r <= t0 + ties);
        if (!hit || warp != __ffs(hit) - 1) return;
        int left = (int)(r - __shfl_sync(0xffffffffu, t0, warp));
        for (int v = d.v0; v < d.v1; v += 32) {
            float x[VE];
            if (v + lane < d.v1) {
                R::values(d.vec(v + lane), x);
            } else {
#pragma unroll
                for (int e = 0; e < VE; e++) x[e] = -INFINITY;
            }
            int n = 0;
#pragma unroll
            for (int e = 0; e < VE; e++) n += x[e] == xT;
            int inc = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += y;
            }
            const int all = __shfl_sync(0xffffffffu, inc, 31);
            if (left > all) {
                left -= all;
                continue;
            }
            int at = inc - n;   // before the lane's
#pragma unroll
            for (int e = 0; e < VE; e++)
                if (x[e] == xT && ++at == left) tell_limits(T, (v + lane) * VE - d.off + e + 1, sum);
            return;
        }
        return;
    }
    u64 target = __umul64hi(kept, fraction(u));   // the first token whose running sum exceeds u times the total
    if (target < base || target >= base + own) return;
    {
        const u64 t0 = tb + scan((u64)ties) - ties;   // tokens at T before the lane's warp
        if (ties && t0 < r) mass += at_T(t0 + ties) - at_T(t0);
        const u64 m0 = base + scan(mass) - mass;
        const unsigned hit = __ballot_sync(0xffffffffu, target >= m0 && target < m0 + mass);
        if (warp != __ffs(hit) - 1) return;
        target -= __shfl_sync(0xffffffffu, m0, warp), tb = __shfl_sync(0xffffffffu, t0, warp);
        mass = __shfl_sync(0xffffffffu, mass, warp);
    }
    // this warp's: 32 vectors at a time, in units in which its sum is about
    // 2^62, so that it has a token to choose however little it weighs.  Its
    // lanes' sums were rounded otherwise: where the running sum stays below the
    // target to the end, the last kept token is the one.
    const int up = max(__clzll((long long)mass) - 2, 0);
    target <<= up, base = 0;
    int last = -1;
    for (int v = d.v0; v < d.v1; v += 32) {
        float x[VE];
        if (v + lane < d.v1) {
            R::values(d.vec(v + lane), x);
        } else {
#pragma unroll
            for (int e = 0; e < VE; e++) x[e] = -INFINITY;
        }
        int mt = 0;
#pragma unroll
        for (int e = 0; e < VE; e++) mt += T && x[e] == xT;
        u64 rt = tb;   // tokens at T before this lane's
        if (__any_sync(0xffffffffu, mt)) {
            int it = mt;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, it, o);
                if (lane >= o) it += y;
            }
            rt += it - mt;
            tb += __shfl_sync(0xffffffffu, it, 31);
        }
        // the lane's weight at once, its tokens' only where the choice is among them
        float w[VE], mine = 0.f;
        uint32_t keep = 0;
#pragma unroll
        for (int e = 0; e < VE; e++) {
            w[e] = weight(x[e]);
            const bool in = mt && x[e] == xT ? rt++ < r : x[e] > xT;
            if (in && w[e] >= least && w[e] > 0.f) keep |= 1u << e, mine += w[e];
        }
        if (keep) last = (v + lane) * VE - d.off + 31 - __clz(keep);
        const u64 m = units(1, mine, up), here = warp_sum(m);
        if (target >= base + here) {
            base += here;
            continue;
        }
        u64 at = base + scan(m) - m;
        if (target >= at && target < at + m) {
            int id = last;
#pragma unroll
            for (int e = 0; e < VE; e++) {
                const u64 one = keep >> e & 1 ? units(1, w[e], up) : 0;
                if (target >= at && target < at + one) id = (v + lane) * VE - d.off + e;
                at += one;
            }
            a.ids[row] = id;
        }
        return;
    }
    last = __reduce_max_sync(0xffffffffu, last);
    if (lane == 0) a.ids[row] = last;
}

// Clusters of C CTAs, 1 .. kMaxCluster, that the device runs at once with one
// CTA an SM: sizes of clusters and of the device's partitions need not go into
// one another.
struct Fits {
    int n[kMaxCluster + 1];
    bool known;
};
template <bool BF16>
cudaError_t sample_fits(const Fits *&out) {
    static PerDevice<Fits> fits;
    static PerDevice<bool> opted;
    int dev = 0;
    cudaError_t e = current_device_slot(&dev);
    if (e != cudaSuccess) return e;
    Fits &f = fits.v[dev];
    out = &f;
    if (f.known) return cudaSuccess;
    e = smem_optin_once(moe_sample_kernel<BF16, true, 1024, false>, opted);
    for (int C = 1; C <= kMaxCluster && e == cudaSuccess; C++) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(C), cfg.blockDim = dim3(1024), cfg.dynamicSmemBytes = kAloneBytes;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = C, attr[0].val.clusterDim.y = 1, attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr, cfg.numAttrs = 1;
        e = cudaOccupancyMaxActiveClusters(&f.n[C], moe_sample_kernel<BF16, true, 1024, false>, &cfg);
    }
    f.known = e == cudaSuccess;
    return e;
}

template <bool BF16, bool RES, int NT, bool LIMITS>
cudaError_t sample_launch(const SampleArgs &a, int C, size_t smem, cudaStream_t st) {
    static PerDevice<bool> opted;
    cudaError_t e = smem_optin_once(moe_sample_kernel<BF16, RES, NT, LIMITS>, opted);
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
    return cudaLaunchKernelEx(&cfg, moe_sample_kernel<BF16, RES, NT, LIMITS>, a);
}

template <bool BF16, bool LIMITS>
cudaError_t sample_plan(SampleArgs a, cudaStream_t st) {
    const int VE = BF16 ? 8 : 4;
    const long long vecs = ((long long)a.V + VE - 1) / VE + 1;   // one more where the first is cut
    // CTAs of a row: as many as run at once with one an SM, each with at least
    // 128 vectors (one row of 32 K fp32: 19, 15, 11, 10 us with 1, 2, 4, 8, before
    // the other steps to 9; 16 x 200 K: 52 with 8, where the 16th cluster had to
    // wait for another's SMs, 28 with the most that all fit),
    // and where there are more rows, as many as two an SM need to keep their
    // parts in shared memory (256 x 128 K bf16, mixed: 143 and 108 us with 1 and
    // 2 that read it from L2 again, 95 with 4, 124 with 8, before the other
    // steps to 88).
    const Fits *fits;
    const cudaError_t e = sample_fits<BF16>(fits);
    if (e != cudaSuccess) return e;
    int C = kMaxCluster;
    while (C > 1 && (a.rows > fits->n[C] || vecs / C < 128)) C--;
    const bool alone = a.rows <= fits->n[C] && vecs * 16 / C <= kAloneBytes - 16;   // one CTA an SM
    while (!alone && C < kMaxCluster && vecs * 16 / C > kSharedBytes) C++;
    // Rows that no cluster holds are read anew by every pass: as many CTAs as
    // two an SM allow, four at least (fp32 rows of 200 K, C = 1, 2, 4, 8: 24 of
    // them 156, 84, 57, 47 us, 100 of them 184, 119, 99, 115, 256 of them 281,
    // 249, 224, 278; bf16 rows of 1 M: 24 of them 771, 400, 263, 196, 256 of
    // them 1489, 1266, 1186, 1204).
    if (!alone && vecs * 16 / C > kSharedBytes) C = std::min(std::max(2 * fits->n[1] / a.rows, 4), kMaxCluster);
    a.seg = (int)((vecs + C - 1) / C);
    const size_t smem = (size_t)a.seg * 16;
    a.drop = 0;
    while (((long long)a.V << 24) >> a.drop > 0xFFFFFFFFll - a.V) a.drop++;
    if (smem > (alone ? kAloneBytes : kSharedBytes)) return sample_launch<BF16, false, 512, LIMITS>(a, C, 0, st);
    // (alone, with much to do: all its warps)
    return alone && a.seg >= 2048 ? sample_launch<BF16, true, 1024, LIMITS>(a, C, smem, st) : sample_launch<BF16, true, 512, LIMITS>(a, C, smem, st);
}

}  // namespace

cudaError_t launch_sample_limits(const SampleArgs &a, bool bf16, cudaStream_t st) {
    return bf16 ? sample_plan<true, true>(a, st) : sample_plan<false, true>(a, st);
}

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
    const cudaError_t e = is_bf16 ? sample_plan<true, false>(a, st) : sample_plan<false, false>(a, st);
    return e == cudaSuccess ? MOE_OK : moe_fail_status(MOE_ECUDA, "moe_sample: %s", cudaGetErrorString(e));
}
