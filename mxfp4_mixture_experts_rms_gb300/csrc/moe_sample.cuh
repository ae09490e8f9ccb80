// moe_sample.cuh -- what choosing a row's token and verifying drafted ones
// share: a row's logits, their weights and the limits of what is kept.
#pragma once
#include "moe_common.cuh"

struct SampleLimits;
struct SampleArgs {
    const void *x;
    int rows, V;
    long long stride;
    const float *temperature;
    const int32_t *top_k;
    const float *top_p, *min_p, *u;
    int32_t *ids;
    int seg;         // 16-byte vectors of a row's part
    int drop;        // mantissa bits that a sum of V weights in 32 bits has no room for
    // Of rows that verify drafted tokens: sequence b has rows starts[b] ..
    // starts[b + 1] - 1, settings are a sequence's, and what the tokens' choice
    // would be made from is told instead.
    const int32_t *starts;
    int n_seqs;
    SampleLimits *limits;   // [rows]
};

// The tokens of a row that may be chosen: those whose logit's key is above T,
// and those whose key is T below index `cut`; of these the ones that min-p keeps.
struct SampleLimits {
    uint32_t top, T;   // keys of the largest logit (0: no token) and of the least that is kept
    int cut;
    float least;       // min-p's least weight, the largest logit's being 1
    float inv, inv_lo; // 1 over their weights' sum, in two parts
};

namespace {

constexpr float kLog2e = 1.4426950408889634f;

// Larger logit, larger key; NaN and -inf (never chosen): 0.
__device__ __forceinline__ uint32_t order_key(float l) {
    const uint32_t b = __float_as_uint(l + 0.f);  // -0 becomes +0
    return l > -INFINITY ? (b & 0x80000000u ? ~b : b | 0x80000000u) : 0u;
}
__device__ __forceinline__ float key_logit(uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k);
}

// The weight 2^((l - top) scale) of a logit.  An infinite largest logit: then
// only infinite ones weigh anything.  A row of steep scale: differences first,
// so that 0 stays 0.  Else the weights are 2^(x scale - top scale), the constant
// rounded: one factor, within 2^-14 of 1, on all of them.  FINE: with what
// log2(e) / t has beyond fp32, so that no error grows with the distance from the
// largest logit.
template <bool FINE>
struct Weight {
    float top, scale, shift, lo;
    bool endless, steep;
    __device__ __forceinline__ Weight(float top_, float t) : top(top_), lo(0.f) {
        scale = t > 0.f ? fminf(kLog2e / t, 1e30f) : 0.f;
        endless = top == INFINITY, steep = !(fabsf(top * scale) < 1000.f);
        shift = endless || steep ? 0.f : -top * scale;
        if (FINE && t > 0.f && scale < 1e30f && scale > 1e-30f) lo = (fmaf(-scale, t, kLog2e) + 1.925963033500e-8f) / t;   // log2(e) less its fp32
    }
    __device__ __forceinline__ float operator()(float x) const {
        float w, e = steep ? (x - top) * scale : fmaf(x, scale, shift);
        if (FINE && !endless && !steep) e += fmaf(x, lo, -top * lo);
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(w) : "f"(e));
        return endless ? (x == top ? 1.f : 0.f) : w;
    }
};
// A temperature as it is used: infinity as the largest float (NaN stays NaN: the
// first token, as t > 0 is false); a min_p in 0 .. 1, NaN 0.
__device__ __forceinline__ float used_temperature(float t) { return t == INFINITY ? 3.402823466e38f : t; }
__device__ __forceinline__ float used_min_p(float mp) { return fminf(fmaxf(mp, 0.f), 1.f); }

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
    // f(logits, first one's index) for the warp's vectors, a lane a vector; in
    // order of index; the next vector is read ahead
    template <class F>
    __device__ __forceinline__ void each(F f) const {
        int v = v0 + (threadIdx.x & 31);
        if (v >= v1) return;
        uint4 next = vec(v);
#pragma unroll 1
        for (; v < v1; v += 32) {
            const uint4 w = next;
            if (v + 32 < v1) next = vec(v + 32);
            float x[VE];
            values(w, x);
            f(x, v * VE - off);
        }
    }
};

// The sequence that a row belongs to, -1 for a row of none; starts do not
// decrease.  For a whole warp: 32 of them are looked at at a time.
__device__ __forceinline__ int sequence_of(const int32_t *starts, int n_seqs, int row) {
    const int lane = threadIdx.x & 31;
    int lo = 0, hi = n_seqs + 1;   // starts before lo are at most row, those from hi on larger
    while (lo < hi) {
        const int step = (hi - lo + 31) / 32, i = lo + (lane + 1) * step - 1;
        const int n = __popc(__ballot_sync(0xffffffffu, i < hi && __ldg(starts + i) <= row));
        lo += n * step;
        hi = min(hi, lo + step - 1);
    }
    return lo - 1 < n_seqs ? lo - 1 : -1;
}

}  // namespace

// Fills a.limits (seg and drop are set here).
cudaError_t launch_sample_limits(const SampleArgs &a, bool bf16, cudaStream_t st);
