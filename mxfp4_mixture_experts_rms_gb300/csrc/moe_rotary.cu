// moe_rotary.cu -- queries and keys before a cache: each head's norm and the
// rotation by its token's positions, in one pass.
//
//   y = x / sqrt(mean(x^2) + eps) * gamma        (where the side has a gamma)
//   (a, b) -> (a cos - b sin, b cos + a sin)     angle = position[axis] * freq
//
// for the pairs (a, b) of a head: dims i and i + n_pairs, or 2 i and 2 i + 1.
// Everything in fp32, rounded once, to bf16.  An angle is taken in turns: the
// frequency's turns a position as a 64-bit fraction F, so that the low 64 bits
// of position * F are the turn's fraction, exact to 2^-33 of a turn wherever the
// position is (an fp32 product is off by whole radians at 2^24).
//
// Bound by HBM: 4 bytes an element.  A CTA takes the tokens' angles first, once
// for all heads, then a group of D / 8 lanes a head: a lane holds four dims of
// each half, so that no pair crosses lanes and the norm's sum is the only
// exchange.
#include "moe_common.cuh"
#include "../../include/moe.h"

#include <climits>
#include <cmath>
#include <cstring>
#include <new>

namespace {

constexpr int kThreads = 128;
constexpr int kMaxAxes = 4;
constexpr int kTokens = 2;      // of a CTA, at most

struct RotaryArgs {
    const uint16_t *q, *k;      // rows of heads
    uint16_t *qo, *ko;
    long long qs, ks, qos, kos;  // elements from row to row
    int QH, KVH, n, pairs, axes, tokens;   // tokens: of a CTA
    const int32_t *pos;          // [axes][pos_stride]
    long long pos_stride;
    const double *freqs;         // [pairs], radians a position
    const uint8_t *of;           // [pairs]: axis of each pair, or null
    const float *qg, *kg;        // [D] or null
    float eps, factor;
};

__device__ __forceinline__ float lo16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi16(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t pack(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}
__device__ __forceinline__ void unpack(uint2 w, float *x) { x[0] = lo16(w.x), x[1] = hi16(w.x), x[2] = lo16(w.y), x[3] = hi16(w.y); }

template <int D, bool INTER>
__global__ void __launch_bounds__(kThreads) moe_rotary_kernel(const RotaryArgs a) {
    constexpr int L = D / 8, G = kThreads / L, U = 4;   // lanes of a head; heads at once; heads a group loads ahead
    __shared__ float2 table[kTokens * D / 2];            // factor * (cos, sin)
    __shared__ int skip[kTokens];
    const int tid = threadIdx.x, t0 = blockIdx.x * a.tokens, nt = min(a.tokens, a.n - t0);
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (tid < kTokens) {
        int s = 0;
        if (tid < nt)
            for (int x = 0; x < a.axes; x++) s |= a.pos[x * a.pos_stride + t0 + tid] < 0;
        skip[tid] = s;
    }
    for (int i = tid; i < nt * a.pairs; i += kThreads) {
        const int t = i / a.pairs, p = i - t * a.pairs;
        const int axis = a.of ? min((int)a.of[p], a.axes - 1) : 0;
        double turns = a.freqs[p] * 0.15915494309189533577;
        turns -= floor(turns);
        const unsigned long long f = __double2ull_rn(turns * 18446744073709551616.0);
        const unsigned long long at = (unsigned long long)(long long)a.pos[axis * a.pos_stride + t0 + t] * f;
        float s, c;
        sincospif((float)(int)(at >> 32) * 0x1p-31f, &s, &c);
        table[i] = make_float2(c * a.factor, s * a.factor);
    }
    __syncthreads();

    // the lane's dims: d0 .. d0 + 3 and d1 .. d1 + 3; its pairs p0 .. p0 + 3 (past a.pairs: not rotated)
    const int l = tid % L, g = tid / L;
    const int quads = a.pairs / 4;
    int d0, d1;
    const bool turned = l < quads;
    if (INTER || !turned) {
        d0 = 8 * l, d1 = d0 + 4;
        // (halves: what lies behind the pairs' dims, two quads a lane, is at 8 l as well)
    } else {
        d0 = 4 * l, d1 = a.pairs + 4 * l;
    }
    const int heads = a.QH + a.KVH, items = nt * heads;
    const bool norm = a.qg || a.kg;
    for (int base = blockIdx.y * G; base < items; base += U * G * gridDim.y) {   // the same for the whole CTA
        const int i0 = base + g;
        uint2 w[U][2];
#pragma unroll
        for (int u = 0; u < U; u++) {
            const int i = i0 + u * G * gridDim.y;
            if (i < items) {
                const int t = i / heads, h = i - t * heads;
                const uint16_t *row = h < a.QH ? a.q + (long long)(t0 + t) * a.qs + h * D : a.k + (long long)(t0 + t) * a.ks + (h - a.QH) * D;
                w[u][0] = *reinterpret_cast<const uint2 *>(row + d0), w[u][1] = *reinterpret_cast<const uint2 *>(row + d1);
            } else {
                w[u][0] = w[u][1] = make_uint2(0, 0);
            }
        }
#pragma unroll
        for (int u = 0; u < U; u++) {
            const int i = i0 + u * G * gridDim.y;
            const bool on = i < items;
            const int ii = on ? i : 0, t = ii / heads, h = ii - t * heads;
            const bool is_q = h < a.QH;
            float x[8];
            unpack(w[u][0], x), unpack(w[u][1], x + 4);
            const float *gamma = is_q ? a.qg : a.kg;
            float ss = 0.f;
            if (norm) {
#pragma unroll
                for (int e = 0; e < 8; e++) ss = fmaf(x[e], x[e], ss);
#pragma unroll
                for (int o = L / 2; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            }
            if (gamma) {
                const float mean = ss * (1.f / D) + a.eps;
                const float4 g0 = __ldg(reinterpret_cast<const float4 *>(gamma + d0)), g1 = __ldg(reinterpret_cast<const float4 *>(gamma + d1));
                if (mean > 1e-30f && mean < 1e37f) {
                    const float inv = rsqrtf(mean);
#pragma unroll
                    for (int e = 0; e < 8; e++) x[e] *= inv;
                } else {
                    // squares beyond fp32: the head again, in 64 bits (its lanes have one mean, so they come here together)
                    const unsigned mask = (L == 32 ? 0xffffffffu : (1u << (L & 31)) - 1) << (tid & 31 & ~(L - 1));
                    double sd = 0.;
#pragma unroll 1
                    for (int e = 0; e < 8; e++) sd += (double)x[e] * x[e];
#pragma unroll 1
                    for (int o = L / 2; o; o >>= 1) sd += __shfl_xor_sync(mask, sd, o);
                    const double inv = 1. / sqrt(sd / D + (double)a.eps);
#pragma unroll
                    for (int e = 0; e < 8; e++) x[e] = (float)(x[e] * inv);
                }
                x[0] *= g0.x, x[1] *= g0.y, x[2] *= g0.z, x[3] *= g0.w;
                x[4] *= g1.x, x[5] *= g1.y, x[6] *= g1.z, x[7] *= g1.w;
            }
            if (turned) {
                const float4 *cs = reinterpret_cast<const float4 *>(table + t * a.pairs + 4 * l);   // two pairs each
                const float4 c0 = cs[0], c1 = cs[1];
                const float c[4] = {c0.x, c0.z, c1.x, c1.z}, s[4] = {c0.y, c0.w, c1.y, c1.w};
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    float &A = INTER ? x[2 * e] : x[e], &B = INTER ? x[2 * e + 1] : x[4 + e];
                    const float y = A * c[e] - B * s[e], z = B * c[e] + A * s[e];
                    A = y, B = z;
                }
            }
            if (on && !skip[t]) {
                uint16_t *row = is_q ? a.qo + (long long)(t0 + t) * a.qos + h * D : a.ko + (long long)(t0 + t) * a.kos + (h - a.QH) * D;
                *reinterpret_cast<uint2 *>(row + d0) = make_uint2(pack(x[0], x[1]), pack(x[2], x[3]));
                *reinterpret_cast<uint2 *>(row + d1) = make_uint2(pack(x[4], x[5]), pack(x[6], x[7]));
            }
        }
    }
}

template <int D>
cudaError_t rotary_launch(const RotaryArgs &a, bool inter, dim3 grid, cudaStream_t st) {
    return inter ? launch_pdl(moe_rotary_kernel<D, true>, grid, dim3(kThreads), 0, st, a)
                 : launch_pdl(moe_rotary_kernel<D, false>, grid, dim3(kThreads), 0, st, a);
}

}  // namespace

struct moe_rotary {
    int D = 0, pairs = 0, axes = 1;
    bool inter = false;
    float eps = 1e-5f, factor = 1.f;
    const double *freqs = nullptr;
    const uint8_t *of = nullptr;
    const float *qg = nullptr, *kg = nullptr;
};

extern "C" {

moe_rotary *moe_rotary_create(int head_dim, int n_pairs, int n_axes, int interleaved) {
    if ((head_dim != 64 && head_dim != 128 && head_dim != 256) || n_pairs < 0 || n_pairs % 8 || 2 * n_pairs > head_dim || n_axes < 1 ||
        n_axes > kMaxAxes || (interleaved != 0 && interleaved != 1)) {
        moe_set_error("moe_rotary_create: bad arguments (head_dim 64, 128 or 256, n_pairs a multiple of 8 and at most head_dim / 2, "
                      "1..%d axes, interleaved 0 or 1)", kMaxAxes);
        return nullptr;
    }
    moe_rotary *p = new (std::nothrow) moe_rotary;
    if (!p) {
        moe_set_error("moe_rotary_create: out of host memory");
        return nullptr;
    }
    p->D = head_dim, p->pairs = n_pairs, p->axes = n_axes, p->inter = interleaved == 1;
    return p;
}

void moe_rotary_destroy(moe_rotary *p) { delete p; }

int moe_rotary_set_f(moe_rotary *p, const char *key, double v) {
    if (!p || !key) return moe_fail_status(MOE_EINVAL, "NULL argument");
    if (!strcmp(key, "eps")) {
        if (!(v >= 0. && v <= 1e30)) return moe_fail_status(MOE_EINVAL, "eps must be 0 .. 1e30");
        p->eps = (float)v;
    } else if (!strcmp(key, "factor")) {
        if (!(v > 1e-30 && v < 1e30)) return moe_fail_status(MOE_EINVAL, "factor must be positive (1e-30 .. 1e30)");
        p->factor = (float)v;
    } else {
        return moe_fail_status(MOE_EINVAL, "unknown floating option '%s'", key);
    }
    return MOE_OK;
}

int moe_rotary_set_freqs(moe_rotary *p, const double *freqs, const uint8_t *axes) {
    if (!p || (!freqs && p->pairs)) return moe_fail_status(MOE_EINVAL, "NULL argument");
    if ((uintptr_t)freqs & 7u) return moe_fail_status(MOE_EINVAL, "freqs must be 8-byte aligned");
    p->freqs = freqs, p->of = axes;
    return MOE_OK;
}

int moe_rotary_set_norm(moe_rotary *p, const float *q_gamma, const float *k_gamma) {
    if (!p) return moe_fail_status(MOE_EINVAL, "NULL plan");
    if (((uintptr_t)q_gamma | (uintptr_t)k_gamma) & 15u) return moe_fail_status(MOE_EINVAL, "gammas must be 16-byte aligned");
    p->qg = q_gamma, p->kg = k_gamma;
    return MOE_OK;
}

int moe_rotary_apply(moe_rotary *p, const uint16_t *q, long long q_stride, int q_heads, const uint16_t *k, long long k_stride,
                     int kv_heads, const int32_t *positions, long long pos_stride, int n_tokens, uint16_t *q_out,
                     long long q_out_stride, uint16_t *k_out, long long k_out_stride, void *stream) {
    if (!p) return moe_fail_status(MOE_EINVAL, "NULL plan");
    if (p->pairs && !p->freqs) return moe_fail_status(MOE_ENOTREADY, "moe_rotary_set_freqs has not been called");
    if (q_heads < 0 || kv_heads < 0 || q_heads > 65536 || kv_heads > 65536)
        return moe_fail_status(MOE_EINVAL, "q_heads and kv_heads must be 0..65536");
    if (n_tokens < 0 || n_tokens > (1 << 30)) return moe_fail_status(MOE_EINVAL, "n_tokens must be 0..2^30");
    if (n_tokens == 0 || q_heads + kv_heads == 0) return MOE_OK;
    if (!positions || (q_heads && (!q || !q_out)) || (kv_heads && (!k || !k_out))) return moe_fail_status(MOE_EINVAL, "NULL argument");
    if ((uintptr_t)positions & 3u) return moe_fail_status(MOE_EINVAL, "positions must be 4-byte aligned");
    if (p->axes > 1 && pos_stride < n_tokens) return moe_fail_status(MOE_EINVAL, "pos_stride must be at least n_tokens");
    struct Side {
        const uint16_t *x;
        long long xs;
        const uint16_t *o;
        long long os;
        long long row;
    } sides[2] = {{q, q_stride, q_out, q_out_stride, (long long)q_heads * p->D}, {k, k_stride, k_out, k_out_stride, (long long)kv_heads * p->D}};
    for (const Side &s : sides) {
        if (!s.row) continue;
        if (((uintptr_t)s.x | (uintptr_t)s.o) & 7u) return moe_fail_status(MOE_EINVAL, "rows must be 8-byte aligned");
        if (s.xs < s.row || s.os < s.row || s.xs % 4 || s.os % 4)
            return moe_fail_status(MOE_EINVAL, "row strides must be multiples of 4 and at least %lld elements", s.row);
    }
    // An output lies apart from every input and from the other output, or in rows
    // of one stride at other places, or on its own input exactly.
    auto clash = [&](const uint16_t *x, long long xs, long long xr, const uint16_t *y, long long ys, long long yr) {
        const uint16_t *xe = x + (long long)(n_tokens - 1) * xs + xr, *ye = y + (long long)(n_tokens - 1) * ys + yr;
        if (x >= ye || y >= xe) return false;
        if (xs != ys) return true;
        const long long d = (((long long)(y - x)) % xs + xs) % xs;   // places of y's rows in x's
        return d < xr || d + yr > xs;
    };
    for (int o = 0; o < 2; o++) {
        if (!sides[o].row) continue;
        for (int i = 0; i < 2; i++) {
            if (!sides[i].row || (i == o && sides[i].x == sides[o].o && sides[i].xs == sides[o].os)) continue;
            if (clash(sides[i].x, sides[i].xs, sides[i].row, sides[o].o, sides[o].os, sides[o].row))
                return moe_fail_status(MOE_EINVAL, "outputs must not overlap inputs other than their own in place");
        }
    }
    if (sides[0].row && sides[1].row && clash(q_out, q_out_stride, sides[0].row, k_out, k_out_stride, sides[1].row))
        return moe_fail_status(MOE_EINVAL, "q_out and k_out must not overlap");
    RotaryArgs a{};
    a.q = q, a.k = k, a.qo = q_out, a.ko = k_out, a.qs = q_stride, a.ks = k_stride, a.qos = q_out_stride, a.kos = k_out_stride;
    a.QH = q_heads, a.KVH = kv_heads, a.n = n_tokens, a.pairs = p->pairs, a.axes = p->axes;
    a.pos = positions, a.pos_stride = pos_stride, a.freqs = p->freqs, a.of = p->of, a.qg = p->qg, a.kg = p->kg;
    a.eps = p->eps, a.factor = p->factor;
    a.tokens = n_tokens >= 1024 ? kTokens : 1;
    const int groups = kThreads / (p->D / 8), per = groups * 4;   // heads that a CTA loads at once
    const long long items = (long long)a.tokens * (q_heads + kv_heads);
    const int split = n_tokens >= 512 ? 1 : (int)((items + per - 1) / per);
    const dim3 grid((unsigned)((n_tokens + a.tokens - 1) / a.tokens), (unsigned)(split < 1024 ? split : 1024));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = p->D == 64 ? rotary_launch<64>(a, p->inter, grid, st) : p->D == 128 ? rotary_launch<128>(a, p->inter, grid, st)
                                                                                              : rotary_launch<256>(a, p->inter, grid, st);
    return e == cudaSuccess ? MOE_OK : moe_fail_status(MOE_ECUDA, "moe_rotary_apply: %s", cudaGetErrorString(e));
}

}  // extern "C"
