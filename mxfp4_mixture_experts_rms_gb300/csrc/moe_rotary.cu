// moe_rotary.cu -- queries and keys before a cache: each head's norm and the
// rotation by its token's positions, in one pass.
//
//   y = x / sqrt(mean(x^2) + eps) * gamma        (where the side has a gamma)
//   (a, b) -> (a cos - b sin, b cos + a sin)     angle = position[axis] * freq
//
// for the pairs (a, b) of a head: dims i and i + n_pairs, or 2 i and 2 i + 1.
// Everything in fp32, rounded once, to bf16.  An angle is taken in turns: the
// frequency's turns a position as a 64-bit fraction F, so that the low 64 bits
// of position * F are the turn's fraction, exact to 2^-33 of a turn and 2^-52 of the
// angle (an fp32 product is off by whole radians at 2^24).  Its upper 32 bits are
// what sine and cosine take, as fp32: within 2^-26 of a turn near half a turn,
// nearer where it is less.
//
// Bound by HBM: 4 bytes an element.  A CTA takes its tokens' angles first, once
// for all heads, then a group of D / 16 lanes has two heads of each token: a lane
// holds eight dims of each half, so that no pair crosses lanes and the norm's sum
// is the only exchange.  As many groups as the heads need; a head's places move on
// by a stride from token to token, and the next token is loaded before this one
// is computed.  fp32 by twos.  15 001 tokens of 32 heads of 128 take 55 us, 37 at
// HBM's rate, 44 without norms and rotation: HBM and issue slots are 45 % busy
// each, a CTA's waits before its first row (angles, barriers) are the rest.  (With
// eight dims a lane and heads' places found anew for each, 71; tokens by
// asynchronous copies through shared memory, 72.)
#include "moe_common.cuh"
#include "../../include/moe.h"

#include <climits>
#include <cmath>
#include <cstring>
#include <new>

namespace {

constexpr int kMaxThreads = 256;
constexpr int kHeads = 2;       // of a group
constexpr int kMaxAxes = 4;
constexpr int kTokens = 4;      // of a CTA, at most

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

typedef unsigned long long u64;   // (also: two fp32)
__device__ __forceinline__ u64 two(float x, float y) {
    u64 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ float2 of_two(u64 v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ u64 mul2(u64 x, u64 y) {
    u64 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
    return r;
}
__device__ __forceinline__ u64 fma2(u64 x, u64 y, u64 z) {
    u64 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(x), "l"(y), "l"(z));
    return r;
}
__device__ __forceinline__ u64 unpack(uint32_t w) { return two(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u)); }
__device__ __forceinline__ uint32_t pack(u64 v) {
    const float2 f = of_two(v);
    const __nv_bfloat162 r = __floats2bfloat162_rn(f.x, f.y);
    return *reinterpret_cast<const uint32_t *>(&r);
}

__device__ __forceinline__ void lds2(const float *p, u64 (&v)[4]) {   // eight floats
    const ulonglong2 a = *reinterpret_cast<const ulonglong2 *>(p), b = *reinterpret_cast<const ulonglong2 *>(p + 4);
    v[0] = a.x, v[1] = a.y, v[2] = b.x, v[3] = b.y;
}

// NORMS: is either side normed?  Where none is, three CTAs of 256 threads an SM
// (80 registers: more rows in flight; 4099 tokens of 36 heads of 128 take 17.5
// us, 19.6 with 120).
template <int D, bool INTER, bool NORMS>
__global__ void __launch_bounds__(kMaxThreads, NORMS ? 2 : 3) moe_rotary_kernel(const RotaryArgs a) {
    constexpr int L = D / 16, U = kHeads;                 // lanes of a head
    __shared__ u64 turns[D / 2];                          // of a position, in units of 2^-64
    __shared__ __align__(16) float cosines[kTokens][D / 2], sines[kTokens][D / 2];   // times the factor
    __shared__ __align__(16) float gammas[NORMS ? 2 : 1][NORMS ? D : 4];
    __shared__ int skip[kTokens];
    const int tid = threadIdx.x, threads = blockDim.x, t0 = blockIdx.x * a.tokens, nt = min(a.tokens, a.n - t0);
    asm volatile("griddepcontrol.launch_dependents;");
    // the lane's dims: d0 .. d0 + 7 and d1 .. d1 + 7; its pairs 8 l .. 8 l + 7 (from a.pairs on: not rotated)
    const int l = tid % L, g = tid / L, groups = threads / L;
    const bool turned = l < a.pairs / 8;
    int d0 = 16 * l, d1 = d0 + 8;   // (halves: what lies behind the pairs' dims, too)
    if (!INTER && turned) d0 = 8 * l, d1 = a.pairs + 8 * l;
    // the group's heads, queries before keys, and where its lane's dims of the running token are
    const uint16_t *in[U];
    uint16_t *out[U];
    int side[U];
    bool on[U], norm[U];
#pragma unroll
    for (int u = 0; u < U; u++) {
        const int h = (blockIdx.y * U + u) * groups + g, x = h >= a.QH;
        side[u] = x, on[u] = h < a.QH + a.KVH, norm[u] = (x ? a.kg : a.qg) != nullptr;
        in[u] = (x ? a.k - a.QH * D + t0 * a.ks : a.q + t0 * a.qs) + h * D, out[u] = (x ? a.ko - a.QH * D + t0 * a.kos : a.qo + t0 * a.qos) + h * D;
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    uint4 next[U][2];
    auto load = [&](bool more) {
#pragma unroll
        for (int u = 0; u < U; u++) {
            next[u][0] = next[u][1] = make_uint4(0, 0, 0, 0);
            if (more && on[u]) next[u][0] = *reinterpret_cast<const uint4 *>(in[u] + d0), next[u][1] = *reinterpret_cast<const uint4 *>(in[u] + d1);
            in[u] += side[u] ? a.ks : a.qs;
        }
    };
    load(true);
    for (int i = tid; i < a.pairs; i += threads) {
        // (a negative one by its magnitude: next to 1 a fraction has no bits for it)
        const double freq = a.freqs[i];
        double t = fabs(freq) * 0.15915494309189533577;
        t -= floor(t);
        const u64 turn = __double2ull_rn(t * 18446744073709551616.0);
        turns[i] = freq < 0. ? 0 - turn : turn;
    }
    if (NORMS)
        for (int i = tid; i < 2 * D; i += threads) {
            const float *gamma = i < D ? a.qg : a.kg;
            gammas[i / D][i % D] = gamma ? gamma[i % D] : 1.f;
        }
    for (int t = tid; t < nt; t += threads) {
        int s = 0;
        for (int x = 0; x < a.axes; x++) s |= a.pos[x * a.pos_stride + t0 + t];
        skip[t] = s < 0;
    }
    __syncthreads();
    for (int t = 0; t < nt; t++)
        for (int i = tid; i < a.pairs; i += threads) {
            const int axis = a.of ? min((int)__ldg(a.of + i), a.axes - 1) : 0;
            const u64 at = (u64)(long long)a.pos[axis * a.pos_stride + t0 + t] * turns[i];
            float s, c;
            sincospif((float)(int)(at >> 32) * 0x1p-31f, &s, &c);
            cosines[t][i] = c * a.factor, sines[t][i] = s * a.factor;
        }
    __syncthreads();
#pragma unroll 1
    for (int t = 0; t < nt; t++) {
        uint4 w[U][2];
#pragma unroll
        for (int u = 0; u < U; u++) w[u][0] = next[u][0], w[u][1] = next[u][1];
        load(t + 1 < nt);
        const bool live = !skip[t];
        u64 cs[4], sn[4];
        auto angles = [&] { lds2(&cosines[t][8 * l], cs), lds2(&sines[t][8 * l], sn); };
        if (NORMS && turned) angles();
#pragma unroll
        for (int u = 0; u < U; u++) {
            u64 x[4] = {unpack(w[u][0].x), unpack(w[u][0].y), unpack(w[u][0].z), unpack(w[u][0].w)};
            u64 y[4] = {unpack(w[u][1].x), unpack(w[u][1].y), unpack(w[u][1].z), unpack(w[u][1].w)};
            if constexpr (NORMS) {
                auto squares = [&](unsigned lanes) {
                    u64 sq = mul2(x[0], x[0]), sr = mul2(y[0], y[0]);
#pragma unroll
                    for (int e = 1; e < 4; e++) sq = fma2(x[e], x[e], sq), sr = fma2(y[e], y[e], sr);
                    const float2 f = of_two(sq), h = of_two(sr);
                    float ss = (f.x + f.y) + (h.x + h.y);
#pragma unroll
                    for (int o = L / 2; o; o >>= 1) ss += __shfl_xor_sync(lanes, ss, o);
                    return ss * (1.f / D);
                };
                float mean = squares(0xffffffffu) + a.eps;
                if (norm[u]) {
                    if (!(mean > 1e-30f && mean < 1e37f)) {
                        // squares that fp32 does not hold, or the norm of next to nothing: 2^100 times or 2^-100 of the head
                        // (its lanes have one mean, so they come here together)
                        const float k = mean < 1.f ? 0x1p100f : 0x1p-100f;
                        const u64 k2 = two(k, k);
#pragma unroll
                        for (int e = 0; e < 4; e++) x[e] = mul2(x[e], k2), y[e] = mul2(y[e], k2);
                        mean = squares(((1u << L) - 1) << (tid & 31 & ~(L - 1))) + a.eps * k * k;
                    }
                    const float inv = rsqrtf(mean);
                    const u64 inv2 = two(inv, inv);
                    u64 ga[4], gb[4];
                    lds2(&gammas[side[u]][d0], ga), lds2(&gammas[side[u]][d1], gb);
#pragma unroll
                    for (int e = 0; e < 4; e++) x[e] = mul2(mul2(x[e], inv2), ga[e]), y[e] = mul2(mul2(y[e], inv2), gb[e]);
                }
            }
            if (turned) {
                if (!NORMS) angles();   // (once for each head, for the registers)
                auto turn = [](u64 &a, u64 &b, u64 c, u64 s) {
                    const u64 y = fma2(b, s ^ 0x8000000080000000ull, mul2(a, c));
                    b = fma2(a, s, mul2(b, c));
                    a = y;
                };
                if (INTER) {
                    // pairs side by side: (a, b) apart, and back
                    auto apart = [&](u64 &a, u64 &b, u64 c, u64 s) {
                        const float2 f = of_two(a), h = of_two(b);
                        u64 p = two(f.x, h.x), q = two(f.y, h.y);
                        turn(p, q, c, s);
                        const float2 v = of_two(p), z = of_two(q);
                        a = two(v.x, z.x), b = two(v.y, z.y);
                    };
                    apart(x[0], x[1], cs[0], sn[0]), apart(x[2], x[3], cs[1], sn[1]);
                    apart(y[0], y[1], cs[2], sn[2]), apart(y[2], y[3], cs[3], sn[3]);
                } else {
#pragma unroll
                    for (int e = 0; e < 4; e++) turn(x[e], y[e], cs[e], sn[e]);
                }
            }
            if (live && on[u]) {
                *reinterpret_cast<uint4 *>(out[u] + d0) = make_uint4(pack(x[0]), pack(x[1]), pack(x[2]), pack(x[3]));
                *reinterpret_cast<uint4 *>(out[u] + d1) = make_uint4(pack(y[0]), pack(y[1]), pack(y[2]), pack(y[3]));
            }
            out[u] += side[u] ? a.kos : a.qos;
        }
    }
}

template <int D, bool INTER>
cudaError_t rotary_launch(const RotaryArgs &a, dim3 grid, int threads, cudaStream_t st) {
    return a.qg || a.kg ? launch_pdl(moe_rotary_kernel<D, INTER, true>, grid, dim3(threads), 0, st, a)
                        : launch_pdl(moe_rotary_kernel<D, INTER, false>, grid, dim3(threads), 0, st, a);
}
template <int D>
cudaError_t rotary_launch(const RotaryArgs &a, bool inter, dim3 grid, int threads, cudaStream_t st) {
    return inter ? rotary_launch<D, true>(a, grid, threads, st) : rotary_launch<D, false>(a, grid, threads, st);
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
        if (((uintptr_t)s.x | (uintptr_t)s.o) & 15u) return moe_fail_status(MOE_EINVAL, "rows must be 16-byte aligned");
        if (s.xs < s.row || s.os < s.row || s.xs % 8 || s.os % 8)
            return moe_fail_status(MOE_EINVAL, "row strides must be multiples of 8 and at least %lld elements", s.row);
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
    // several tokens a CTA where there are enough for all SMs' CTAs; few tokens:
    // heads over CTAs, a warp or two each
    a.tokens = n_tokens >= 4096 ? kTokens : n_tokens >= 1024 ? 2 : 1;
    const int lanes = p->D / 16, groups = (q_heads + kv_heads + kHeads - 1) / kHeads, most = (n_tokens >= 512 ? kMaxThreads : 64) / lanes;
    const int parts = (groups + most - 1) / most, threads = (((groups + parts - 1) / parts) * lanes + 31) / 32 * 32;
    const dim3 grid((unsigned)((n_tokens + a.tokens - 1) / a.tokens), (unsigned)parts);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = p->D == 64 ? rotary_launch<64>(a, p->inter, grid, threads, st) : p->D == 128 ? rotary_launch<128>(a, p->inter, grid, threads, st)
                                                                                              : rotary_launch<256>(a, p->inter, grid, threads, st);
    return e == cudaSuccess ? MOE_OK : moe_fail_status(MOE_ECUDA, "moe_rotary_apply: %s", cudaGetErrorString(e));
}

}  // extern "C"
