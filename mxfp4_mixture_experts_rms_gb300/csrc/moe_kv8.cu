// moe_kv8.cu -- the 8-bit paged key/value cache: the entry points, and the
// append.  Codes are E4M3 with one E8M0 scale for each page of tokens and kv
// head (moe_kv8.cuh has the layout); the attention over it is in
// moe_kv8_attend.cu.
#include "moe_kv8.cuh"
#include "../../include/moe.h"

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstring>
#include <new>

namespace {

// ---- append ----
// Tokens whose slots follow one another inside a page form a run.  A run is
// written by one warp per kv head and side (keys, values): the largest
// magnitude, the page's new exponent, the earlier tokens' codes re-rounded if
// the exponent rose, the new codes.  With amax = m * 2^e (m in [1, 2)) the
// exponent ceil(log2(amax / 448)) is e - 8 + (m > 1.75): no division.
//
// A run that fills its page (all but the ends of a prompt) is read once, into
// registers, 16 bytes a load; values' codes are turned through shared memory.
// Other runs are read likewise, a page's places with those of others left out,
// and merged into the words that hold them.
// Bound by HBM for prompts (4 bytes read, 2 written a value pair; 22 559 tokens
// of 8 heads of 128: 30 us, 21 at HBM's rate).  What is above it is the CTAs
// with a page's part: the pages that are filled are done after 25 us, and a CTA
// with the end of one prompt and the beginning of the next takes 11 (47 us when
// those loaded value after value, 39 with a group of values at a time).  Four
// CTAs an SM that hold a page in registers: 30.0 us, five that hold less 31.7.
// A decode step is a chain of four dependent loads (48 tokens: 4.3 us).
__device__ __forceinline__ int kv8_exponent(float amax) {
    const uint32_t b = min(max(__float_as_uint(amax), 0x04E00000u), 0x7F7FFFFFu);  // at least 448 * 2^-126, finite
    return (int)(b >> 23) - 135 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);
}
__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
// The larger of am and the magnitudes of four bf16 pairs (NaN passes over).
__device__ __forceinline__ float amax8(float am, const uint4 v) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; i++) am = fmaxf(am, fmaxf(fabsf(bf16_lo(w[i])), fabsf(bf16_hi(w[i]))));
    return am;
}
// The same on the bits, as two 16-bit lanes; a NaN shows as more than 0x7F80.
__device__ __forceinline__ uint32_t bits8(uint32_t m, const uint4 v) {
    m = __vmaxu2(__vmaxu2(m, v.x & 0x7FFF7FFFu), v.y & 0x7FFF7FFFu);
    return __vmaxu2(__vmaxu2(m, v.z & 0x7FFF7FFFu), v.w & 0x7FFF7FFFu);
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int m = 16; m; m >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, m));
    return v;
}
// Four bf16 pairs times a power of two -> eight codes.
__device__ __forceinline__ uint2 encode8(const uint4 v, float inv) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; i++) c[i] = f32x2_to_e4m3(bf16_lo(w[i]) * inv, bf16_hi(w[i]) * inv);
    return make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
}
// Four codes times f (a power of two at most 1), rounded again.
__device__ __forceinline__ uint32_t requant4(uint32_t w, float f) {
    const float2 a = e4m3x2_to_f32(w), b = e4m3x2_to_f32(w >> 16);
    return f32x2_to_e4m3(a.x * f, a.y * f) | (f32x2_to_e4m3(b.x * f, b.y * f) << 16);
}

constexpr int kAppendWarps = 4;
constexpr int kMaxWindow = 64;  // tokens of one CTA

// 16 tokens of 4 dims from [token][dim] bytes to the page's words: word q of a
// dim holds tokens 2 q, 2 q + 1, 8 + 2 q, 9 + 2 q.
template <int D>
__device__ __forceinline__ void turn_words(const uint8_t *from, uint32_t (&out)[4][4]) {
    uint32_t in[16];
#pragma unroll
    for (int t = 0; t < 16; t++) in[t] = *reinterpret_cast<const uint32_t *>(from + t * D);
#pragma unroll
    for (int q = 0; q < 4; q++) {
        const uint32_t a0 = __byte_perm(in[2 * q], in[2 * q + 1], 0x5140), a1 = __byte_perm(in[2 * q], in[2 * q + 1], 0x7362);
        const uint32_t b0 = __byte_perm(in[8 + 2 * q], in[9 + 2 * q], 0x5140), b1 = __byte_perm(in[8 + 2 * q], in[9 + 2 * q], 0x7362);
        out[0][q] = __byte_perm(a0, b0, 0x5410), out[1][q] = __byte_perm(a0, b0, 0x7632);
        out[2][q] = __byte_perm(a1, b1, 0x5410), out[3][q] = __byte_perm(a1, b1, 0x7632);
    }
}

// A page's run; x: its first row, at this kv head; base: the page's codes;
// turn: P * D bytes of the warp's own; returns the scale byte.
template <int D, int P>
__device__ __forceinline__ int append_page(bool keys, const uint16_t *x, long long stride, uint8_t *base, uint8_t *turn, int lane) {
    // a warp reads kTok tokens at a time, 16 bytes (8 dims) a lane; up to 16
    // loads held, the others read again
    constexpr int kTok = 256 / D, N = P / kTok, HELD = N < 16 ? N : 16;
    const int tok = lane / (D / 8), ch = lane % (D / 8);
    const uint16_t *p = x + (long long)tok * stride + 8 * ch;
    const long long step = kTok * stride;
    uint4 v[HELD];
#pragma unroll
    for (int i = 0; i < HELD; i++) v[i] = __ldg(reinterpret_cast<const uint4 *>(p + i * step));
    uint32_t m = 0;
#pragma unroll 4
    for (int i = HELD; i < N; i++) m = bits8(m, __ldg(reinterpret_cast<const uint4 *>(p + i * step)));
#pragma unroll
    for (int i = 0; i < HELD; i++) m = bits8(m, v[i]);
    m = __reduce_max_sync(0xffffffffu, max(m & 0xFFFFu, m >> 16));
    float am = __uint_as_float(m << 16);
    if (m > 0x7F80u) {
        am = 0.f;
#pragma unroll 1
        for (int i = 0; i < N; i++) am = amax8(am, __ldg(reinterpret_cast<const uint4 *>(p + i * step)));
        am = warp_max(am);
    }
    const int byte = kv8_exponent(am) + 127;
    const float inv = pow2i(127 - byte);
    uint8_t *to = keys ? base + (ch / 2) * (P * 16) + tok * 16 + (ch % 2) * 8 : turn + tok * D + ch * 8;
    const int next = keys ? kTok * 16 : kTok * D;
#pragma unroll
    for (int i = 0; i < HELD; i++, to += next) *reinterpret_cast<uint2 *>(to) = encode8(v[i], inv);
#pragma unroll 4
    for (int i = HELD; i < N; i++, to += next) *reinterpret_cast<uint2 *>(to) = encode8(__ldg(reinterpret_cast<const uint4 *>(p + i * step)), inv);
    if (!keys) {
        // values lie [token][dim]: 4 dims and 16 tokens a lane, turned by words
        __syncwarp();
#pragma unroll 1
        for (int w = lane; w < P / 16 * (D / 4); w += 32) {
            const int g = w / (D / 4), d = 4 * (w % (D / 4));
            uint32_t out[4][4];
            turn_words<D>(turn + 16 * g * D + d, out);
            uint4 *o = reinterpret_cast<uint4 *>(base + g * (D * 16) + d * 16);
#pragma unroll
            for (int e = 0; e < 4; e++) o[e] = make_uint4(out[e][0], out[e][1], out[e][2], out[e][3]);
        }
        __syncwarp();   // the buffer is the next run's
    }
    return byte;
}

// A run of len tokens from place o0 on; old: the page's scale byte (0: it starts here).
template <int D, int P>
__device__ __forceinline__ int append_run(bool keys, const uint16_t *x, long long stride, uint8_t *base, uint8_t *turn, int o0, int len, int old, int lane) {
    // places as append_page has them, loaded where they are the run's
    constexpr int kTok = 256 / D, N = P / kTok, HELD = N < 16 ? N : 16;
    const int tok = lane / (D / 8), ch = lane % (D / 8);
    const uint16_t *p = x + (long long)(tok - o0) * stride + 8 * ch;
    const long long step = kTok * stride;
    auto mine = [&](int i) { return (unsigned)(i * kTok + tok - o0) < (unsigned)len; };
    auto load = [&](int i) { return mine(i) ? __ldg(reinterpret_cast<const uint4 *>(p + i * step)) : make_uint4(0, 0, 0, 0); };
    const int i0 = o0 / kTok, i1 = (o0 + len - 1) / kTok + 1;   // of any lane
    uint4 v[HELD];
#pragma unroll
    for (int i = 0; i < HELD; i++) v[i] = load(i);
    uint32_t m = 0;
#pragma unroll 4
    for (int i = HELD; i < N; i++) m = bits8(m, load(i));
#pragma unroll
    for (int i = 0; i < HELD; i++) m = bits8(m, v[i]);
    m = __reduce_max_sync(0xffffffffu, max(m & 0xFFFFu, m >> 16));
    float am = __uint_as_float(m << 16);
    if (m > 0x7F80u) {
        am = 0.f;
#pragma unroll 1
        for (int i = i0; i < i1; i++) am = amax8(am, load(i));
        am = warp_max(am);
    }
    const int now = max(kv8_exponent(am) + 127, old);
    const float inv = pow2i(127 - now), shrink = pow2i(old - now);
    const bool again = o0 > 0 && now > old;
    uint8_t *to = keys ? base + (ch / 2) * (P * 16) + tok * 16 + (ch % 2) * 8 : turn + tok * D + ch * 8;
    const int next = keys ? kTok * 16 : kTok * D;
#pragma unroll
    for (int i = 0; i < HELD; i++)
        if (mine(i)) *reinterpret_cast<uint2 *>(to + i * next) = encode8(v[i], inv);
#pragma unroll 4
    for (int i = HELD; i < N; i++)
        if (mine(i)) *reinterpret_cast<uint2 *>(to + i * next) = encode8(load(i), inv);
    if (keys) {
        if (again)
#pragma unroll 4
            for (int u = lane; u < o0 * (D / 16); u += 32) {
                uint4 *q = reinterpret_cast<uint4 *>(base + (size_t)(u % (D / 16)) * P * 16 + u / (D / 16) * 16);
                uint4 w = *q;
                w.x = requant4(w.x, shrink), w.y = requant4(w.y, shrink);
                w.z = requant4(w.z, shrink), w.w = requant4(w.w, shrink);
                *q = w;
            }
        return now;
    }
    // values: 4 dims and 16 tokens a lane; bytes of tokens outside the run keep
    // their codes (earlier ones re-rounded if the exponent rose)
    __syncwarp();
    const int g0 = again ? 0 : o0 / 16, g1 = (o0 + len + 15) / 16;
#pragma unroll 1
    for (int w = lane; w < (g1 - g0) * (D / 4); w += 32) {
        const int g = g0 + w / (D / 4), d = 4 * (w % (D / 4));
        uint4 *o = reinterpret_cast<uint4 *>(base + g * (D * 16) + d * 16);
        uint4 was[4];
#pragma unroll
        for (int e = 0; e < 4; e++) was[e] = o[e];
        uint32_t out[4][4], fresh[4], past[4];   // of the words' bytes: the run's, those before
        turn_words<D>(turn + 16 * g * D + d, out);
#pragma unroll
        for (int q = 0; q < 4; q++) {
            fresh[q] = past[q] = 0;
#pragma unroll
            for (int e = 0; e < 4; e++) {
                const int place = 16 * g + 2 * q + (e & 1) + 8 * (e >> 1);
                if ((unsigned)(place - o0) < (unsigned)len) fresh[q] |= 0xFFu << (8 * e);
                if (place < o0) past[q] |= 0xFFu << (8 * e);
            }
        }
#pragma unroll
        for (int e = 0; e < 4; e++) {
            uint32_t x4[4] = {was[e].x, was[e].y, was[e].z, was[e].w};
#pragma unroll
            for (int q = 0; q < 4; q++) {
                if (again) x4[q] = (x4[q] & ~past[q]) | (requant4(x4[q], shrink) & past[q]);
                x4[q] = (x4[q] & ~fresh[q]) | (out[e][q] & fresh[q]);
            }
            o[e] = make_uint4(x4[0], x4[1], x4[2], x4[3]);
        }
    }
    __syncwarp();   // the buffer is the next run's
    return now;
}

// Window of tokens blockIdx.x; warps over (kv head, side) pairs.
template <int D, int P>
__global__ void __launch_bounds__(kAppendWarps * 32, 4) moe_kv8_append_kernel(Kv8Cache c, const uint16_t *k, const uint16_t *v,
                                                                           long long k_stride, long long v_stride,
                                                                           const int32_t *slots, int n, int window) {
    __shared__ __align__(16) uint8_t turn[kAppendWarps][P * D];
    __shared__ int s[kMaxWindow + 1 + 64];  // slot of the token before, the window's, those a run can reach into
    const int tid = threadIdx.x, lane = tid & 31, pair = blockIdx.y * kAppendWarps + (tid >> 5);
    const int t0 = blockIdx.x * window, total = c.n_pages * P;
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    for (int i = tid; i < window + 65; i += kAppendWarps * 32) {
        const int t = t0 - 1 + i;
        const int x = t >= 0 && t < n ? slots[t] : -1;
        s[i] = x >= 0 && x < total ? x : -1;
    }
    __syncthreads();
    if (pair >= 2 * c.KVH) return;
    const int h = pair >> 1;
    const bool keys = (pair & 1) == 0;
    const uint16_t *x = (keys ? k : v) + h * D;
    const long long stride = keys ? k_stride : v_stride;
    uint8_t *codes = keys ? c.k : c.v, *scales = keys ? c.ks : c.vs;
    // does token i of the window (i >= 0) continue the run of the one before?
    auto cont = [&](int i) { return s[i + 1] > 0 && s[i] + 1 == s[i + 1] && s[i + 1] % P != 0; };
    for (int w0 = 0; w0 < window; w0 += 32) {
        const int i = w0 + lane;
        unsigned lead = __ballot_sync(0xffffffffu, i < window && s[i + 1] >= 0 && !cont(i));
        for (; lead; lead &= lead - 1) {
            const int at = w0 + __ffs(lead) - 1;
            // the run's length: continuations that follow, at most P - 1
            const unsigned c0 = __ballot_sync(0xffffffffu, !(at + 1 + lane < window + 64 && cont(at + 1 + lane)));
            const unsigned c1 = __ballot_sync(0xffffffffu, !(at + 33 + lane < window + 64 && cont(at + 33 + lane)));
            const int len = 1 + (c0 ? __ffs(c0) - 1 : 32 + (c1 ? __ffs(c1) - 1 : 32));
            const int slot = s[at + 1], page = slot / P, o0 = slot % P;
            const size_t ph = (size_t)page * c.KVH + h;
            const uint16_t *row = x + (long long)(t0 + at) * stride;
            uint8_t *base = codes + ph * (size_t)(P * D);
            const int byte = len == P ? append_page<D, P>(keys, row, stride, base, turn[tid >> 5], lane)
                                      : append_run<D, P>(keys, row, stride, base, turn[tid >> 5], o0, len, o0 ? scales[ph] : 0, lane);
            __syncwarp();
            if (lane == 0) scales[ph] = (uint8_t)byte;
        }
    }
}

template <int D, int P>
cudaError_t append_launch(const Kv8Cache &c, const uint16_t *k, const uint16_t *v, long long k_stride, long long v_stride,
                          const int32_t *slots, int n, cudaStream_t st) {
    // Prompts: a page of tokens a CTA, as a rule one run.  Few tokens: each its
    // own run as a rule, two a warp keep a decode step's launch to one wave.  us
    // at 512, 1024, 2048 tokens, 8 heads of 64, pages of 64, windows of two and of
    // a page: tokens of as many sequences 12.6 and 112, 20.6 and 113, 36.8 and 118
    // (pages of 16: 9.9 and 23.6, 15.4 and 24.9, 26.7 and 27.2); one prompt's 4.5
    // and 5.1, 5.9 and 5.1, 8.6 and 5.3.
    const int window = n <= 1024 ? 2 : P;
    const dim3 grid((n + window - 1) / window, (2 * c.KVH + kAppendWarps - 1) / kAppendWarps), block(kAppendWarps * 32);
    return launch_pdl(moe_kv8_append_kernel<D, P>, grid, block, 0, st, c, k, v, k_stride, v_stride, slots, n, window);
}
template <int D>
cudaError_t append_size(const Kv8Cache &c, const uint16_t *k, const uint16_t *v, long long k_stride, long long v_stride,
                        const int32_t *slots, int n, cudaStream_t st) {
    return c.P == 16   ? append_launch<D, 16>(c, k, v, k_stride, v_stride, slots, n, st)
           : c.P == 32 ? append_launch<D, 32>(c, k, v, k_stride, v_stride, slots, n, st)
                       : append_launch<D, 64>(c, k, v, k_stride, v_stride, slots, n, st);
}

bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }

}  // namespace

cudaError_t launch_kv8_append(const Kv8Cache &c, const uint16_t *k, const uint16_t *v, long long k_stride,
                              long long v_stride, const int32_t *slots, int n, cudaStream_t st) {
    return c.D == 64 ? append_size<64>(c, k, v, k_stride, v_stride, slots, n, st) : append_size<128>(c, k, v, k_stride, v_stride, slots, n, st);
}

struct moe_kv8 {
    Kv8Cache c{};
    int QH = 0, window = 0;
    float scale = 0.f;
    const float *sinks = nullptr;
    unsigned char *ws = nullptr;
};

extern "C" {

moe_kv8 *moe_kv8_create(int q_heads, int kv_heads, int head_dim, int page_size, int n_pages) {
    if (kv_heads < 1 || kv_heads > 256 || q_heads < 1 || q_heads % kv_heads != 0 || q_heads / kv_heads > kKv8MaxGroup ||
        (head_dim != 64 && head_dim != 128) || (page_size != 16 && page_size != 32 && page_size != 64) || n_pages < 1 ||
        (long long)n_pages * page_size > INT_MAX) {
        moe_set_error("moe_kv8_create: bad arguments (1..256 kv heads, q_heads a multiple of kv_heads with at most %d "
                      "per kv head, head_dim 64 or 128, page_size 16, 32 or 64, n_pages * page_size at most 2^31 - 1)",
                      kKv8MaxGroup);
        return nullptr;
    }
    moe_kv8 *p = new (std::nothrow) moe_kv8;
    if (!p) {
        moe_set_error("moe_kv8_create: out of host memory");
        return nullptr;
    }
    p->c.KVH = kv_heads, p->c.D = head_dim, p->c.P = page_size, p->c.n_pages = n_pages;
    p->QH = q_heads;
    p->scale = 1.0f / std::sqrt((float)head_dim);
    return p;
}

void moe_kv8_destroy(moe_kv8 *p) { delete p; }

int moe_kv8_get_device_status(moe_kv8 *p, int *status, void *stream) {
    if (!p || !status) return moe_fail_status(MOE_EINVAL, "NULL argument");
    if (!p->ws) return moe_fail_status(MOE_ENOTREADY, "moe_kv8_set_workspace has not been called");
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    int32_t h[2] = {0, 0};
    cudaError_t e = cudaMemcpyAsync(h, p->ws, sizeof h, cudaMemcpyDeviceToHost, st);
    if (e == cudaSuccess) e = cudaStreamSynchronize(st);
    if (e == cudaSuccess && h[0]) {
        // a share that gave up may have left its tickets: all of them start over
        e = cudaMemsetAsync(p->ws, 0, kKv8ClearBytes, st);
        if (e == cudaSuccess) e = cudaStreamSynchronize(st);
    }
    if (e != cudaSuccess) return moe_fail_status(MOE_ECUDA, "moe_kv8_get_device_status: %s", cudaGetErrorString(e));
    *status = h[0];
    if (h[0]) return moe_fail_status(MOE_EDEVICE, "device status %d (detail %d)", h[0], h[1]);
    return MOE_OK;
}

int moe_kv8_set_i(moe_kv8 *p, const char *key, long long v) {
    if (!p || !key) return moe_fail_status(MOE_EINVAL, "NULL argument");
    if (strcmp(key, "sliding_window")) return moe_fail_status(MOE_EINVAL, "unknown integer option '%s'", key);
    if (v < 0 || v > INT_MAX) return moe_fail_status(MOE_EINVAL, "sliding_window must be 0..2^31 - 1");
    p->window = (int)v;
    return MOE_OK;
}

int moe_kv8_set_f(moe_kv8 *p, const char *key, double v) {
    if (!p || !key) return moe_fail_status(MOE_EINVAL, "NULL argument");
    if (strcmp(key, "softmax_scale")) return moe_fail_status(MOE_EINVAL, "unknown floating option '%s'", key);
    if (!(v > 1e-30 && v < 1e30)) return moe_fail_status(MOE_EINVAL, "softmax_scale must be positive (1e-30 .. 1e30)");
    p->scale = (float)v;
    return MOE_OK;
}

int moe_kv8_set_cache(moe_kv8 *p, uint8_t *k, uint8_t *v, uint8_t *k_scales, uint8_t *v_scales) {
    if (!p || !k || !v || !k_scales || !v_scales) return moe_fail_status(MOE_EINVAL, "NULL argument");
    if (!aligned16(k) || !aligned16(v)) return moe_fail_status(MOE_EINVAL, "the code arrays must be 16-byte aligned");
    p->c.k = k, p->c.v = v, p->c.ks = k_scales, p->c.vs = v_scales;
    return MOE_OK;
}

int moe_kv8_set_sinks(moe_kv8 *p, const float *sinks) {
    if (!p) return moe_fail_status(MOE_EINVAL, "NULL plan");
    if ((uintptr_t)sinks & 3u) return moe_fail_status(MOE_EINVAL, "sinks must be 4-byte aligned");
    p->sinks = sinks;
    return MOE_OK;
}

size_t moe_kv8_workspace_bytes(const moe_kv8 *p) { return p ? kv8_workspace_bytes(p->c.D) : 0; }

int moe_kv8_set_workspace(moe_kv8 *p, void *dev, size_t bytes) {
    if (!p || !dev) return moe_fail_status(MOE_EINVAL, "NULL argument");
    if ((uintptr_t)dev & 255u) return moe_fail_status(MOE_EINVAL, "the workspace must be 256-byte aligned");
    const size_t need = kv8_workspace_bytes(p->c.D);
    if (bytes < need) return moe_fail_status(MOE_ENOMEM, "workspace of %zu bytes, %zu needed", bytes, need);
    // what is queued on any stream may still use the memory, and what is queued
    // next may be on a stream that does not wait for the one of the memset
    cudaError_t e = cudaDeviceSynchronize();
    if (e == cudaSuccess) e = cudaMemset(dev, 0, kKv8ClearBytes);
    if (e == cudaSuccess) e = cudaDeviceSynchronize();
    if (e != cudaSuccess) return moe_fail_status(MOE_ECUDA, "moe_kv8_set_workspace: %s", cudaGetErrorString(e));
    p->ws = static_cast<unsigned char *>(dev);
    return MOE_OK;
}

int moe_kv8_append(moe_kv8 *p, const uint16_t *k, const uint16_t *v, long long k_stride, long long v_stride,
                   const int32_t *slots, int n_tokens, void *stream) {
    if (!p) return moe_fail_status(MOE_EINVAL, "NULL plan");
    if (!p->c.k) return moe_fail_status(MOE_ENOTREADY, "moe_kv8_set_cache has not been called");
    if (n_tokens < 0) return moe_fail_status(MOE_EINVAL, "n_tokens must be >= 0");
    if (n_tokens == 0) return MOE_OK;
    if (!k || !v || !slots) return moe_fail_status(MOE_EINVAL, "NULL k, v or slots");
    if (!aligned16(k) || !aligned16(v) || ((uintptr_t)slots & 3u))
        return moe_fail_status(MOE_EINVAL, "k and v must be 16-byte aligned, slots 4-byte aligned");
    const long long row = (long long)p->c.KVH * p->c.D;
    if (k_stride < row || v_stride < row || k_stride % 8 || v_stride % 8)
        return moe_fail_status(MOE_EINVAL, "row strides must be multiples of 8 and at least %lld elements", row);
    const cudaError_t e = launch_kv8_append(p->c, k, v, k_stride, v_stride, slots, n_tokens, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? MOE_OK : moe_fail_status(MOE_ECUDA, "moe_kv8_append: %s", cudaGetErrorString(e));
}

int moe_kv8_attend(moe_kv8 *p, const uint16_t *q, long long q_stride, const int32_t *starts, const int32_t *lens,
                   const int32_t *table, int table_width, int n_seqs, int max_new, int n_rows, uint16_t *out,
                   long long out_stride, void *stream) {
    if (!p) return moe_fail_status(MOE_EINVAL, "NULL plan");
    if (!p->c.k) return moe_fail_status(MOE_ENOTREADY, "moe_kv8_set_cache has not been called");
    if (!p->ws) return moe_fail_status(MOE_ENOTREADY, "moe_kv8_set_workspace has not been called");
    if (n_seqs < 0 || n_seqs > kKv8MaxSeqs) return moe_fail_status(MOE_EINVAL, "n_seqs must be 0..%d", kKv8MaxSeqs);
    if (n_rows < 0 || table_width < 0 || max_new < 0)
        return moe_fail_status(MOE_EINVAL, "n_rows, table_width and max_new must be >= 0");
    if ((long long)table_width * p->c.P > (1ll << 30) ||
        ((long long)table_width * p->c.P / 64 + 2) * 4 * n_seqs * p->c.KVH > INT_MAX)
        return moe_fail_status(MOE_EINVAL, "table_width %d: at most 2^30 tokens a sequence, and 2^35 token places over "
                               "all sequences and kv heads", table_width);
    if (max_new > 65535) return moe_fail_status(MOE_EINVAL, "max_new must be at most 65535");
    if (!starts && (n_rows != n_seqs || max_new != 1))
        return moe_fail_status(MOE_EINVAL, "without starts every sequence has one row: n_rows = n_seqs, max_new = 1");
    if (n_seqs == 0 || n_rows == 0 || max_new == 0) return MOE_OK;
    if (!q || !lens || !out || (!table && table_width)) return moe_fail_status(MOE_EINVAL, "NULL q, lens, table or out");
    if (!aligned16(q) || !aligned16(out) || (((uintptr_t)lens | (uintptr_t)table | (uintptr_t)starts) & 3u))
        return moe_fail_status(MOE_EINVAL, "q and out must be 16-byte aligned, starts, lens and table 4-byte aligned");
    const long long row = (long long)p->QH * p->c.D;
    if (q_stride < row || out_stride < row || q_stride % 8 || out_stride % 8)
        return moe_fail_status(MOE_EINVAL, "row strides must be multiples of 8 and at least %lld elements", row);
    // their extents lie apart, or (rows of one array) their places in a row do
    const uint16_t *qe = q + (long long)(n_rows - 1) * q_stride + row, *oe = out + (long long)(n_rows - 1) * out_stride + row;
    const long long apart = q_stride == out_stride ? (((long long)(out - q)) % q_stride + q_stride) % q_stride : 0;
    if (q < oe && out < qe && (apart < row || apart > q_stride - row))
        return moe_fail_status(MOE_EINVAL, "q and out must not overlap");
    Kv8Attend a{};
    a.c = p->c;
    a.QH = p->QH, a.window = p->window, a.n_seqs = n_seqs, a.n_rows = n_rows, a.max_new = max_new, a.width = table_width;
    a.scale = p->scale, a.sinks = p->sinks, a.q = q, a.out = out, a.q_stride = q_stride, a.o_stride = out_stride;
    a.starts = starts, a.lens = lens, a.table = table;
    const cudaError_t e = launch_kv8_attend(a, p->ws, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? MOE_OK : moe_fail_status(MOE_ECUDA, "moe_kv8_attend: %s", cudaGetErrorString(e));
}

}  // extern "C"
