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
__device__ __forceinline__ int kv8_exponent(float amax) {
    const uint32_t b = min(max(__float_as_uint(amax), 0x04E00000u), 0x7F7FFFFFu);  // at least 448 * 2^-126, finite
    return (int)(b >> 23) - 135 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);
}

__device__ __forceinline__ void bf16x8(const uint4 v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; i++) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

// Four codes times f (a power of two at most 1), rounded again.
__device__ __forceinline__ uint32_t requant4(uint32_t w, float f) {
    const float2 a = e4m3x2_to_f32(w), b = e4m3x2_to_f32(w >> 16);
    return f32x2_to_e4m3(a.x * f, a.y * f) | (f32x2_to_e4m3(b.x * f, b.y * f) << 16);
}

constexpr int kAppendWarps = 4;
constexpr int kMaxWindow = 128;  // tokens of one CTA

template <int D>
__global__ void __launch_bounds__(kAppendWarps * 32, 6) moe_kv8_append_kernel(Kv8Cache c, const uint16_t *k, const uint16_t *v,
                                                                   long long k_stride, long long v_stride,
                                                                   const int32_t *slots, int n, int window) {
    __shared__ int s[kMaxWindow + 1 + 64];  // slot of the token before, the window's, those a run can reach into
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int t0 = blockIdx.x * window, h = blockIdx.y;
    const bool keys = blockIdx.z == 0;
    const int total = c.n_pages * c.P;
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    for (int i = tid; i < window + 65; i += kAppendWarps * 32) {
        const int t = t0 - 1 + i;
        const int x = t >= 0 && t < n ? slots[t] : -1;
        s[i] = x >= 0 && x < total ? x : -1;
    }
    __syncthreads();
    const uint16_t *x = keys ? k : v;
    const long long stride = keys ? k_stride : v_stride;
    uint8_t *codes = keys ? c.k : c.v, *scales = keys ? c.ks : c.vs;
    // does token i of the window (i >= 0) continue the run of the one before?
    auto cont = [&](int i) { return s[i + 1] > 0 && s[i] + 1 == s[i + 1] && s[i + 1] % c.P != 0; };
    int rank = 0;
    for (int w0 = 0; w0 < window; w0 += 32) {
        const int i = w0 + lane;
        unsigned lead = __ballot_sync(0xffffffffu, i < window && s[i + 1] >= 0 && !cont(i));
        while (lead) {
            const int at = w0 + __ffs(lead) - 1;
            lead &= lead - 1;
            if (rank++ % kAppendWarps != warp) continue;
            // the run's length: continuations that follow, at most P - 1
            const unsigned c0 = __ballot_sync(0xffffffffu, !(at + 1 + lane < window + 64 && cont(at + 1 + lane)));
            const unsigned c1 = __ballot_sync(0xffffffffu, !(at + 33 + lane < window + 64 && cont(at + 33 + lane)));
            const int len = 1 + (c0 ? __ffs(c0) - 1 : 32 + (c1 ? __ffs(c1) - 1 : 32));
            const int slot = s[at + 1], page = slot / c.P, o0 = slot % c.P;
            const uint16_t *x0 = x + (long long)(t0 + at) * stride + h * D;
            // largest magnitude of the run (NaN passes over)
            float am = 0.f;
            for (int u = lane; u < len * (D / 8); u += 32) {
                float f[8];
                bf16x8(__ldg(reinterpret_cast<const uint4 *>(x0 + (long long)(u / (D / 8)) * stride) + u % (D / 8)), f);
#pragma unroll
                for (int i2 = 0; i2 < 8; i2++) am = fmaxf(am, fabsf(f[i2]));
            }
#pragma unroll
            for (int m = 16; m; m >>= 1) am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, m));
            const size_t ph = (size_t)page * c.KVH + h;
            const int need = kv8_exponent(am) + 127, old = o0 ? scales[ph] : 0;
            const int now = max(need, old);
            __syncwarp();
            if (lane == 0) scales[ph] = (uint8_t)now;
            const float inv = pow2i(127 - now), shrink = pow2i(old - now);
            const bool again = o0 > 0 && now > old;
            uint8_t *base = codes + ph * (size_t)(c.P * D);
            if (keys) {
                if (again)
                    for (int u = lane; u < o0 * (D / 16); u += 32) {
                        uint4 *p = reinterpret_cast<uint4 *>(base + (size_t)(u % (D / 16)) * c.P * 16 + u / (D / 16) * 16);
                        uint4 w = *p;
                        w.x = requant4(w.x, shrink), w.y = requant4(w.y, shrink);
                        w.z = requant4(w.z, shrink), w.w = requant4(w.w, shrink);
                        *p = w;
                    }
                for (int u = lane; u < len * (D / 16); u += 32) {
                    const int j = u / (D / 16), ch = u % (D / 16);
                    const uint4 *src = reinterpret_cast<const uint4 *>(x0 + (long long)j * stride) + 2 * ch;
                    uint32_t w[4];
#pragma unroll
                    for (int hf = 0; hf < 2; hf++) {
                        float f[8];
                        bf16x8(__ldg(src + hf), f);
#pragma unroll
                        for (int q = 0; q < 2; q++)
                            w[2 * hf + q] = f32x2_to_e4m3(f[4 * q] * inv, f[4 * q + 1] * inv) |
                                            (f32x2_to_e4m3(f[4 * q + 2] * inv, f[4 * q + 3] * inv) << 16);
                    }
                    *reinterpret_cast<uint4 *>(base + (size_t)ch * c.P * 16 + (o0 + j) * 16) = make_uint4(w[0], w[1], w[2], w[3]);
                }
            } else {
                // (16 tokens, 2 dims) at a time: bytes of tokens outside the
                // run keep their codes (re-rounded if the exponent rose)
                const int g0 = again ? 0 : o0 / 16, g1 = (o0 + len + 15) / 16;
                for (int u = lane; u < (g1 - g0) * (D / 2); u += 32) {
                    const int gr = g0 + u / (D / 2), d = 2 * (u % (D / 2));
                    uint4 *p = reinterpret_cast<uint4 *>(base + (size_t)gr * D * 16 + d * 16);
                    uint32_t w[8];
                    const bool whole = gr * 16 >= o0 && gr * 16 + 16 <= o0 + len;
                    if (!whole) {
                        const uint4 a = p[0], b = p[1];
                        w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
                        w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
                    }
#pragma unroll
                    for (int q = 0; q < 4; q++) {
                        // tokens 2q, 2q + 1, 8 + 2q, 9 + 2q of the group in byte order
                        uint32_t n0 = whole ? 0 : w[q], n1 = whole ? 0 : w[4 + q];
                        const uint32_t r0 = again ? requant4(n0, shrink) : n0, r1 = again ? requant4(n1, shrink) : n1;
#pragma unroll
                        for (int e = 0; e < 4; e++) {
                            const int tok = gr * 16 + 2 * q + (e & 1) + 8 * (e >> 1), sh = 8 * e;
                            if (tok >= o0 && tok < o0 + len) {
                                const uint32_t pr = __ldg(reinterpret_cast<const uint32_t *>(x0 + (long long)(tok - o0) * stride + d));
                                const uint32_t cd = f32x2_to_e4m3(__uint_as_float(pr << 16) * inv, __uint_as_float(pr & 0xFFFF0000u) * inv);
                                n0 = (n0 & ~(0xFFu << sh)) | ((cd & 0xFFu) << sh);
                                n1 = (n1 & ~(0xFFu << sh)) | ((cd >> 8) << sh);
                            } else if (again && tok < o0) {
                                n0 = (n0 & ~(0xFFu << sh)) | (r0 & (0xFFu << sh));
                                n1 = (n1 & ~(0xFFu << sh)) | (r1 & (0xFFu << sh));
                            }
                        }
                        w[q] = n0, w[4 + q] = n1;
                    }
                    p[0] = make_uint4(w[0], w[1], w[2], w[3]);
                    p[1] = make_uint4(w[4], w[5], w[6], w[7]);
                }
            }
        }
    }
}

bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }

}  // namespace

cudaError_t launch_kv8_append(const Kv8Cache &c, const uint16_t *k, const uint16_t *v, long long k_stride,
                              long long v_stride, const int32_t *slots, int n, cudaStream_t st) {
    const int window = 8;
    const dim3 grid((n + window - 1) / window, c.KVH, 2), block(kAppendWarps * 32);
    if (c.D == 64)
        return launch_pdl(moe_kv8_append_kernel<64>, grid, block, 0, st, c, k, v, k_stride, v_stride, slots, n, window);
    return launch_pdl(moe_kv8_append_kernel<128>, grid, block, 0, st, c, k, v, k_stride, v_stride, slots, n, window);
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
    const cudaError_t e = cudaMemset(dev, 0, kKv8ClearBytes);
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
    const uint16_t *qe = q + (long long)(n_rows - 1) * q_stride + row, *oe = out + (long long)(n_rows - 1) * out_stride + row;
    if (q < oe && out < qe) return moe_fail_status(MOE_EINVAL, "q and out must not overlap");
    Kv8Attend a{};
    a.c = p->c;
    a.QH = p->QH, a.window = p->window, a.n_seqs = n_seqs, a.n_rows = n_rows, a.max_new = max_new, a.width = table_width;
    a.scale = p->scale, a.sinks = p->sinks, a.q = q, a.out = out, a.q_stride = q_stride, a.o_stride = out_stride;
    a.starts = starts, a.lens = lens, a.table = table;
    const cudaError_t e = launch_kv8_attend(a, p->ws, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? MOE_OK : moe_fail_status(MOE_ECUDA, "moe_kv8_attend: %s", cudaGetErrorString(e));
}

}  // extern "C"
