// moe_kv4.cu -- the 4-bit paged key/value cache: the entry points, the append
// and the read.  Its format is MXFP4, that of the expert weights and of the
// activation encoder (moe_mxq.cu), one block a token, kv head, side and 32 dims
// (moe_kv4.cuh has the layout); the attention over it is in moe_kv4_attend.cu.
//
// A block does not depend on other tokens, so tokens may come in any order and
// nothing that the cache holds is rounded twice (the 8-bit cache's pages share a
// scale).  Four lanes hold a block, eight dims each, and a warp 128 dims of one
// side of eight tokens: it reads 64 bytes of each token at a time, and where the
// slots follow one another writes 128 in a row.  Bound by HBM, as long as no
// place is found by division: 22 559 tokens, 8 heads of 128, appended and read
// back take 44 us, 37 at HBM's rate (the append alone took 47 with divisions; now its
// integer pipe is 73 % busy, of the exponents and codes).
#include "moe_kv4.cuh"
#include "../../include/moe.h"

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstring>
#include <new>

namespace {

constexpr int kWarps = 4;
constexpr int kBlocks = 4;     // of a warp's tokens: 128 dims

struct RowArgs {
    Kv4Cache c;
    const uint16_t *k, *v;     // append: rows of [KVH][D]
    uint16_t *ko, *vo;         // read: the same
    long long ks, vs;          // elements from row to row
    const int32_t *slots;
    int n, shift;              // P = 1 << shift
};

// A lane's token and its slot (-1: none), the side and first kv head of its
// warp's 128 dims, and where they lie.
template <int D>
struct Place {
    static constexpr int NB = D / 32;
    int tok, slot, quarter, h;
    bool values, on;           // on: is the warp's part one of the heads'?
    size_t codes, scale;       // of block 0; block b of head h + x: + x * page bytes + b * P * 16 (codes), + b * P (scales)
    int page_bytes, P;
    __device__ __forceinline__ Place(const RowArgs &a) {
        const int lane = threadIdx.x & 31, part = blockIdx.y * kWarps + (threadIdx.x >> 5), parts = (a.c.KVH * D + 127) / 128;   // of a side
        quarter = lane & 3;
        values = part >= parts, on = part < 2 * parts;
        h = (part - (values ? parts : 0)) * (128 / D);
        tok = blockIdx.x * 8 + (lane >> 2);
        P = 1 << a.shift, page_bytes = kv4_page_bytes(P, D);
        const int s = tok < a.n ? __ldg(a.slots + tok) : -1;
        slot = s >= 0 && s < a.c.n_pages << a.shift ? s : -1;
        const int page = max(slot, 0) >> a.shift, place = max(slot, 0) & (P - 1);
        const size_t at = ((size_t)page * a.c.KVH + h) * page_bytes;
        codes = at + (values ? P * D / 2 : 0) + place * 16 + 4 * quarter;
        scale = at + P * D + (values ? P * NB : 0) + (place & ~15) + kv4_scale_byte(place & 15);
    }
    __device__ __forceinline__ bool has(const RowArgs &a, int i) const { return on && slot >= 0 && h + i / NB < a.c.KVH; }   // block i of the 128 dims
    __device__ __forceinline__ size_t code_at(int i) const { return codes + (size_t)(i / NB) * page_bytes + (i % NB) * P * 16; }
    __device__ __forceinline__ size_t scale_at(int i) const { return scale + (size_t)(i / NB) * page_bytes + (i % NB) * P; }
};

template <int D>
__global__ void __launch_bounds__(kWarps * 32) moe_kv4_append_kernel(const RowArgs a) {
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const Place<D> p(a);
    const uint4 *row = reinterpret_cast<const uint4 *>((p.values ? a.v + p.tok * a.vs : a.k + p.tok * a.ks) + p.h * D) + p.quarter;
    uint4 w[kBlocks];
#pragma unroll
    for (int i = 0; i < kBlocks; i++) w[i] = p.has(a, i) ? __ldg(row + 4 * i) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < kBlocks; i++) {
        const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
        float f[8];
#pragma unroll
        for (int q = 0; q < 4; q++) f[2 * q] = __uint_as_float(u[q] << 16), f[2 * q + 1] = __uint_as_float(u[q] & 0xFFFF0000u);
        // the largest magnitude by its bits, two at a time; a NaN shows as more than infinity
        uint32_t m = __vmaxu2(__vmaxu2(u[0] & 0x7FFF7FFFu, u[1] & 0x7FFF7FFFu), __vmaxu2(u[2] & 0x7FFF7FFFu, u[3] & 0x7FFF7FFFu));
        m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 2));
        m = max(m & 0xFFFFu, m >> 16);
        float am = __uint_as_float(m << 16);
        if (__any_sync(0xffffffffu, m > 0x7F80u)) {
            am = 0.f;
#pragma unroll
            for (int e = 0; e < 8; e++) am = fmaxf(am, fabsf(f[e]));   // NaN passes over
            am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, 1));
            am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, 2));
        }
        const int k = min(mxq_exponent(am), kKv4MaxByte - 127);
        const float inv = mxq_inv_scale(k);
#pragma unroll
        for (int e = 0; e < 8; e++) f[e] = fminf(fmaf(f[e], inv, 0.0f), 6.0f);   // as the activation encoder: -0 is 0, NaN 6
        const uint32_t codes = e2m1x4(f[0], f[1], f[2], f[3]) | (e2m1x4(f[4], f[5], f[6], f[7]) << 16);
        if (p.has(a, i)) {
            *reinterpret_cast<uint32_t *>(a.c.c + p.code_at(i)) = codes;
            if (p.quarter == 0) a.c.c[p.scale_at(i)] = (uint8_t)(k + 127);
        }
    }
}

template <int D>
__global__ void __launch_bounds__(kWarps * 32) moe_kv4_read_kernel(const RowArgs a) {
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const Place<D> p(a);
    uint32_t w[kBlocks], s[kBlocks];
#pragma unroll
    for (int i = 0; i < kBlocks; i++) {
        w[i] = s[i] = 0;
        if (p.has(a, i)) w[i] = *reinterpret_cast<const uint32_t *>(a.c.c + p.code_at(i)), s[i] = a.c.c[p.scale_at(i)];
    }
    uint4 *row = reinterpret_cast<uint4 *>((p.values ? a.vo + p.tok * a.vs : a.ko + p.tok * a.ks) + p.h * D) + p.quarter;
#pragma unroll
    for (int i = 0; i < kBlocks; i++) {
        uint32_t h[4], o[4];
        e2m1x8_to_f16(w[i], h);
        const float f = kv4_scale(s[i]);
#pragma unroll
        for (int q = 0; q < 4; q++) {
            const float2 y = __half22float2(*reinterpret_cast<const __half2 *>(&h[q]));
            const __nv_bfloat162 r = __floats2bfloat162_rn(y.x * f, y.y * f);   // exact
            o[q] = *reinterpret_cast<const uint32_t *>(&r);
        }
        if (p.has(a, i)) row[4 * i] = make_uint4(o[0], o[1], o[2], o[3]);
    }
}

cudaError_t launch_rows(bool append, RowArgs a, cudaStream_t st) {
    a.shift = a.c.P == 16 ? 4 : a.c.P == 32 ? 5 : 6;
    const int parts = 2 * ((a.c.KVH * a.c.D + 127) / 128);
    const dim3 grid((a.n + 7) / 8, (parts + kWarps - 1) / kWarps), block(kWarps * 32);
    if (append) return a.c.D == 64 ? launch_pdl(moe_kv4_append_kernel<64>, grid, block, 0, st, a) : launch_pdl(moe_kv4_append_kernel<128>, grid, block, 0, st, a);
    return a.c.D == 64 ? launch_pdl(moe_kv4_read_kernel<64>, grid, block, 0, st, a) : launch_pdl(moe_kv4_read_kernel<128>, grid, block, 0, st, a);
}

bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }

}  // namespace

struct moe_kv4 {
    Kv4Cache c{};
    int QH = 0, window = 0;
    float scale = 0.f;
    const float *sinks = nullptr;
    unsigned char *ws = nullptr;
};

extern "C" {

moe_kv4 *moe_kv4_create(int q_heads, int kv_heads, int head_dim, int page_size, int n_pages) {
    if (kv_heads < 1 || kv_heads > 256 || q_heads < 1 || q_heads % kv_heads != 0 || q_heads / kv_heads > kKv8MaxGroup ||
        (head_dim != 64 && head_dim != 128) || (page_size != 16 && page_size != 32 && page_size != 64) || n_pages < 1 ||
        (long long)n_pages * page_size > INT_MAX) {
        moe_set_error("moe_kv4_create: bad arguments (1..256 kv heads, q_heads a multiple of kv_heads with at most %d "
                      "per kv head, head_dim 64 or 128, page_size 16, 32 or 64, n_pages * page_size at most 2^31 - 1)",
                      kKv8MaxGroup);
        return nullptr;
    }
    moe_kv4 *p = new (std::nothrow) moe_kv4;
    if (!p) {
        moe_set_error("moe_kv4_create: out of host memory");
        return nullptr;
    }
    p->c.KVH = kv_heads, p->c.D = head_dim, p->c.P = page_size, p->c.n_pages = n_pages;
    p->QH = q_heads;
    p->scale = 1.0f / std::sqrt((float)head_dim);
    return p;
}

void moe_kv4_destroy(moe_kv4 *p) { delete p; }

int moe_kv4_get_device_status(moe_kv4 *p, int *status, void *stream) {
    if (!p || !status) return moe_fail_status(MOE_EINVAL, "NULL argument");
    if (!p->ws) return moe_fail_status(MOE_ENOTREADY, "moe_kv4_set_workspace has not been called");
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    int32_t h[2] = {0, 0};
    cudaError_t e = cudaMemcpyAsync(h, p->ws, sizeof h, cudaMemcpyDeviceToHost, st);
    if (e == cudaSuccess) e = cudaStreamSynchronize(st);
    if (e == cudaSuccess && h[0]) {
        // a share that gave up may have left its tickets: all of them start over
        e = cudaMemsetAsync(p->ws, 0, kKv8ClearBytes, st);
        if (e == cudaSuccess) e = cudaStreamSynchronize(st);
    }
    if (e != cudaSuccess) return moe_fail_status(MOE_ECUDA, "moe_kv4_get_device_status: %s", cudaGetErrorString(e));
    *status = h[0];
    if (h[0]) return moe_fail_status(MOE_EDEVICE, "device status %d (detail %d)", h[0], h[1]);
    return MOE_OK;
}

int moe_kv4_set_i(moe_kv4 *p, const char *key, long long v) {
    if (!p || !key) return moe_fail_status(MOE_EINVAL, "NULL argument");
    if (strcmp(key, "sliding_window")) return moe_fail_status(MOE_EINVAL, "unknown integer option '%s'", key);
    if (v < 0 || v > INT_MAX) return moe_fail_status(MOE_EINVAL, "sliding_window must be 0..2^31 - 1");
    p->window = (int)v;
    return MOE_OK;
}

int moe_kv4_set_f(moe_kv4 *p, const char *key, double v) {
    if (!p || !key) return moe_fail_status(MOE_EINVAL, "NULL argument");
    if (strcmp(key, "softmax_scale")) return moe_fail_status(MOE_EINVAL, "unknown floating option '%s'", key);
    if (!(v > 1e-30 && v < 1e30)) return moe_fail_status(MOE_EINVAL, "softmax_scale must be positive (1e-30 .. 1e30)");
    p->scale = (float)v;
    return MOE_OK;
}

size_t moe_kv4_page_bytes(const moe_kv4 *p) { return p ? (size_t)p->c.KVH * kv4_page_bytes(p->c.P, p->c.D) : 0; }

int moe_kv4_set_cache(moe_kv4 *p, uint8_t *cache) {
    if (!p || !cache) return moe_fail_status(MOE_EINVAL, "NULL argument");
    if (!aligned16(cache)) return moe_fail_status(MOE_EINVAL, "the cache must be 16-byte aligned");
    p->c.c = cache;
    return MOE_OK;
}

int moe_kv4_set_sinks(moe_kv4 *p, const float *sinks) {
    if (!p) return moe_fail_status(MOE_EINVAL, "NULL plan");
    if ((uintptr_t)sinks & 3u) return moe_fail_status(MOE_EINVAL, "sinks must be 4-byte aligned");
    p->sinks = sinks;
    return MOE_OK;
}

size_t moe_kv4_workspace_bytes(const moe_kv4 *p) { return p ? kv4_workspace_bytes(p->c.D) : 0; }

int moe_kv4_set_workspace(moe_kv4 *p, void *dev, size_t bytes) {
    if (!p || !dev) return moe_fail_status(MOE_EINVAL, "NULL argument");
    if ((uintptr_t)dev & 255u) return moe_fail_status(MOE_EINVAL, "the workspace must be 256-byte aligned");
    const size_t need = kv4_workspace_bytes(p->c.D);
    if (bytes < need) return moe_fail_status(MOE_ENOMEM, "workspace of %zu bytes, %zu needed", bytes, need);
    // what is queued on any stream may still use the memory, and what is queued
    // next may be on a stream that does not wait for the one of the memset
    cudaError_t e = cudaDeviceSynchronize();
    if (e == cudaSuccess) e = cudaMemset(dev, 0, kKv8ClearBytes);
    if (e == cudaSuccess) e = cudaDeviceSynchronize();
    if (e != cudaSuccess) return moe_fail_status(MOE_ECUDA, "moe_kv4_set_workspace: %s", cudaGetErrorString(e));
    p->ws = static_cast<unsigned char *>(dev);
    return MOE_OK;
}

// What append and read refuse alike.
static int rows_check(moe_kv4 *p, const void *k, const void *v, long long k_stride, long long v_stride, const int32_t *slots) {
    if (!k || !v || !slots) return moe_fail_status(MOE_EINVAL, "NULL k, v or slots");
    if (!aligned16(k) || !aligned16(v) || ((uintptr_t)slots & 3u))
        return moe_fail_status(MOE_EINVAL, "k and v must be 16-byte aligned, slots 4-byte aligned");
    const long long row = (long long)p->c.KVH * p->c.D;
    if (k_stride < row || v_stride < row || k_stride % 8 || v_stride % 8)
        return moe_fail_status(MOE_EINVAL, "row strides must be multiples of 8 and at least %lld elements", row);
    return MOE_OK;
}

int moe_kv4_append(moe_kv4 *p, const uint16_t *k, const uint16_t *v, long long k_stride, long long v_stride,
                   const int32_t *slots, int n_tokens, void *stream) {
    if (!p) return moe_fail_status(MOE_EINVAL, "NULL plan");
    if (!p->c.c) return moe_fail_status(MOE_ENOTREADY, "moe_kv4_set_cache has not been called");
    if (n_tokens < 0 || n_tokens > (1 << 30)) return moe_fail_status(MOE_EINVAL, "n_tokens must be 0..2^30");
    if (n_tokens == 0) return MOE_OK;
    const int rc = rows_check(p, k, v, k_stride, v_stride, slots);
    if (rc) return rc;
    RowArgs a{};
    a.c = p->c, a.k = k, a.v = v, a.ks = k_stride, a.vs = v_stride, a.slots = slots, a.n = n_tokens;
    const cudaError_t e = launch_rows(true, a, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? MOE_OK : moe_fail_status(MOE_ECUDA, "moe_kv4_append: %s", cudaGetErrorString(e));
}

int moe_kv4_read(moe_kv4 *p, const int32_t *slots, int n_tokens, uint16_t *k, uint16_t *v, long long k_stride, long long v_stride,
                 void *stream) {
    if (!p) return moe_fail_status(MOE_EINVAL, "NULL plan");
    if (!p->c.c) return moe_fail_status(MOE_ENOTREADY, "moe_kv4_set_cache has not been called");
    if (n_tokens < 0 || n_tokens > (1 << 30)) return moe_fail_status(MOE_EINVAL, "n_tokens must be 0..2^30");
    if (n_tokens == 0) return MOE_OK;
    const int rc = rows_check(p, k, v, k_stride, v_stride, slots);
    if (rc) return rc;
    // their extents lie apart, or (rows of one array) their places in a row do
    const long long row = (long long)p->c.KVH * p->c.D;
    const uint16_t *ke = k + (long long)(n_tokens - 1) * k_stride + row, *ve = v + (long long)(n_tokens - 1) * v_stride + row;
    const long long apart = k_stride == v_stride ? (((long long)(v - k)) % k_stride + k_stride) % k_stride : 0;
    if (k < ve && v < ke && (apart < row || apart > k_stride - row)) return moe_fail_status(MOE_EINVAL, "k and v must not overlap");
    RowArgs a{};
    a.c = p->c, a.ko = k, a.vo = v, a.ks = k_stride, a.vs = v_stride, a.slots = slots, a.n = n_tokens;
    const cudaError_t e = launch_rows(false, a, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? MOE_OK : moe_fail_status(MOE_ECUDA, "moe_kv4_read: %s", cudaGetErrorString(e));
}

int moe_kv4_attend(moe_kv4 *p, const uint16_t *q, long long q_stride, const int32_t *starts, const int32_t *lens,
                   const int32_t *table, int table_width, int n_seqs, int max_new, int n_rows, uint16_t *out,
                   long long out_stride, void *stream) {
    if (!p) return moe_fail_status(MOE_EINVAL, "NULL plan");
    if (!p->c.c) return moe_fail_status(MOE_ENOTREADY, "moe_kv4_set_cache has not been called");
    if (!p->ws) return moe_fail_status(MOE_ENOTREADY, "moe_kv4_set_workspace has not been called");
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
    Kv4Attend a{};
    a.c = p->c;
    a.QH = p->QH, a.window = p->window, a.n_seqs = n_seqs, a.n_rows = n_rows, a.max_new = max_new, a.width = table_width;
    a.scale = p->scale, a.sinks = p->sinks, a.q = q, a.out = out, a.q_stride = q_stride, a.o_stride = out_stride;
    a.starts = starts, a.lens = lens, a.table = table;
    const cudaError_t e = launch_kv4_attend(a, p->ws, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? MOE_OK : moe_fail_status(MOE_ECUDA, "moe_kv4_attend: %s", cudaGetErrorString(e));
}

}  // extern "C"
