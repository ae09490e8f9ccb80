// moe_kv8.cuh -- what the kernels of the 8-bit paged key/value cache share:
// the cache's layout, the E4M3 conversions and the plan.
#pragma once
#include "moe_common.cuh"

// One layer's cache (device memory, borrowed).  Per page of P tokens and kv
// head, P * D codes: keys as [D / 16][P][16], so that 16 consecutive dims of a
// token and of the tokens after it form the 16-byte rows of an 8 x 16 matrix
// fragment; values as [P / 16][D][16], so that 16 consecutive tokens of a dim
// do.  Inside a value's 16 bytes, token 2 t + e (t < 4, e < 2) is byte
// 4 t + e and token 8 + 2 t + e byte 4 t + 2 + e: the four bytes at 4 t are
// then the four tokens whose probabilities one thread of an m16n8 score tile
// pair holds.
struct Kv8Cache {
    uint8_t *k, *v;    // [n_pages][KVH][P * D]
    uint8_t *ks, *vs;  // E8M0 [n_pages][KVH]
    int n_pages, KVH, P, D;
};

__host__ __device__ __forceinline__ int kv8_value_byte(int tok) {  // of 16
    return 4 * ((tok & 7) >> 1) + ((tok >> 3) << 1) + (tok & 1);
}

// Two E4M3 codes (low 16 bits) -> fp16 pair, exact.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t w) {
    uint32_t r;
    asm("{ .reg .b16 l, h; mov.b32 {l, h}, %1; cvt.rn.f16x2.e4m3x2 %0, l; }" : "=r"(r) : "r"(w));
    return r;
}
// Four codes -> two fp16 pairs.
__device__ __forceinline__ void e4m3x4_to_f16(uint32_t w, uint32_t &lo, uint32_t &hi) {
    asm("{ .reg .b16 l, h; mov.b32 {l, h}, %2; cvt.rn.f16x2.e4m3x2 %0, l; cvt.rn.f16x2.e4m3x2 %1, h; }"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}
__device__ __forceinline__ float2 e4m3x2_to_f32(uint32_t w) {
    const uint32_t h = e4m3x2_to_f16x2(w);
    return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}
// Two floats -> two codes (x in the low byte): nearest, ties to even, beyond
// +-448 (infinities too) +-448, NaN the NaN code.
__device__ __forceinline__ uint32_t f32x2_to_e4m3(float x, float y) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %2, %1;" : "=h"(r) : "f"(x), "f"(y));
    return r;
}
// 2^e for e in [-149, 127], 0 below.
__device__ __forceinline__ float pow2i(int e) {
    return e >= -126 ? __uint_as_float((uint32_t)(min(e, 127) + 127) << 23)
                     : (e >= -149 ? __uint_as_float(1u << (e + 149)) : 0.f);
}

constexpr size_t kKv8ClearBytes = 8192;  // head of the workspace: status word and detail, tickets (zero between calls)
constexpr int kKv8MaxSeqs = 4096;
constexpr int kKv8MaxGroup = 16;  // query heads of one kv head

struct Kv8Attend {
    Kv8Cache c;
    int QH, window, n_seqs, n_rows, max_new, width;
    float scale;          // of the scores
    const float *sinks;   // [QH] or null
    const uint16_t *q;    // rows of q_stride elements
    uint16_t *out;
    long long q_stride, o_stride;
    const int32_t *starts;  // [n_seqs + 1] or null: one row a sequence
    const int32_t *lens;    // [n_seqs]
    const int32_t *table;   // [n_seqs][width]
};

// The rows of sequence b: first row, rows that are computed, and the position
// of the first (lens - the sequence's rows from it on, past n_rows too;
// negative: those see nothing).  Whatever starts holds, the rows stay inside
// 0 .. n_rows - 1.
__device__ __forceinline__ void kv8_rows(const Kv8Attend &a, int b, int &row0, int &n, int &pos0) {
    const int len = max(a.lens[b], 0);
    if (!a.starts) {
        row0 = b, n = 1, pos0 = len - 1;
        return;
    }
    row0 = min(max(a.starts[b], 0), a.n_rows);
    const int e = max(a.starts[b + 1], row0);
    n = min(min(e, a.n_rows) - row0, a.max_new);
    pos0 = len - (e - row0);
}

// The first token that a row at position pos sees (one below 0 sees none).
__device__ __forceinline__ int kv8_first(int pos, int window) { return window > 0 ? max(0, max(pos, 0) - window + 1) : 0; }

cudaError_t launch_kv8_append(const Kv8Cache &c, const uint16_t *k, const uint16_t *v, long long k_stride,
                              long long v_stride, const int32_t *slots, int n, cudaStream_t st);
cudaError_t launch_kv8_attend(const Kv8Attend &a, unsigned char *ws, cudaStream_t st);
cudaError_t launch_kv8_prompt(const Kv8Attend &a, int32_t *status, cudaStream_t st);
size_t kv8_workspace_bytes(int head_dim);
