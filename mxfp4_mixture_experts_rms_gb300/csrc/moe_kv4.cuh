// moe_kv4.cuh -- what the kernels of the 4-bit paged key/value cache share: the
// cache's layout, the conversions and the plan.
#pragma once
#include "moe_kv8.cuh"   // lengths, windows

// One layer's cache (device memory, borrowed), MXFP4: E2M1 codes and an E8M0
// scale for each token, kv head, side and block of 32 dims.  Per page of P
// tokens and kv head, side by side: key codes [D / 32][P][16], so that the 16
// bytes of a token's block are a row of an 8 x 16-byte matrix fragment and the
// tokens after it the next rows; value codes likewise; key scales [D / 32][P];
// value scales.  All of it is one copy of P * D * 17 / 16 bytes.  Of 16 tokens'
// scales, token 2 t + e (t < 4, e < 2) is byte 4 t + e and token 8 + 2 t + e
// byte 4 t + 2 + e: the word at 4 t is that of the tokens whose scores one
// thread of an m16n8 tile pair holds.
struct Kv4Cache {
    uint8_t *c;   // [n_pages][KVH][kv4_page_bytes(P, D)]
    int n_pages, KVH, P, D;
};
__host__ __device__ constexpr int kv4_page_bytes(int P, int D) { return P * D / 16 * 17; }
__host__ __device__ constexpr int kv4_scale_byte(int tok) {  // of 16
    return 4 * ((tok & 7) >> 1) + ((tok >> 3) << 1) + (tok & 1);
}

// Scales are at most 2^125, so that every value is finite (6 * 2^125): what a
// row does not see can meet a weight of 0, whatever the cache holds there.
constexpr int kKv4MaxByte = 252;
// A scale byte as a float; 0 counts as 0 (an append writes at least 1).
__device__ __forceinline__ float kv4_scale(uint32_t byte) { return __uint_as_float(min(byte, (uint32_t)kKv4MaxByte) << 23); }

struct Kv4Attend {
    Kv4Cache c;
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

cudaError_t launch_kv4_attend(const Kv4Attend &a, unsigned char *ws, cudaStream_t st);
cudaError_t launch_kv4_prompt(const Kv4Attend &a, int32_t *status, cudaStream_t st);
size_t kv4_workspace_bytes(int head_dim);
