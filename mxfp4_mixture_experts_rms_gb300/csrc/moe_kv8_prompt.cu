// moe_kv8_prompt.cu -- attention over the 8-bit paged cache for many new
// tokens a sequence (prompts, or pieces of them): tensor-core products on
// tcgen05 with accumulators in tensor memory.
//
// One CTA per (sequence, kv head, 256 rows), a row being a new token and one of
// the kv head's query heads; 64 cached tokens a step.  Its warps:
//  * 0..3 and 4..7 are the halves' softmax, a thread a row: scores by
//    tcgen05.ld, no shuffles, weights as fp16 into the half's P tile;
//  * 8..11 turn E4M3 codes into fp16 (exact) and write them as the K-major,
//    128-byte-swizzled operand tiles K [64 tokens][D] and V^T [D][64 tokens];
//  * 12 has the pages copied into shared memory steps ahead (bulk copies);
//  * 13 and 14 (one lane each) issue a half's products, S = Q K^T (M 128, N 64)
//    into one of two score buffers one step ahead, and O += P V (N = D), fp32
//    in tensor memory.
// Softmax references as in the kernel for a few tokens (m of the scores, m + N
// of score + value exponent e), but moved only when a score passes one by more
// than 2^8, so that the accumulator in tensor memory is rarely rescaled:
// weights are w = 2^(7 + s - m + e - N) <= 2^15, and a page's share of the sum
// l is its weights' sum times 2^(N - e - 7).  There e - N is taken as at least
// -80: a page that small adds nothing to the values, but its weights count.
// Bound by the softmax warps' chains: a step takes them about 2050 cycles (wait
// for the scores 400, read 200, maxima 250, wait for the products 250, weights
// 750, hand over 150), the tensor cores about 540 of them and the exponentials
// 512.  2430 new tokens of 3 sequences over 6416 cached, 64 / 8 heads of 64: 159 us
// (205 with one issuing warp for both halves and page copies by a decoder;
// 193 with 16 softmax warps of 32 scores a thread, whose fixed work a step is
// the same for half the scores; 170 before a tile's heads came together).
//
// A NaN value that only some of a tile's rows see would reach the others as
// 0 * NaN: where the pages hold one in a step that not all rows see, the CTA's
// rows are computed once more, one at a time.
#include "moe_kv_prompt.cuh"

#include <algorithm>

namespace {

template <int D>
struct Smem {   // offsets from a 1024-byte boundary
    static constexpr int kStages = D == 64 ? 3 : 2, kRaw = D == 64 ? 4 : 3;   // operand tiles; steps of copied pages
    static constexpr int kQ = 0;
    static constexpr int kQ1 = kM * D * 2;                  // of a half: Q [128][D], P [128][64]
    static constexpr int kP = 2 * kQ1, kP1 = kM * kT * 2;
    static constexpr int kK = kP + 2 * kP1;                 // kStages x [64][D]
    static constexpr int kV = kK + kStages * kT * D * 2;    // kStages x [D][64]
    static constexpr int kCodes = kV + kStages * kT * D * 2; // kRaw x keys, values as they lie in the pages
    static constexpr int kBytes = kCodes + kRaw * kT * D * 2;
};

struct PromptArgs {
    Kv8Attend a;
    int G;
    int32_t *status;
};

// Sixteen codes -> two 16-byte chunks of fp16.  keys: in order; values: the
// bytes of word t are tokens 2 t, 2 t + 1, 8 + 2 t, 9 + 2 t.
__device__ __forceinline__ void decode16(uint4 w, bool keys, uint4 &c0, uint4 &c1) {
    uint32_t l[4], h[4];
    e4m3x4_to_f16(w.x, l[0], h[0]);
    e4m3x4_to_f16(w.y, l[1], h[1]);
    e4m3x4_to_f16(w.z, l[2], h[2]);
    e4m3x4_to_f16(w.w, l[3], h[3]);
    if (keys) c0 = make_uint4(l[0], h[0], l[1], h[1]), c1 = make_uint4(l[2], h[2], l[3], h[3]);
    else c0 = make_uint4(l[0], l[1], l[2], l[3]), c1 = make_uint4(h[0], h[1], h[2], h[3]);
}

// One row (position pos) of query head `head` by 128 threads, keys 128 at a
// time: what the tiles cannot do (see the top).  scratch: D + 384 floats, 128
// pointers.
template <int D>
__device__ void slow_row(const Kv8Attend &a, int b, int kvh, int head, int row, int pos, int tid, float *scratch) {
    const int P = a.c.P;
    float *qs = scratch, *p = qs + D, *vsc = p + 128, *red = vsc + 128;
    const uint8_t **vat = reinterpret_cast<const uint8_t **>(red + 128);
    auto sync = [] { asm volatile("bar.sync 1, 128;" ::: "memory"); };
    const int last = (int)min((long long)pos, (long long)a.width * P - 1), first = kv8_first(pos, a.window);
    const uint16_t *q = a.q + (long long)row * a.q_stride + head * D;
    sync();
    for (int d = tid; d < D; d += 128) qs[d] = bf16_to_f32(q[d]) * a.scale;
    sync();
    float m = -INFINITY, l = 0.f, acc = 0.f;
    const int dim = tid % D, part = tid / D, parts = 128 / D;
    for (int k0 = first; k0 <= last; k0 += 128) {
        const int t = k0 + tid;
        float s = -INFINITY;
        vat[tid] = nullptr;
        if (t <= last) {
            const int page = a.table[(size_t)b * a.width + t / P], off = t % P;
            if (page >= 0 && page < a.c.n_pages) {
                const size_t ph = (size_t)page * a.c.KVH + kvh;
                const uint8_t *kp = a.c.k + ph * (P * D) + off * 16;
                float dot = 0.f;
                for (int c = 0; c < D; c += 2) {
                    const float2 x = e4m3x2_to_f32(*reinterpret_cast<const uint16_t *>(kp + (size_t)(c / 16) * P * 16 + c % 16));
                    dot += x.x * qs[c] + x.y * qs[c + 1];
                }
                s = dot * pow2i(a.c.ks[ph] - 127);
                vat[tid] = a.c.v + ph * (P * D) + (size_t)(off / 16) * D * 16 + kv8_value_byte(off % 16);
                vsc[tid] = pow2i(a.c.vs[ph] - 127);
            }
        }
        red[tid] = s;
        sync();
        float mn = m;
        for (int j = 0; j < 128; j++) mn = fmaxf(mn, red[j]);
        const float f = mn == -INFINITY ? 1.f : expf(m - mn);
        p[tid] = vat[tid] ? expf(s - (mn == -INFINITY ? 0.f : mn)) : 0.f;
        sync();
        acc *= f, l *= f, m = mn;
        for (int j = part; j < 128; j += parts)
            if (vat[j]) acc += p[j] * (vsc[j] * e4m3x2_to_f32(vat[j][dim * 16]).x);
        for (int j = 0; j < 128; j++) l += p[j];
        sync();
    }
    if (parts == 2) {
        p[tid] = acc;
        sync();
        acc += p[(tid + D) % 128];
    }
    if (a.sinks) {
        const float mn = fmaxf(m, a.sinks[head]), f = mn == -INFINITY ? 0.f : expf(m - mn);
        acc *= f, l = l * f + (mn == -INFINITY ? 0.f : expf(a.sinks[head] - mn));
    }
    if (part == 0) {
        const __nv_bfloat16 r = __float2bfloat16_rn(l == 0.f ? 0.f : acc / l);
        a.out[(long long)row * a.o_stride + head * D + dim] = *reinterpret_cast<const uint16_t *>(&r);
    }
}

template <int D, int P>
__global__ void __launch_bounds__(kThreads, 1) moe_kv8_prompt_kernel(const __grid_constant__ PromptArgs f) {
    constexpr int NP = kT / P, NU = kT * (D / 16), KU = NU / kLoaders;   // pages; 16-byte units of keys (and of values): all, a thread's
    typedef Smem<D> L;
    constexpr int kStages = L::kStages, kRaw = L::kRaw;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *smem = reinterpret_cast<unsigned char *>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    __shared__ __align__(8) uint64_t raw[kRaw], raw_empty[kRaw], full[kStages], empty[kStages], s_full[2][2], q_full[2], p_full[2], o_done[2], drain[2];
    __shared__ uint32_t rmeta[kRaw][NP], meta[kStages][NP];   // key exponent byte, value's, 1 if the page is there
    __shared__ uint32_t tmem_slot;
    __shared__ int job[2], odd;
    const Kv8Attend &a = f.a;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, kvh = blockIdx.x % a.c.KVH;
    if (tid == 0) {
        for (int s = 0; s < kStages; s++) bar_init(&full[s], kLoaders / 32), bar_init(&empty[s], 2);
        for (int s = 0; s < kRaw; s++) bar_init(&raw[s], 2), bar_init(&raw_empty[s], kLoaders / 32);
        for (int h = 0; h < 2; h++)
            bar_init(&s_full[h][0], 1), bar_init(&s_full[h][1], 1), bar_init(&q_full[h], kSoftmax / 2), bar_init(&p_full[h], kSoftmax / 2), bar_init(&o_done[h], 1), bar_init(&drain[h], 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        odd = 0;
    }
    if (warp == kIssuer) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&tmem_slot)));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (warp == 0) {
        // a tile of 256 rows: sequences in order, a sequence's last (longest)
        // tile first, its heads together, so that the last to start are short
        int x = blockIdx.x / a.c.KVH, found = -1, rt = 0;
        for (int b0 = 0; b0 < a.n_seqs && found < 0; b0 += 32) {
            int row0, n = 0, pos0;
            if (b0 + lane < a.n_seqs) kv8_rows(a, b0 + lane, row0, n, pos0);
            const int mine = (n * f.G + 2 * kM - 1) / (2 * kM);
            int inc = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += y;
            }
            const unsigned hit = __ballot_sync(0xffffffffu, x < inc);
            if (hit) {
                const int at = __ffs(hit) - 1;
                found = b0 + at;
                rt = __shfl_sync(0xffffffffu, inc, at) - 1 - x;
            } else {
                x -= __shfl_sync(0xffffffffu, inc, 31);
            }
        }
        if (lane == 0) job[0] = found, job[1] = rt;
    }
    fence_before();
    __syncthreads();
    fence_after();
    // only now: a dependent's CTA that got tensor memory first would wait for
    // this grid, and this grid for it
    asm volatile("griddepcontrol.launch_dependents;");
    const uint32_t tmem = tmem_slot;
    const int b = job[0];
    if (b >= 0) {
        int row0, n, pos0;
        kv8_rows(a, b, row0, n, pos0);
        const int r0 = job[1] * 2 * kM, rows = min(2 * kM, n * f.G - r0), halves = rows > kM ? 2 : 1;
        const int p_first = pos0 + r0 / f.G, p_last = pos0 + (r0 + rows - 1) / f.G;
        // tokens that any row sees, and the steps over them (aligned to 64)
        const int seen = (int)max(0ll, min((long long)p_last + 1, (long long)a.width * P));
        const int lo = kv8_first(p_first, a.window);
        const int step0 = lo / kT, steps = max(1, (seen + kT - 1) / kT - step0);
        int32_t *status = f.status;

        if (warp < kSoftmax) {
            // ---- the softmax ----
            const int h = warp >> 2;
            if (h < halves) {
                const int r = tid & (kM - 1), rr = r0 + h * kM + r, i2 = rr / f.G, head = kvh * f.G + rr - i2 * f.G;
                const bool on = h * kM + r < rows;
                // tokens from .. to that the row sees, and all_from .. all_to that all rows of the half see (where their pages are)
                const int to = on ? min(seen - 1, pos0 + i2) : -1, from = kv8_first(pos0 + i2, a.window);
                const int all_to = min(seen - 1, pos0 + (r0 + h * kM) / f.G);
                const int all_from = kv8_first(pos0 + (r0 + min(rows, (h + 1) * kM) - 1) / f.G, a.window);
                int up;
                {
                    // the row's queries, scaled by a power of two: largest magnitude in [2^14, 2^15)
                    const uint4 *q = reinterpret_cast<const uint4 *>(a.q + (long long)(row0 + i2) * a.q_stride + head * D);
                    uint32_t am = 0;
#pragma unroll 8
                    for (int c = 0; c < D / 8; c++) {
                        const uint4 w = on ? __ldg(q + c) : make_uint4(0, 0, 0, 0);
                        const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                        for (int e = 0; e < 4; e++) am = max(am, max(x[e] & 0x7FFFu, (x[e] >> 16) & 0x7FFFu));
                    }
                    up = min(141 - (int)(am >> 7), 127);
                    const float mul = pow2i(up);
#pragma unroll 8
                    for (int c = 0; c < D / 8; c++) {
                        const uint4 w = on ? __ldg(q + c) : make_uint4(0, 0, 0, 0);
                        const uint32_t x[4] = {w.x, w.y, w.z, w.w};
                        uint32_t y[4];
#pragma unroll
                        for (int e = 0; e < 4; e++) y[e] = pack_f16(__uint_as_float(x[e] << 16) * mul, __uint_as_float(x[e] & 0xFFFF0000u) * mul);
                        *reinterpret_cast<uint4 *>(smem + L::kQ + h * L::kQ1 + (c / 8) * (kM * 128) + swizzled(r, c % 8)) = make_uint4(y[0], y[1], y[2], y[3]);
                    }
                    fence_async();
                    bar_arrive_warp(&q_full[h]);
                }
                const float sc = a.scale * kLog2e;
                float m = -INFINITY, N = -INFINITY, l = 0.f;
                const uint32_t lanes = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + 256 * h;
                unsigned char *pt = smem + L::kP + h * L::kP1;
                bool ok = true;
                for (int j = 0; j < steps; j++) {
                    const int st = j % kStages, t0 = (step0 + j) * kT;
                    // (a wait that gave up is only found out below: what it waited for is then read as it is)
                    ok = bar_wait(&s_full[h][j & 1], (uint32_t)(j >> 1) & 1, status, 100);
                    __syncwarp();
                    fence_after();
                    float s[kT];
                    tmem_ld32(lanes + (j & 1) * kT, s);
                    tmem_ld32(lanes + (j & 1) * kT + 32, s + 32);
                    uint32_t mt[NP];
                    bool all = t0 >= all_from && t0 + kT - 1 <= all_to;
#pragma unroll
                    for (int p = 0; p < NP; p++) mt[p] = meta[st][p], all = all && (mt[p] >> 16);
                    tmem_wait(s);
                    tmem_wait(s + 32);
                    if (!all) {
#pragma unroll
                        for (int c = 0; c < kT; c++) {
                            const int t = t0 + c;
                            if (!(t >= from && t <= to && (mt[c / P] >> 16))) s[c] = -INFINITY;
                        }
                    }
                    auto key_scale = [&](int p) { return fmaxf(pow2i((int)(mt[p] & 255u) - 127 - up) * sc, 1e-37f); };   // > 0: -inf stays
                    auto value_exp = [&](int p) { return (float)((int)((mt[p] >> 8) & 255u) - 127); };
                    float mx = -INFINITY, mv = -INFINITY, pm[NP];   // mv: over m
#pragma unroll
                    for (int p = 0; p < NP; p++) {
                        float x[4];   // four chains
#pragma unroll
                        for (int c = 0; c < 4; c++) x[c] = max3(s[p * P + c], s[p * P + 4 + c], s[p * P + 8 + c]);
#pragma unroll
                        for (int c = 12; c < P; c++) {
                            if (c + 4 < P && (c / 4) % 2 == 1) x[c % 4] = max3(x[c % 4], s[p * P + c], s[p * P + c + 4]);
                            else if (c + 4 >= P && (c / 4) % 2 == 1) x[c % 4] = fmaxf(x[c % 4], s[p * P + c]);
                        }
                        pm[p] = fmaxf(max3(x[0], x[1], x[2]), x[3]) * key_scale(p);
                        mx = fmaxf(mx, pm[p]), mv = fmaxf(mv, pm[p] - m + value_exp(p));   // (-inf - -inf passes over)
                    }
                    // the references follow when passed by more than 2^8
                    float corr = 1.f;
                    const bool move = mx > m + 8.f || mv > N + 8.f;
                    if (move) {
                        const float mn = fmaxf(m, mx), was = N + (m - mn);
                        float nn = was;
#pragma unroll
                        for (int p = 0; p < NP; p++) nn = fmaxf(nn, pm[p] - mn + value_exp(p));
                        l *= ex2(m - mn);
                        corr = ex2(was - nn);
                        m = mn, N = nn;
                    }
                    const float ms = m == -INFINITY ? 0.f : m, Ns = N == -INFINITY ? 0.f : N;
                    // large scores: differences first, each product rounded as the maximum was
                    const bool large = __any_sync(0xffffffffu, fabsf(ms) >= 0x1p17f);
                    if (large) {
#pragma unroll
                        for (int c = 0; c < kT; c++) s[c] = __fsub_rn(__fmul_rn(s[c], key_scale(c / P)), ms);
                    }
                    // the products of the step before have read the P tile
                    if (j > 0) ok = bar_wait(&o_done[h], (uint32_t)(j - 1) & 1, status, 101) && ok;
                    if (__any_sync(0xffffffffu, move || !ok)) {
                        ok = __all_sync(0xffffffffu, ok);
                        if (!ok) break;
                        fence_after();
                        if (j > 0) {
#pragma unroll 1
                            for (int c = 0; c < D; c += 16) tmem_scale16(lanes + 2 * kT + c, corr);
                        }
                    }
#pragma unroll
                    for (int p = 0; p < NP; p++) {
                        const float fe = fmaxf(value_exp(p) - Ns, -80.f) + 7.f, bias = large ? fe : fe - ms, ks = large ? 1.f : key_scale(p);
                        float s0 = 0.f, s1 = 0.f;
#pragma unroll
                        for (int c = p * P; c < (p + 1) * P; c += 8) {
                            uint32_t y[4];
#pragma unroll
                            for (int e = 0; e < 4; e++) {
                                float w0, w1;
                                fma2(w0, w1, s[c + 2 * e], s[c + 2 * e + 1], ks, bias);
                                w0 = ex2(w0), w1 = ex2(w1);
                                add2(s0, s1, w0, w1);
                                y[e] = pack_f16(w0, w1);
                            }
                            *reinterpret_cast<uint4 *>(pt + swizzled(r, c / 8)) = make_uint4(y[0], y[1], y[2], y[3]);
                        }
                        l = fmaf(s0 + s1, ex2(-fe), l);
                    }
                    fence_async();
                    fence_before();
                    bar_arrive_warp(&p_full[h]);
                }
                if (ok) ok = bar_wait_warp(&o_done[h], (uint32_t)(steps - 1) & 1, status, 102);
                if (ok) {
                    fence_after();
                    const float sink = on && a.sinks ? a.sinks[head] * kLog2e : -INFINITY;
                    const float top = fmaxf(m, sink);
                    const float den = top == -INFINITY ? l : (m == -INFINITY ? l : l * ex2(m - top)) + ex2(sink - top);
                    // two factors: their product may be below 2^-126 where the output is not
                    const float k1 = den == 0.f || N == -INFINITY ? 0.f : ex2(0.5f * (N - 7.f + (m - top))), k2 = k1 == 0.f ? 0.f : k1 / den;
                    uint4 *o = reinterpret_cast<uint4 *>(a.out + (long long)(row0 + i2) * a.o_stride + head * D);
#pragma unroll 1
                    for (int c = 0; c < D; c += 32) {
                        float v[32];
                        tmem_ld32(lanes + 2 * kT + c, v);
                        tmem_wait(v);
                        if (!on) continue;
#pragma unroll
                        for (int x = 0; x < 32; x++) v[x] = v[x] * k1 * k2;
#pragma unroll
                        for (int x = 0; x < 4; x++)
                            o[c / 8 + x] = make_uint4(bits_of(__floats2bfloat162_rn(v[8 * x], v[8 * x + 1])),
                                                      bits_of(__floats2bfloat162_rn(v[8 * x + 2], v[8 * x + 3])),
                                                      bits_of(__floats2bfloat162_rn(v[8 * x + 4], v[8 * x + 5])),
                                                      bits_of(__floats2bfloat162_rn(v[8 * x + 6], v[8 * x + 7])));
                    }
                }
            }
        } else if (warp < kCopier) {
            // ---- pages to operand tiles ----
            const int x = tid - kSoftmax * 32;
            bool ok = true;
            for (int j = 0; j < steps; j++) {
                const int st = j % kStages, slot = j % kRaw, t0 = (step0 + j) * kT;
                ok = bar_wait_warp(&raw[slot], (uint32_t)(j / kRaw) & 1, status, 108);
                if (!ok) break;
                if (j >= kStages) {
                    ok = bar_wait_warp(&empty[st], (uint32_t)(j / kStages - 1) & 1, status, 103);
                    if (!ok) break;
                }
                const uint32_t mw = x < NP ? rmeta[slot][x] : 0u;
                uint32_t there = 0;   // pages of the step that are there
#pragma unroll
                for (int p = 0; p < NP; p++) there |= (rmeta[slot][p] >> 16) << p;
                const bool part = t0 + kT > seen || t0 + kT - 1 > p_first || (a.window && t0 <= p_last - a.window) || there != (1u << NP) - 1;
                // unit u: keys of token u % 64, dims 16 (u / 64) ..; values of dim u % D, tokens 16 (u / D) ..; what no
                // page brought is what the slot held before, and never seen
                const unsigned char *codes = smem + L::kCodes + slot * (2 * kT * D);
                unsigned char *K = smem + L::kK + st * (kT * D * 2), *V = smem + L::kV + st * (kT * D * 2);
#pragma unroll 2
                for (int i = 0; i < KU; i++) {
                    const int u = x + kLoaders * i, tok = u % kT, ch = 2 * (u / kT);   // 16-byte chunk of the row: dims 8 ch ..
                    const uint4 w = *reinterpret_cast<const uint4 *>(codes + (tok / P) * (P * D) + (u / kT) * (P * 16) + (tok % P) * 16);
                    uint4 c0, c1;
                    decode16(w, true, c0, c1);
                    unsigned char *to = K + (ch / 8) * (kT * 128);
                    *reinterpret_cast<uint4 *>(to + swizzled(tok, ch % 8)) = c0;
                    *reinterpret_cast<uint4 *>(to + swizzled(tok, ch % 8 + 1)) = c1;
                }
#pragma unroll 2
                for (int i = 0; i < KU; i++) {
                    const int u = x + kLoaders * i, dim = u % D, blk = u / D;
                    uint4 v = *reinterpret_cast<const uint4 *>(codes + kT * D + u * 16);
                    if (part) {
                        // tokens that no row sees to zero; a NaN among the others: not all rows see it
                        uint32_t w[4] = {v.x, v.y, v.z, v.w}, nan = 0;
#pragma unroll
                        for (int q = 0; q < 4; q++) {
#pragma unroll
                            for (int e = 0; e < 4; e++) {
                                const int t = t0 + 16 * blk + 2 * q + (e & 1) + 8 * (e >> 1);
                                if (t >= seen || t < lo || !(there >> (16 * blk / P) & 1)) w[q] &= ~(0xFFu << (8 * e));
                            }
                            nan |= ((w[q] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
                        }
                        if (nan) odd = 1;
                        v = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                    uint4 c0, c1;
                    decode16(v, false, c0, c1);
                    *reinterpret_cast<uint4 *>(V + swizzled(dim, 2 * blk)) = c0;
                    *reinterpret_cast<uint4 *>(V + swizzled(dim, 2 * blk + 1)) = c1;
                }
                bar_arrive_warp(&raw_empty[slot]);
                if (x < NP) meta[st][x] = mw;
                fence_async();
                bar_arrive_warp(&full[st]);
            }
        } else if (warp == kCopier) {
            // ---- pages into shared memory: lane p page p of a step ----
            const int32_t *tab = a.table + (size_t)b * a.width;
            auto page_of = [&](int j) {   // -1 where there is none
                const int t = (step0 + j) * kT + lane * P;
                const int pg = lane < NP && j < steps && t < seen ? __ldg(tab + t / P) : -1;
                return pg >= 0 && pg < a.c.n_pages ? pg : -1;
            };
            int pg = page_of(0), issued = 0;
            for (; issued < steps; issued++) {
                const int slot = issued % kRaw;
                if (issued >= kRaw && !bar_wait_warp(&raw_empty[slot], (uint32_t)(issued / kRaw - 1) & 1, status, 110)) break;
                const unsigned there = __ballot_sync(0xffffffffu, pg >= 0);
                if (lane == 0)
                    asm volatile("{ .reg .b64 st; mbarrier.arrive.expect_tx.shared::cta.b64 st, [%0], %1; }" ::"r"(smem_u32(&raw[slot])),
                                 "r"((uint32_t)(__popc(there) * 2 * P * D)) : "memory");
                __syncwarp();
                uint32_t scales = 0;
                if (pg >= 0) {
                    const size_t ph = (size_t)pg * a.c.KVH + kvh;
                    const uint32_t dst = smem_u32(smem + L::kCodes + slot * (2 * kT * D)) + lane * (P * D), bar = smem_u32(&raw[slot]);
                    bulk_copy(dst, a.c.k + ph * (P * D), P * D, bar);
                    bulk_copy(dst + kT * D, a.c.v + ph * (P * D), P * D, bar);
                    scales = (uint32_t)__ldg(a.c.ks + ph) | (uint32_t)__ldg(a.c.vs + ph) << 8 | 1u << 16;
                }
                pg = page_of(issued + 1);
                if (lane < NP) rmeta[slot][lane] = scales;
                bar_arrive_warp(&raw[slot]);   // the slot's second arrival
            }
            // copies still in flight land before the shared memory goes
            for (int j = max(0, issued - kRaw); j < issued; j++) bar_wait_warp(&raw[j % kRaw], (uint32_t)(j / kRaw) & 1, status, 109, true);
        } else {
            // ---- a half's products: the warp together, so that descriptors stay in uniform registers; one lane issues ----
            const int h = warp - kIssuer;
            const uint64_t Q = tile_desc(smem_u32(smem + L::kQ + h * L::kQ1)), Pt = tile_desc(smem_u32(smem + L::kP + h * L::kP1));
            const uint64_t K0 = tile_desc(smem_u32(smem + L::kK)), V0 = tile_desc(smem_u32(smem + L::kV));
            const uint32_t S = tmem + 256 * h, O = S + 2 * kT;
            constexpr uint64_t kTile16 = kT * D * 2 / 16;   // descriptors count 16 bytes
            auto scores = [&](int j, int st, uint32_t parity) {   // into score buffer j & 1
                if (!bar_wait_warp(&full[st], parity, status, 105)) return false;
                fence_after();
                const uint64_t K = K0 + st * kTile16;
                const uint32_t to = S + (j & 1) * kT;
                if (elect_one()) {
#pragma unroll
                    for (int c = 0; c < D / 16; c++) {
                        const uint64_t q = Q + (c / 4) * (kM * 8) + (c % 4) * 2, k = K + (c / 4) * (kT * 8) + (c % 4) * 2;
                        if (c == 0) mma<false>(to, q, k, inst_desc(kT));
                        else mma<true>(to, q, k, inst_desc(kT));
                    }
                    commit(&s_full[h][j & 1]);
                }
                __syncwarp();
                return true;
            };
            int st = 0, st1 = 0;          // stages of steps j and j + 1
            uint32_t par1 = 0;
            bool ok = h < halves && bar_wait_warp(&q_full[h], 0, status, 104);
            if (ok) ok = scores(0, 0, 0);
            for (int j = 0; j < steps && ok; j++, st = st1) {
                if (++st1 == kStages) st1 = 0, par1 ^= 1;
                // the next scores go ahead of this step's values: their buffer was read before step j - 1's weights were
                if (j + 1 < steps) ok = scores(j + 1, st1, par1);
                if (ok) ok = bar_wait_warp(&p_full[h], (uint32_t)j & 1, status, 106);
                if (!ok) break;
                fence_after();
                const uint64_t V = V0 + st * kTile16;
                if (elect_one()) {
                    if (j == 0) mma<false>(O, Pt, V, inst_desc(D));
                    else mma<true>(O, Pt, V, inst_desc(D));
#pragma unroll
                    for (int c = 1; c < kT / 16; c++) mma<true>(O, Pt + c * 2, V + c * 2, inst_desc(D));
                    commit(&empty[st]);
                    if (halves == 1) commit(&empty[st]);   // the other half's
                    commit(&o_done[h]);   // (last: the one that is waited for before the CTA ends)
                }
                __syncwarp();
            }
            if (!ok && h < halves) {   // the products already issued finish before tensor memory is released
                if (elect_one()) commit(&drain[h]);
                bar_wait_warp(&drain[h], 0, status, 107, true);
            }
        }
        __syncthreads();
        if (odd && warp < 4) {
            for (int r = 0; r < rows; r++) {
                const int rr = r0 + r, i2 = rr / f.G;
                slow_row<D>(a, b, kvh, kvh * f.G + rr - i2 * f.G, row0 + i2, pos0 + i2, tid, reinterpret_cast<float *>(smem));
            }
        }
    }
    fence_before();
    __syncthreads();
    if (warp == kIssuer) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
}

template <int D, int P>
cudaError_t prompt_launch(const PromptArgs &f, dim3 grid, cudaStream_t st) {
    static PerDevice<bool> opted;
    const cudaError_t e = smem_optin_once(moe_kv8_prompt_kernel<D, P>, opted);
    if (e != cudaSuccess) return e;
    return launch_pdl(moe_kv8_prompt_kernel<D, P>, grid, dim3(kThreads), (size_t)Smem<D>::kBytes + 1024, st, f);
}
template <int D>
cudaError_t prompt_page(const PromptArgs &f, dim3 grid, cudaStream_t st) {
    return f.a.c.P == 16 ? prompt_launch<D, 16>(f, grid, st) : f.a.c.P == 32 ? prompt_launch<D, 32>(f, grid, st) : prompt_launch<D, 64>(f, grid, st);
}

}  // namespace

cudaError_t launch_kv8_prompt(const Kv8Attend &a, int32_t *status, cudaStream_t st) {
    PromptArgs f{a, a.QH / a.c.KVH, status};
    // row tiles: a sequence's last may be partly filled
    const long long tiles = (long long)a.n_rows * f.G / (2 * kM) + a.n_seqs;
    const long long most = (long long)a.n_seqs * (((long long)a.max_new * f.G + 2 * kM - 1) / (2 * kM));
    const dim3 grid((unsigned)(std::min(tiles, most) * a.c.KVH));
    return a.c.D == 64 ? prompt_page<64>(f, grid, st) : prompt_page<128>(f, grid, st);
}
