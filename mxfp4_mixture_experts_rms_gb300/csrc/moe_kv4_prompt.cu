// moe_kv4_prompt.cu -- attention over the 4-bit paged cache for many new tokens
// a sequence (prompts, or pieces of them): tensor-core products on tcgen05 with
// accumulators in tensor memory.
//
// The CTA is that of the 8-bit cache's kernel (moe_kv8_prompt.cu): one per
// (sequence, kv head, 256 rows), 64 cached tokens a step, eight softmax warps,
// four that turn codes into operand tiles, one that copies pages, two that issue
// a half's products.  What differs:
//  * Keys and values become bf16, scale included: exact (E2M1 times a power of
//    two), so that no reference is needed however far the scales are apart.
//    Both tiles are [token][D], the same conversion; V's is read turned.
//  * Weights are bf16, 8 bits where a sum takes fp32 weights in the plain form:
//    with fp16 ones values would need a reference for each block of 32 dims.
//    Results are 2.0e-3 to 2.2e-3 from those in 64 bits (relative, over an
//    output), 1.6e-3 of it their own rounding to bf16; the sum of the weights is
//    fp32's.
//  * One softmax reference m, moved (to 16 above the largest score) only when a
//    score passes it, so that weights are at most 1 and the accumulator in tensor
//    memory is rarely rescaled (at 8 above, a tenth of a step's time was that).
//  * Weights go back to tensor memory, over the scores they come from, and are an
//    operand there: no tile of them in shared memory, and no wait for one.
//  * The values of a block are finite whatever the cache holds, so that a token
//    that a row does not see adds nothing to it.
// 4 x 900 ragged rows over up to 2700 tokens, 32 / 8 heads of 128, take 76 us, 23
// at the rate of large matrix products.  A step takes about 2050 cycles, in which
// the tensor pipe is 80 % and issue 70 % busy; a CTA's start and end, 6 us, and
// what 1.9 CTAs an SM leave idle are the rest.  Two score buffers or one and
// weights beside it, eight warps to decode (83 us), and a table in place of the
// conversions made no difference or a worse one.
#include "moe_kv_prompt.cuh"
#include "moe_kv4.cuh"

#include <algorithm>
#include <climits>

namespace {

template <int D>
struct Smem {   // offsets from a 1024-byte boundary
    static constexpr int kStages = 4, kRaw = D == 64 ? 4 : 2;   // operand tiles; steps of copied pages
    static constexpr int kStep = kT * D / 16 * 17;          // bytes of one
    static constexpr int kQ = 0;
    static constexpr int kQ1 = kM * D * 2;                  // of a half [128][D]
    static constexpr int kK = 2 * kQ1;                      // kStages x [64][D]
    static constexpr int kV = kK + kStages * kT * D * 2;    // kStages x [64][D]
    static constexpr int kCodes = kV + kStages * kT * D * 2; // kRaw x pages
    static constexpr int kBytes = kCodes + kRaw * kStep;
};

// V's tile [64][D], read with its rows as K: halves of 64 dims kT * 128 bytes
// apart, groups of eight rows 1024.
__device__ __forceinline__ uint64_t turned_desc(uint32_t at) {
    return (uint64_t)((at >> 4) & 0x3FFFu) | (uint64_t)(kT * 128 >> 4) << 16 | (uint64_t)(1024 >> 4) << 32 | (uint64_t)1 << 46 | (uint64_t)2 << 61;
}

struct PromptArgs {
    Kv4Attend a;
    int G;
    int32_t *status;
};

// 32 columns of the thread's TMEM lane.
__device__ __forceinline__ void tmem_st32(uint32_t at, const uint32_t (&v)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,"
        "%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32}; tcgen05.wait::st.sync.aligned;" ::"r"(at),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]),
        "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]), "r"(v[19]), "r"(v[20]),
        "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
        : "memory");
}
// The first operand from tensor memory: a lane a row, a column two of K.
template <bool ACC>
__device__ __forceinline__ void mma_tmem(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc) {
    asm volatile("{ .reg .pred p; setp.ne.b32 p, %4, 0; tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p; }" ::"r"(d),
                 "r"(a), "l"(b), "r"(idesc), "n"(ACC ? 1 : 0));
}
// (x0, x1) * k.
__device__ __forceinline__ void mul2(float &y0, float &y1, float x0, float x1, float k) {
    asm("{ .reg .b64 a, b; mov.b64 a, {%2, %3}; mov.b64 b, {%4, %4}; mul.rn.f32x2 a, a, b; mov.b64 {%0, %1}, a; }"
        : "=f"(y0), "=f"(y1) : "f"(x0), "f"(x1), "f"(k));
}
// A block of 32 codes with its scale -> 64 bytes of bf16, exact, by way of fp32:
// the conversions' pipe is what bounds the decoders, and this takes it twice a
// pair (four times with fp16's bits shifted to bf16's places: the kernel took 104
// us with that when it took 87 with this).
__device__ __forceinline__ void decode32(uint4 codes, float scale, uint4 (&out)[4]) {
    const uint32_t w[4] = {codes.x, codes.y, codes.z, codes.w};
#pragma unroll
    for (int c = 0; c < 4; c++) {
        uint32_t h[4];
        e2m1x8_to_f16(w[c], h);
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const float2 x = __half22float2(*reinterpret_cast<const __half2 *>(&h[i]));
            float y, z;
            mul2(y, z, x.x, x.y, scale);
            h[i] = bits_of(__floats2bfloat162_rn(y, z));
        }
        out[c] = make_uint4(h[0], h[1], h[2], h[3]);
    }
}
template <int D, int P>
__global__ void __launch_bounds__(kThreads, 1) moe_kv4_prompt_kernel(const __grid_constant__ PromptArgs f) {
    constexpr int NP = kT / P, NB = D / 32, PB = kv4_page_bytes(P, D);
    typedef Smem<D> L;
    constexpr int kStages = L::kStages, kRaw = L::kRaw;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *smem = reinterpret_cast<unsigned char *>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    __shared__ __align__(8) uint64_t raw[kRaw], raw_empty[kRaw], full[kStages], empty[kStages], s_full[2][2], q_full[2], p_full[2][2], o_done[2][2], drain[2];
    __shared__ uint32_t rmeta[kRaw], meta[kStages];   // the pages that are there
    __shared__ uint32_t tmem_slot;
    __shared__ int job[5];   // sequence (-1: none), tile, and the sequence's first row, rows, first position
    const Kv4Attend &a = f.a;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, kvh = blockIdx.x % a.c.KVH;
    if (tid == 0) {
        for (int s = 0; s < kStages; s++) bar_init(&full[s], kLoaders / 32), bar_init(&empty[s], 2);
        for (int s = 0; s < kRaw; s++) bar_init(&raw[s], 2), bar_init(&raw_empty[s], kLoaders / 32);
        for (int h = 0; h < 2; h++)
            bar_init(&s_full[h][0], 1), bar_init(&s_full[h][1], 1), bar_init(&q_full[h], kSoftmax / 2), bar_init(&p_full[h][0], kSoftmax / 2),
                bar_init(&p_full[h][1], kSoftmax / 2), bar_init(&o_done[h][0], 1), bar_init(&o_done[h][1], 1), bar_init(&drain[h], 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kIssuer) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&tmem_slot)));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (warp == 0) {
        // a tile of 256 rows, its heads together
        int x = blockIdx.x / a.c.KVH, found = -1, rt = 0, row0 = 0, n = 0, pos0 = 0;
        auto take = [&](int at, int tile) {   // lane at's sequence
            found = at, rt = __shfl_sync(0xffffffffu, tile, at);
            row0 = __shfl_sync(0xffffffffu, row0, at), n = __shfl_sync(0xffffffffu, n, at), pos0 = __shfl_sync(0xffffffffu, pos0, at);
        };
        auto running = [&](int v) {
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, v, o);
                if (lane >= o) v += y;
            }
            return v;
        };
        if (a.n_seqs <= 32) {
            // the x-th by the steps up to its last row, longest first, so that the last to start are short (4 x 900 rows over
            // 2700 tokens: 78 us; in the order below 78 to 85, as the sequences come)
            if (lane < a.n_seqs) kv8_rows(a, lane, row0, n, pos0);
            const int rows = n * f.G, tiles = (rows + 2 * kM - 1) / (2 * kM);
            auto longer = [&](int k) {   // how many of the lane's have more than k + 1 steps (all: k < 0)
                const long long r = k < 0 ? 0 : max(((long long)(k + 1) * kT - pos0) * f.G, 0ll);   // the first row that reaches as far
                return r >= rows ? 0 : tiles - (int)(r / (2 * kM));
            };
            if (__reduce_add_sync(0xffffffffu, tiles) > x) {
                // the least k that no more than x are longer than
                int lo = -1, hi = (int)((long long)a.width * P / kT) + 1;
                if (__reduce_add_sync(0xffffffffu, longer(hi)) > x) lo = hi, hi = INT_MAX / kT;   // (positions past the table)
                while (hi - lo > 1) {
                    const int mid = lo + (hi - lo) / 2;
                    if (__reduce_add_sync(0xffffffffu, longer(mid)) > x) lo = mid;
                    else hi = mid;
                }
                const int more = longer(hi), mine = longer(hi - 1) - more;
                x -= __reduce_add_sync(0xffffffffu, more);
                const int inc = running(mine);
                take(__ffs(__ballot_sync(0xffffffffu, x < inc)) - 1, tiles - more - 1 - (x - (inc - mine)));
            }
        } else {
            // sequences in order, a sequence's last (longest) tile first
            for (int b0 = 0; b0 < a.n_seqs && found < 0; b0 += 32) {
                n = 0;
                if (b0 + lane < a.n_seqs) kv8_rows(a, b0 + lane, row0, n, pos0);
                const int inc = running((n * f.G + 2 * kM - 1) / (2 * kM));
                const unsigned hit = __ballot_sync(0xffffffffu, x < inc);
                if (hit) {
                    take(__ffs(hit) - 1, inc - 1 - x);
                    found += b0;
                } else {
                    x -= __shfl_sync(0xffffffffu, inc, 31);
                }
            }
        }
        if (lane == 0) job[0] = found, job[1] = rt, job[2] = row0, job[3] = n, job[4] = pos0;
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
        const int row0 = job[2], n = job[3], pos0 = job[4];
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
                // tokens from .. to that the row sees (where their pages are)
                const int to = on ? min(seen - 1, pos0 + i2) : -1, from = kv8_first(pos0 + i2, a.window);
                {
                    const uint4 *q = reinterpret_cast<const uint4 *>(a.q + (long long)(row0 + i2) * a.q_stride + head * D);
#pragma unroll
                    for (int c = 0; c < D / 8; c++)
                        *reinterpret_cast<uint4 *>(smem + L::kQ + h * L::kQ1 + (c / 8) * (kM * 128) + swizzled(r, c % 8)) = on ? __ldg(q + c) : make_uint4(0, 0, 0, 0);
                    fence_async();
                    bar_arrive_warp(&q_full[h]);
                }
                const float sc = a.scale * kLog2e;
                float m = -INFINITY, l = 0.f;
                const uint32_t lanes = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + 256 * h;
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
                    const uint32_t there = meta[st];
                    tmem_wait(s);
                    tmem_wait(s + 32);
                    if (!(t0 >= from && t0 + kT - 1 <= to && there == (1u << NP) - 1)) {
                        const int c0 = max(from - t0, 0), c1 = min(to - t0, kT - 1);   // columns that the row sees
                        uint64_t sees = c1 < c0 ? 0 : ~0ull >> (kT - 1 - c1) & ~0ull << c0;
#pragma unroll
                        for (int p = 0; p < NP; p++)
                            if (!(there >> p & 1)) sees &= ~(~0ull >> (64 - P) << (p * P));
#pragma unroll
                        for (int c = 0; c < kT; c++)
                            if (!(sees >> c & 1)) s[c] = -INFINITY;
                    }
                    float x[4];   // four chains
#pragma unroll
                    for (int c = 0; c < 4; c++) x[c] = fmaxf(s[c], s[4 + c]);
#pragma unroll
                    for (int c = 8; c < kT; c += 8)
#pragma unroll
                        for (int e = 0; e < 4; e++) x[e] = max3(x[e], s[c + e], s[c + 4 + e]);
                    const float mx = fmaxf(max3(x[0], x[1], x[2]), x[3]) * sc;
                    float corr = 1.f;
                    const bool move = mx > m;
                    if (move) {
                        const float mn = mx + 16.f;
                        corr = ex2(m - mn);
                        l *= corr, m = mn;
                    }
                    const float ms = m == -INFINITY ? 0.f : m;
                    // large scores: products rounded as the maximum was
                    float ks = sc;
                    if (__any_sync(0xffffffffu, fabsf(ms) >= 0x1p17f)) {
#pragma unroll
                        for (int c = 0; c < kT; c++) s[c] = __fmul_rn(s[c], sc);
                        ks = 1.f;
                    }
                    if (__any_sync(0xffffffffu, move || !ok)) {
                        // the accumulator is that of the step before
                        if (j > 0) ok = bar_wait(&o_done[h][(j - 1) & 1], (uint32_t)((j - 1) >> 1) & 1, status, 101) && ok;
                        ok = __all_sync(0xffffffffu, ok);
                        if (!ok) break;
                        fence_after();
                        if (j > 0) {
#pragma unroll 1
                            for (int c = 0; c < D; c += 16) tmem_scale16(lanes + 2 * kT + c, corr);
                        }
                    }
                    float s0 = 0.f, s1 = 0.f;
                    uint32_t y[kT / 2];
#pragma unroll
                    for (int c = 0; c < kT / 2; c++) {
                        float w0, w1;
                        fma2(w0, w1, s[2 * c], s[2 * c + 1], ks, -ms);
                        w0 = ex2(w0), w1 = ex2(w1);
                        add2(s0, s1, w0, w1);
                        y[c] = bits_of(__floats2bfloat162_rn(w0, w1));
                    }
                    l += s0 + s1;
                    tmem_st32(lanes + (j & 1) * kT, y);   // over the scores
                    fence_before();
                    bar_arrive_warp(&p_full[h][j & 1]);   // (the next step's may come before this one is waited for)
                }
                if (ok) ok = bar_wait_warp(&o_done[h][(steps - 1) & 1], (uint32_t)((steps - 1) >> 1) & 1, status, 102);
                if (ok) {
                    fence_after();
                    // (the row anew, so that no registers hold it meanwhile)
                    uint32_t r;
                    asm volatile("mov.u32 %0, %%tid.x;" : "=r"(r));
                    r &= kM - 1;
                    const int row0 = *(volatile int *)&job[2], n = *(volatile int *)&job[3];
                    const int rr = (*(volatile int *)&job[1] * 2 + h) * kM + (int)r, i2 = rr / f.G, head = kvh * f.G + rr - i2 * f.G;
                    const bool on = rr < n * f.G;
                    const float sink = on && a.sinks ? a.sinks[head] * kLog2e : -INFINITY;
                    const float top = fmaxf(m, sink);
                    const float den = top == -INFINITY ? l : (m == -INFINITY ? l : l * ex2(m - top)) + ex2(sink - top);
                    // two factors: their product may be below 2^-126 where the output is not
                    const float k1 = den == 0.f || m == -INFINITY ? 0.f : ex2(0.5f * (m - top)), k2 = k1 == 0.f ? 0.f : k1 / den;
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
                const int st = j % kStages, slot = j % kRaw;
                ok = bar_wait_warp(&raw[slot], (uint32_t)(j / kRaw) & 1, status, 108);
                if (!ok) break;
                if (j >= kStages) {
                    ok = bar_wait_warp(&empty[st], (uint32_t)(j / kStages - 1) & 1, status, 103);
                    if (!ok) break;
                }
                const uint32_t there = rmeta[slot];
                // a block a thread: tokens side by side, so that a tile's rows are stored without conflicts; what no page
                // brought is what the slot held before, and never seen
                const unsigned char *codes = smem + L::kCodes + slot * L::kStep;
                unsigned char *K = smem + L::kK + st * (kT * D * 2), *V = smem + L::kV + st * (kT * D * 2);
#pragma unroll
                for (int i = 0; i < 2 * NB * kT / kLoaders; i++) {
                    const int at = x + i * kLoaders, tok = at % kT, b = at / kT % NB, side = at / kT / NB;
                    const unsigned char *page = codes + tok / P * PB;
                    const uint4 w = *reinterpret_cast<const uint4 *>(page + side * (P * D / 2) + (b * P + tok % P) * 16);
                    uint4 y[4];
                    decode32(w, kv4_scale(page[P * D + (side * NB + b) * P + tok % P / 16 * 16 + kv4_scale_byte(tok % 16)]), y);
                    unsigned char *tile = (side ? V : K) + b / 2 * (kT * 128);
#pragma unroll
                    for (int c = 0; c < 4; c++) *reinterpret_cast<uint4 *>(tile + swizzled(tok, b % 2 * 4 + c)) = y[c];
                }
                bar_arrive_warp(&raw_empty[slot]);
                if (x == 0) meta[st] = there;
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
                                 "r"((uint32_t)(__popc(there) * PB)) : "memory");
                __syncwarp();
                if (pg >= 0)
                    bulk_copy(smem_u32(smem + L::kCodes + slot * L::kStep) + lane * PB, a.c.c + ((size_t)pg * a.c.KVH + kvh) * PB, PB, smem_u32(&raw[slot]));
                pg = page_of(issued + 1);
                if (lane == 0) rmeta[slot] = there;
                bar_arrive_warp(&raw[slot]);   // the slot's second arrival
            }
            // copies still in flight land before the shared memory goes
            for (int j = max(0, issued - kRaw); j < issued; j++) bar_wait_warp(&raw[j % kRaw], (uint32_t)(j / kRaw) & 1, status, 109, true);
        } else {
            // ---- a half's products: the warp together, so that descriptors stay in uniform registers; one lane issues ----
            const int h = warp - kIssuer;
            const uint64_t Q = tile_desc(smem_u32(smem + L::kQ + h * L::kQ1));
            const uint64_t K0 = tile_desc(smem_u32(smem + L::kK)), V0 = turned_desc(smem_u32(smem + L::kV));
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
                        if (c == 0) mma<false>(to, q, k, inst_desc(kT, true));
                        else mma<true>(to, q, k, inst_desc(kT, true));
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
                // the next scores go ahead of this step's values: into the columns of step j - 1's weights, once its products are done
                if (j > 0) ok = bar_wait_warp(&o_done[h][(j - 1) & 1], (uint32_t)((j - 1) >> 1) & 1, status, 111);
                if (ok && j + 1 < steps) ok = scores(j + 1, st1, par1);
                if (ok) ok = bar_wait_warp(&p_full[h][j & 1], (uint32_t)(j >> 1) & 1, status, 106);
                if (!ok) break;
                fence_after();
                const uint64_t V = V0 + st * kTile16;
                if (elect_one()) {
                    // 16 tokens are two groups of eight rows of the tile, 1024 bytes each
                    const uint32_t W = S + (j & 1) * kT;
                    if (j == 0) mma_tmem<false>(O, W, V, inst_desc(D, true, true));
                    else mma_tmem<true>(O, W, V, inst_desc(D, true, true));
#pragma unroll
                    for (int c = 1; c < kT / 16; c++) mma_tmem<true>(O, W + c * 8, V + c * 128, inst_desc(D, true, true));
                    commit(&empty[st]);
                    if (halves == 1) commit(&empty[st]);   // the other half's
                    commit(&o_done[h][j & 1]);   // (last: the one that is waited for before the CTA ends)
                }
                __syncwarp();
            }
            if (!ok && h < halves) {   // the products already issued finish before tensor memory is released
                if (elect_one()) commit(&drain[h]);
                bar_wait_warp(&drain[h], 0, status, 107, true);
            }
        }
        __syncthreads();
    }
    fence_before();
    __syncthreads();
    if (warp == kIssuer) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
}

template <int D, int P>
cudaError_t prompt_launch(const PromptArgs &f, dim3 grid, cudaStream_t st) {
    static PerDevice<bool> opted;
    const cudaError_t e = smem_optin_once(moe_kv4_prompt_kernel<D, P>, opted);
    if (e != cudaSuccess) return e;
    return launch_pdl(moe_kv4_prompt_kernel<D, P>, grid, dim3(kThreads), (size_t)Smem<D>::kBytes + 1024, st, f);
}
template <int D>
cudaError_t prompt_page(const PromptArgs &f, dim3 grid, cudaStream_t st) {
    return f.a.c.P == 16 ? prompt_launch<D, 16>(f, grid, st) : f.a.c.P == 32 ? prompt_launch<D, 32>(f, grid, st) : prompt_launch<D, 64>(f, grid, st);
}

}  // namespace

cudaError_t launch_kv4_prompt(const Kv4Attend &a, int32_t *status, cudaStream_t st) {
    PromptArgs f{a, a.QH / a.c.KVH, status};
    // row tiles: a sequence's last may be partly filled
    const long long tiles = (long long)a.n_rows * f.G / (2 * kM) + a.n_seqs;
    const long long most = (long long)a.n_seqs * (((long long)a.max_new * f.G + 2 * kM - 1) / (2 * kM));
    const dim3 grid((unsigned)(std::min(tiles, most) * a.c.KVH));
    return a.c.D == 64 ? prompt_page<64>(f, grid, st) : prompt_page<128>(f, grid, st);
}
