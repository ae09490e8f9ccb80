// moe_kv8_attend.cu -- attention over the 8-bit paged key/value cache: a few
// new tokens a sequence (decode steps), or prompts.
#include "moe_kv8.cuh"

#include <algorithm>

namespace {

// One CTA per (query head, new token, sequence): 128 keys at a time, a thread
// per key for the scores and per dim for the values.
template <int D>
__global__ void __launch_bounds__(128) moe_kv8_attend_kernel(const Kv8Attend a) {
    __shared__ float qs[D], p[128], vsc[128], red[4];
    __shared__ const uint8_t *vat[128];
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int h = blockIdx.x, i = blockIdx.y, b = blockIdx.z, tid = threadIdx.x, P = a.c.P;
    int row0, n, pos0;
    kv8_rows(a, b, row0, n, pos0);
    if (i >= n) return;
    const int pos = pos0 + i, kvh = h / (a.QH / a.c.KVH);
    const int last = min((long long)pos, (long long)a.width * P - 1);
    const int first = a.window > 0 ? max(0, pos - a.window + 1) : 0;
    const uint16_t *q = a.q + (long long)(row0 + i) * a.q_stride + h * D;
    for (int d = tid; d < D; d += 128) qs[d] = bf16_to_f32(q[d]) * a.scale;
    __syncthreads();
    float m = -INFINITY, l = 0.f, acc = 0.f;
    const int dim = tid % D, part = tid / D, parts = 128 / D;  // the thread's dim and share of the keys
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
                for (int c = 0; c < D / 16; c++) {
                    const uint4 w = *reinterpret_cast<const uint4 *>(kp + (size_t)c * P * 16);
                    const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int j = 0; j < 4; j++) {
                        const float2 x = e4m3x2_to_f32(ww[j]), y = e4m3x2_to_f32(ww[j] >> 16);
                        const float *qq = qs + c * 16 + 4 * j;
                        dot += x.x * qq[0] + x.y * qq[1] + y.x * qq[2] + y.y * qq[3];
                    }
                }
                s = dot * pow2i(a.c.ks[ph] - 127);
                vat[tid] = a.c.v + ph * (P * D) + (size_t)(off / 16) * D * 16 + kv8_value_byte(off % 16);
                vsc[tid] = pow2i(a.c.vs[ph] - 127);
            }
        }
        float cm = s;
        for (int x = 16; x; x >>= 1) cm = fmaxf(cm, __shfl_xor_sync(0xffffffffu, cm, x));
        if (tid % 32 == 0) red[tid / 32] = cm;
        __syncthreads();
        const float mn = fmaxf(m, fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])));
        const float f = mn == -INFINITY ? 1.f : expf(m - mn);
        p[tid] = vat[tid] ? expf(s - mn) : 0.f;
        __syncthreads();
        acc *= f, l *= f, m = mn;
        for (int j = part; j < 128; j += parts)
            if (vat[j]) acc += p[j] * vsc[j] * e4m3x2_to_f32(vat[j][dim * 16]).x;
        for (int j = 0; j < 128; j++) l += p[j];
        __syncthreads();
    }
    if (parts == 2) {
        p[tid] = acc;
        __syncthreads();
        if (part) return;
        acc += p[tid + D];
    }
    if (a.sinks) {
        const float mn = fmaxf(m, a.sinks[h]), f = mn == -INFINITY ? 0.f : expf(m - mn);
        acc *= f, l = l * f + (mn == -INFINITY ? 0.f : expf(a.sinks[h] - mn));
    }
    const __nv_bfloat16 r = __float2bfloat16_rn(l > 0.f ? acc / l : (l == 0.f ? 0.f : l));
    a.out[(long long)(row0 + i) * a.o_stride + h * D + dim] = *reinterpret_cast<const uint16_t *>(&r);
}

// ---- few new tokens a sequence: keys and values streamed once ----
//
// The work is cut into units: 64 consecutive tokens of a sequence for one kv
// head and 16 rows (new tokens x the kv head's query heads).  Units lie in
// order of (sequence, kv head, row tile, tokens); the (sequence, kv head, row
// tile) is a job.  Each CTA takes one contiguous share of the units, each of
// its warps one contiguous share of the CTA's, so ragged lengths balance
// whatever they are, with nothing on the host: every CTA scans the lengths.
// A warp is on its own: it copies its units' pages by bulk copies into a ring
// of its own, and runs scores, softmax and values on mma.sync m16n8k16 (fp16
// operands, E4M3 codes converted exactly; fp32 accumulators).  What a share
// cuts apart is joined in a fixed order: inside the CTA through shared memory,
// across CTAs through the workspace by the last CTA of the job to arrive (one
// ticket per CTA: a CTA begins at most one job that others continue).
//
// Softmax, per row, in units of log2: m the running maximum of the scores s, l
// the sum of 2^(s - m).  The values' accumulator has a reference M of its own,
// M = m + N, the running maximum of (a token's score + its value exponent): it
// holds sum 2^(15 + s + e - M) * code over value codes with
// page exponent e, so that the fp16 weights 2^(15 + s + e - M) <= 2^15 keep 11
// bits down to 2^-29 of the largest, however far the pages' scales are apart.
// q is scaled per row by a power of two into fp16's range: exact for a bf16
// row's values down to 2^-28 of its largest.
constexpr int kTile = 64;             // tokens of a unit
constexpr int kRows = 16;             // rows of a unit
constexpr int kMaxCtas = 256;
constexpr uint64_t kWaitNs = 2000000000ull;
constexpr float kLog2e = 1.4426950408889634f;

template <int D, bool TOP>
struct Few {
    // as many as leave room for two or three units of each in the ring
    static constexpr int kWarps = D == 64 ? (TOP ? 7 : 8) : (TOP ? 5 : 6);
    static constexpr int kStage = 2 * kTile * D;   // bytes of one unit: keys, values
    static constexpr int kPad = D + 8;             // floats of a partial's row: 64-bit stores on distinct banks
};
// A partial: acc [rows][D + 8], then m, l, N [rows] each.
__host__ __device__ constexpr int partial_floats(int rows, int D) { return rows * (D + 8 + 3); }

struct FewArgs {
    Kv8Attend a;
    int G, stages, rows8;      // query heads per kv head; ring stages; rows of a partial (8 or 16)
    int32_t *status;           // [2]
    uint32_t *tickets;         // [kMaxCtas], zero between calls
    float *parts;              // [kMaxCtas][2][partial_floats]
};

__device__ __forceinline__ uint32_t smem_u32(const void *p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }
__device__ __forceinline__ bool bar_try(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile("{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
                 : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
    return ok != 0;
}
// Bounded wait of a whole warp: false (and the status word set) after about 2 s.
__device__ bool bar_wait(uint32_t bar, uint32_t parity, int32_t *status, int where) {
    if (bar_try(bar, parity)) return true;
    uint64_t t0, t1;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t0));
    for (uint32_t i = 1;; i++) {
        if (bar_try(bar, parity)) return true;
        if ((i & 63) == 0) {
            asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t1));
            if (t1 - t0 > kWaitNs) {
                set_device_error(status, MOE_DEV_WAIT_TIMEOUT, where);
                return false;
            }
        }
    }
}
__device__ __forceinline__ void bulk_copy(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ uint32_t pack_f16(float x, float y) {
    const __half2 h = __floats2half2_rn(x, y);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ float quad_max(float v) {
    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
    return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
}
__device__ __forceinline__ float quad_sum(float v) {
    v += __shfl_xor_sync(0xffffffffu, v, 1);
    return v + __shfl_xor_sync(0xffffffffu, v, 2);
}

// A share's boundary c of n over `units`: the even cut, moved down to its
// job's first unit where the job is at most 8 units long (a job that one CTA
// can take at once is not worth joining across two).
struct Plan {
    const int *cum;          // [n_seqs]: units of the sequences before, per kv head
    const int *lo, *len;     // [n_seqs]: first unit's index in the sequence; tokens of it that can be seen
    int n_seqs, KVH, G;
    long long units;
};

struct Job {
    int b, h, rt, n_rt, nt;  // sequence, kv head, row tile of n_rt, units of the job
    long long u0;            // its first unit
};

// The job of unit u (0 <= u < units).
__device__ __forceinline__ void job_of(const Plan &p, const Kv8Attend &a, long long u, Job &j) {
    int lo = 0, hi = p.n_seqs;   // the last sequence with KVH * cum <= u
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if ((long long)p.cum[mid] * p.KVH <= u) lo = mid;
        else hi = mid;
    }
    const int per = (lo + 1 < p.n_seqs ? p.cum[lo + 1] : (int)(p.units / p.KVH)) - p.cum[lo];  // units per kv head
    j.b = lo;
    const int off = (int)(u - (long long)p.cum[lo] * p.KVH);   // < 2^31 (checked on the host)
    j.h = off / per;
    j.nt = max(1, (p.len[lo] + kTile - 1) / kTile - p.lo[lo]);
    j.n_rt = per / j.nt;
    j.rt = off % per / j.nt;
    j.u0 = (long long)p.cum[lo] * p.KVH + (long long)j.h * per + (long long)j.rt * j.nt;
}

// One warp's place in its units: where the next unit's pages come from.
template <int D, int P, bool TOP>
__global__ void __launch_bounds__(Few<D, TOP>::kWarps * 32, 1) moe_kv8_few_kernel(const __grid_constant__ FewArgs f) {
    constexpr int W = Few<D, TOP>::kWarps, NP = kTile / P, NC = D / 16, ST = Few<D, TOP>::kStage, PAD = Few<D, TOP>::kPad;
    extern __shared__ __align__(128) unsigned char smem_raw[];
    __shared__ __align__(8) uint64_t bars[W][4];
    __shared__ uint32_t meta[W][4][NP];           // per stage and page: key exponent byte, value's, 1 if it is there
    __shared__ int scan[W + 1];
    __shared__ long long seg_job[2 * W];          // first unit of the job of each warp's partials, -1: none
    __shared__ int s_last;
    const Kv8Attend &a = f.a;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t4 = lane & 3;
    const int S = f.stages, R = f.rows8, PF = partial_floats(R, D);
    unsigned char *ring = smem_raw + (size_t)warp * S * ST;
    float *part = reinterpret_cast<float *>(smem_raw + (size_t)W * S * ST);   // [W] head partials; tails go over the rings
    int *cum = reinterpret_cast<int *>(part + (size_t)W * PF), *lo_s = cum + a.n_seqs, *len_s = lo_s + a.n_seqs;
    if (lane == 0)
        for (int s = 0; s < S; s++) asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(smem_u32(&bars[warp][s])));
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");

    // every sequence's units: contiguous shares of sequences per thread, one block scan
    const int per_thr = (a.n_seqs + W * 32 - 1) / (W * 32), sb0 = min(tid * per_thr, a.n_seqs), sb1 = min(sb0 + per_thr, a.n_seqs);
    int mine = 0;
    for (int b = sb0; b < sb1; b++) {
        int row0, n, pos0;
        kv8_rows(a, b, row0, n, pos0);
        const int seen = (int)max(0ll, min((long long)a.lens[b], (long long)a.width * P));
        const int first = a.window > 0 ? max(0, pos0 - a.window + 1) / kTile : 0;
        const int cnt = n > 0 ? max(1, (seen + kTile - 1) / kTile - first) * ((n * f.G + kRows - 1) / kRows) : 0;
        lo_s[b] = first, len_s[b] = seen, cum[b] = mine;
        mine += cnt;
    }
    int inc = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, inc, d);
        if (lane >= d) inc += o;
    }
    if (lane == 31) scan[warp] = inc;
    __syncthreads();
    int base = inc - mine, total = 0;
#pragma unroll
    for (int w = 0; w < W; w++) {
        if (w < warp) base += scan[w];
        total += scan[w];
    }
    for (int b = sb0; b < sb1; b++) cum[b] += base;
    __syncthreads();
    Plan pl{cum, lo_s, len_s, a.n_seqs, a.c.KVH, f.G, (long long)total * a.c.KVH};
    const int ctas = (int)min((long long)gridDim.x, (pl.units + 3) / 4);
    if ((int)blockIdx.x >= ctas) return;
    auto cut = [&](int c) {
        long long u = pl.units * c / ctas;
        if (u > 0 && u < pl.units) {
            Job j;
            job_of(pl, a, u, j);
            if (j.nt <= 8) u = j.u0;
        }
        return u;
    };
    const long long c0 = cut(blockIdx.x), c1 = cut(blockIdx.x + 1);
    const long long u0 = c0 + (c1 - c0) * warp / W, u1 = c0 + (c1 - c0) * (warp + 1) / W;

    // the issuing side: place of the next unit to copy, its pages read one unit ahead
    Job ij;
    ij.nt = 1, ij.u0 = 0, ij.b = 0, ij.h = 0;
    long long iu = u0;
    int pg = -1;
    auto fetch_page = [&]() {   // lane p < NP: page of the unit iu
        pg = -1;
        if (iu < u1 && lane < NP) {
            const int tile = lo_s[ij.b] + (int)(iu - ij.u0);
            const int t0 = tile * kTile + lane * P;
            if (t0 < len_s[ij.b]) pg = __ldg(a.table + (size_t)ij.b * a.width + t0 / P);
        }
    };
    uint32_t pend = 0;
    int pend_stage = -1;
    auto flush = [&]() {
        if (pend_stage >= 0 && lane < NP) meta[warp][pend_stage][lane] = pend;
        pend_stage = -1;
    };
    auto issue = [&](int stage) {
        flush();
        const bool ok = lane < NP && pg >= 0 && pg < a.c.n_pages;
        const unsigned okm = __ballot_sync(0xffffffffu, ok);
        const uint32_t bar = smem_u32(&bars[warp][stage]);
        if (lane == 0)
            asm volatile("{ .reg .b64 st; mbarrier.arrive.expect_tx.shared::cta.b64 st, [%0], %1; }" ::"r"(bar),
                         "r"((uint32_t)(__popc(okm) * 2 * P * D)) : "memory");
        __syncwarp();
        pend = 0;
        if (ok) {
            const size_t ph = (size_t)pg * a.c.KVH + ij.h;
            const uint32_t dst = smem_u32(ring + stage * ST) + lane * (P * D);
            bulk_copy(dst, a.c.k + ph * (P * D), P * D, bar);
            bulk_copy(dst + kTile * D, a.c.v + ph * (P * D), P * D, bar);
            pend = (uint32_t)__ldg(a.c.ks + ph) | (uint32_t)__ldg(a.c.vs + ph) << 8 | 1u << 16;
        }
        pend_stage = stage;
        iu++;
        if (iu < u1 && iu >= ij.u0 + ij.nt) job_of(pl, a, iu, ij);
        fetch_page();
    };
    if (lane < 2) seg_job[2 * warp + lane] = -1;
    if (u0 < u1) {
        job_of(pl, a, u0, ij);
        fetch_page();
    }
    bool fine = true;
    int filled = 0;
    for (; filled < S && u0 + filled < u1; filled++) issue(filled);

    // the computing side
    float acc[D / 8][4], m[2], l[2], N[2];
    const float sc = a.scale * kLog2e;
    int up[2] = {0, 0};   // the rows' queries carry 2^up
    uint32_t qf[NC][4];
    Job j = ij;
    int pos[2] = {0, 0}, pmin = 0, pmax = 0;
    long long seg0 = u0;     // first unit of the running segment
    float *tail = nullptr;
    auto store_partial = [&](float *p) {
#pragma unroll
        for (int r = 0; r < (TOP ? 2 : 1); r++) {
            const float ls = quad_sum(l[r]);
            float *row = p + (g + 8 * r) * PAD;
#pragma unroll
            for (int d = 0; d < D / 8; d++)
                *reinterpret_cast<float2 *>(row + 8 * d + 2 * t4) = make_float2(acc[d][2 * r], acc[d][2 * r + 1]);
            if (t4 == 0) {
                float *ml = p + R * PAD + (g + 8 * r);
                ml[0] = m[r], ml[R] = ls, ml[2 * R] = N[r];
            }
        }
    };
    for (long long u = u0; u < u1 && fine; u++) {
        const int i = (int)(u - u0), stage = i % S;
        if (u == u0 || u == j.u0 + j.nt) {
            // a new job: its rows' queries, scaled per row into fp16
            job_of(pl, a, u, j);
            seg0 = u;
            int row0, n, pos0;
            kv8_rows(a, j.b, row0, n, pos0);
            pmin = pos0 + j.rt * kRows / f.G;
            pmax = pos0 + min(n * f.G - 1, j.rt * kRows + kRows - 1) / f.G;
#pragma unroll
            for (int r = 0; r < 2; r++) {
                const int rr = j.rt * kRows + g + 8 * r;
                const bool on = (TOP || r == 0) && rr < n * f.G;
                pos[r] = on ? pos0 + rr / f.G : -1;
                const uint16_t *q = a.q + (long long)(row0 + rr / f.G) * a.q_stride + (j.h * f.G + rr % f.G) * D + 4 * t4;
                uint2 w[NC];
                uint32_t am = 0;
#pragma unroll
                for (int c = 0; c < NC; c++) {
                    w[c] = on ? __ldg(reinterpret_cast<const uint2 *>(q + 16 * c)) : make_uint2(0, 0);
                    am = max(am, max(max(w[c].x & 0x7FFFu, (w[c].x >> 16) & 0x7FFFu), max(w[c].y & 0x7FFFu, (w[c].y >> 16) & 0x7FFFu)));
                }
                am = max(am, __shfl_xor_sync(0xffffffffu, am, 1));
                am = max(am, __shfl_xor_sync(0xffffffffu, am, 2));
                // largest magnitude to [2^14, 2^15): exponent field e means 2^(e - 127)
                const int e = (int)(am >> 7);
                up[r] = min(141 - e, 127);
                const float mul = pow2i(up[r]);
                m[r] = -INFINITY, l[r] = 0.f, N[r] = -INFINITY;
#pragma unroll
                for (int c = 0; c < NC; c++) {
                    qf[c][r] = pack_f16(__uint_as_float(w[c].x << 16) * mul, __uint_as_float(w[c].x & 0xFFFF0000u) * mul);
                    qf[c][2 + r] = pack_f16(__uint_as_float(w[c].y << 16) * mul, __uint_as_float(w[c].y & 0xFFFF0000u) * mul);
                }
            }
#pragma unroll
            for (int d = 0; d < D / 8; d++) acc[d][0] = acc[d][1] = acc[d][2] = acc[d][3] = 0.f;
        }
        if (pend_stage == stage) flush();
        __syncwarp();
        fine = bar_wait(smem_u32(&bars[warp][stage]), (uint32_t)(i / S) & 1, f.status, 90);
        fine = __all_sync(0xffffffffu, fine);
        if (!fine) break;
        const int t0 = (lo_s[j.b] + (int)(u - j.u0)) * kTile, seen = len_s[j.b];
        uint32_t mt[NP];
        bool whole = t0 + kTile <= seen && t0 + kTile - 1 <= pmin && (a.window == 0 || t0 > pmax - a.window);
#pragma unroll
        for (int p = 0; p < NP; p++) {
            mt[p] = meta[warp][stage][p];
            whole = whole && (mt[p] >> 16);
        }
        const uint32_t kb = smem_u32(ring + stage * ST), vb = kb + kTile * D;
        // scores: 8 token octets x (rows g: c0, c1; rows g + 8: c2, c3)
        float s[8][4];
#pragma unroll
        for (int n = 0; n < 8; n++) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
#pragma unroll
        for (int c = 0; c < NC; c++)
#pragma unroll
            for (int hf = 0; hf < 2; hf++) {
                // 32 tokens (lane: one) of dims 16 c ..: pages hold [D / 16][P][16]
                const int tok = 32 * hf + lane;
                uint32_t w[4];
                ldsm4(w, kb + (tok / P) * (P * D) + c * (P * 16) + (tok % P) * 16);
#pragma unroll
                for (int n = 0; n < 4; n++) {
                    uint32_t b0, b1;
                    e4m3x4_to_f16(w[n], b0, b1);
                    mma_f16(s[4 * hf + n], qf[c], b0, b1);
                }
            }
        uint32_t keep[4] = {0, 0, 0, 0};    // where not whole, per 16 tokens: bytes of the thread's value words some row sees
        uint32_t vis[2] = {0, 0};           // and the tokens that each row sees: bit 2 n + e
#pragma unroll
        for (int r = 0; r < (TOP ? 2 : 1); r++)
#pragma unroll
            for (int n = 0; n < 8; n++) {
                const float k = pow2i((int)(mt[n * 8 / P] & 255u) - 127 - up[r]) * sc;
                s[n][2 * r] *= k, s[n][2 * r + 1] *= k;
            }
        if (!whole) {
#pragma unroll
            for (int n = 0; n < 8; n++)
#pragma unroll
                for (int e = 0; e < 2; e++) {
                    const int t = t0 + 8 * n + 2 * t4 + e;
                    const bool there = t < seen && (mt[n * 8 / P] >> 16);
#pragma unroll
                    for (int r = 0; r < (TOP ? 2 : 1); r++) {
                        if (there && t <= pos[r] && (a.window == 0 || t > pos[r] - a.window)) vis[r] |= 1u << (2 * n + e);
                        else s[n][2 * r + e] = -INFINITY;
                    }
                    // token 8 (n & 1) + 2 t4 + e of its 16: byte 2 (n & 1) + e of the thread's word
                    if (there && t <= pmax && (a.window == 0 || t > pmin - a.window)) keep[n / 2] |= 0xFFu << (8 * (2 * (n & 1) + e));
                }
        }
        bool moved = false;
        float corr[2] = {1.f, 1.f}, fac[2][NP];
#pragma unroll
        for (int r = 0; r < (TOP ? 2 : 1); r++) {
            float mx = -INFINITY, pmx[NP];
#pragma unroll
            for (int p = 0; p < NP; p++) {
                float pm = -INFINITY;
#pragma unroll
                for (int n = p * (8 / NP); n < (p + 1) * (8 / NP); n++) pm = fmaxf(pm, fmaxf(s[n][2 * r], s[n][2 * r + 1]));
                pmx[p] = pm, mx = fmaxf(mx, pm);
            }
            mx = quad_max(mx);
            const float mn = fmaxf(m[r], mx), ms = mn == -INFINITY ? 0.f : mn;
            const float was = N[r] + (m[r] - ms);                    // the old reference, over the new m
            float mvr = -INFINITY;   // over the new m, as scores may be too large for an exponent beside them
#pragma unroll
            for (int p = 0; p < NP; p++) mvr = fmaxf(mvr, pmx[p] - ms + (float)((int)((mt[p] >> 8) & 255u) - 127));
            const float Nn = fmaxf(was, quad_max(mvr)), Ns = Nn == -INFINITY ? 0.f : Nn;
            l[r] *= ex2(m[r] - ms);
            corr[r] = ex2(was - Ns);
            moved |= Nn != was;
            m[r] = mn, N[r] = Nn;
#pragma unroll
            for (int p = 0; p < NP; p++) fac[r][p] = ex2(fminf((float)((int)((mt[p] >> 8) & 255u) - 112) - Ns, 126.f));
            float sum = 0.f;
#pragma unroll
            for (int n = 0; n < 8; n++)
#pragma unroll
                for (int e = 0; e < 2; e++) {
                    const float p = ex2(s[n][2 * r + e] - ms);
                    sum += p;
                    s[n][2 * r + e] = p * fac[r][n * 8 / P];
                }
            l[r] += sum;
        }
        if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
            for (int d = 0; d < D / 8; d++) {
                acc[d][0] *= corr[0], acc[d][1] *= corr[0];
                if (TOP) acc[d][2] *= corr[1], acc[d][3] *= corr[1];
            }
        }
#pragma unroll
        for (int kk = 0; kk < 4; kk++) {
            const uint32_t pf[4] = {pack_f16(s[2 * kk][0], s[2 * kk][1]), TOP ? pack_f16(s[2 * kk][2], s[2 * kk][3]) : 0u,
                                    pack_f16(s[2 * kk + 1][0], s[2 * kk + 1][1]),
                                    TOP ? pack_f16(s[2 * kk + 1][2], s[2 * kk + 1][3]) : 0u};
            const uint32_t blk = vb + (16 * kk / P) * (P * D) + (16 * kk % P) * D;   // [D][16] of these 16 tokens
#pragma unroll
            for (int q = 0; q < D / 32; q++) {
                uint32_t w[4];
                ldsm4(w, blk + (32 * q + lane) * 16);
#pragma unroll
                for (int n = 0; n < 4; n++) {
                    uint32_t b0, b1;
                    if (!whole) {
                        w[n] &= keep[kk];
                        // a NaN that only later rows see must not reach the others as 0 * NaN
                        const uint32_t nan = pmin == pmax ? 0 : ((w[n] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
                        if (__any_sync(0xffffffffu, nan != 0)) {
                            const uint32_t all = (nan >> 7) * 255u;
                            uint32_t seen1[4];
#pragma unroll
                            for (int x = 0; x < 4; x++) {
                                const uint32_t bits = vis[x & 1] >> (4 * kk + 2 * (x >> 1));
                                seen1[x] = (bits & 1u) * 0x3C00u | (bits >> 1 & 1u) * 0x3C000000u;
                            }
                            float hit[4] = {0.f, 0.f, 0.f, 0.f};
                            e4m3x4_to_f16(all & 0x38383838u, b0, b1);   // ones where the value is NaN
                            mma_f16(hit, seen1, b0, b1);
#pragma unroll
                            for (int x = 0; x < 4; x++)
                                if (hit[x] > 0.f) acc[4 * q + n][x] = NAN;
                            w[n] &= ~all;
                        }
                    }
                    e4m3x4_to_f16(w[n], b0, b1);
                    mma_f16(acc[4 * q + n], pf, b0, b1);
                }
            }
        }
        __syncwarp();
        if (u + S < u1) issue(stage);
        if (u + 1 == j.u0 + j.nt || u + 1 == u1) {
            if (seg0 == j.u0 && u + 1 == j.u0 + j.nt) {
                // the whole job was this warp's
                int row0, n, pos0;
                kv8_rows(a, j.b, row0, n, pos0);
#pragma unroll
                for (int r = 0; r < (TOP ? 2 : 1); r++) {
                    const int rr = j.rt * kRows + g + 8 * r;
                    const float ls = quad_sum(l[r]);
                    if (rr >= n * f.G) continue;
                    const int head = j.h * f.G + rr % f.G;
                    float den = ls, top = m[r];
                    if (a.sinks) {
                        const float sk = a.sinks[head] * kLog2e;
                        top = fmaxf(top, sk);
                        den = top == -INFINITY ? 0.f : ls * ex2(m[r] - top) + ex2(sk - top);
                    }
                    // an empty row: 0; NaN stays NaN
                    const float k = den == 0.f || N[r] == -INFINITY ? 0.f : ex2(N[r] - 15.f + (m[r] - top)) / den;
                    uint16_t *o = a.out + (long long)(row0 + rr / f.G) * a.o_stride + head * D + 2 * t4;
#pragma unroll
                    for (int d = 0; d < D / 8; d++) {
                        const __nv_bfloat162 v = __floats2bfloat162_rn(acc[d][2 * r] * k, acc[d][2 * r + 1] * k);
                        *reinterpret_cast<__nv_bfloat162 *>(o + 8 * d) = v;
                    }
                }
            } else {
                const bool head_seg = seg0 != j.u0;
                if (!head_seg || u + 1 == u1) {
                    // the warp's last segment: over its ring, once that is drained (below)
                    tail = reinterpret_cast<float *>(ring);
                } else {
                    store_partial(part + (size_t)warp * PF);
                    if (lane == 0) seg_job[2 * warp] = j.u0;
                }
            }
        }
    }
    // the ring is drained: every unit issued was waited for, or the wait ran out
    if (!fine) {
        for (int s = 0; s < S; s++) {
            // copies may still be in flight: wait for each stage's last phase, with a limit
            const int n = (int)(iu - u0);
            if (s < n) {
                const int last = (n - 1 - s) / S;
                bar_wait(smem_u32(&bars[warp][s]), (uint32_t)last & 1, f.status, 91);
            }
        }
        tail = nullptr;
    }
    __syncwarp();
    if (tail) {
        store_partial(tail);
        if (lane == 0) seg_job[2 * warp + 1] = j.u0;
    }
    __syncthreads();

    // joining: the CTA's segments in order; those of one job are neighbours
    for (int i = 0; i < 2 * W;) {
        const long long ju = seg_job[i];
        if (ju < 0) {
            i++;
            continue;
        }
        int z = i + 1, cnt = 1;
        for (int x = z; x < 2 * W; x++) {
            if (seg_job[x] < 0) continue;
            if (seg_job[x] != ju) break;
            z = x + 1, cnt++;
        }
        Job jj;
        job_of(pl, a, ju, jj);
        int row0, n, pos0;
        kv8_rows(a, jj.b, row0, n, pos0);
        const int rows = min(kRows, n * f.G - jj.rt * kRows);
        const bool inside = ju >= c0 && ju + jj.nt <= c1;    // the whole job was this CTA's
        auto at = [&](int x) { return x & 1 ? reinterpret_cast<const float *>(smem_raw + (size_t)(x >> 1) * S * ST) : part + (size_t)(x >> 1) * PF; };
        // which CTAs share it, and where their partials are
        const int fc = inside ? 0 : (int)(((ju + 1) * ctas - 1) / pl.units), ec = inside ? 0 : (int)(((ju + jj.nt) * ctas - 1) / pl.units);
        float *mine_p = f.parts + ((size_t)blockIdx.x * 2 + (ju >= c0 ? 1 : 0)) * PF;
        bool finish = inside;
        int n_parts = cnt;
        if (!inside) {
            for (int x = tid; x < rows * (D / 2); x += W * 32) {
                const int r = x / (D / 2), d = 2 * (x % (D / 2));
                float mm = -INFINITY, NN = -INFINITY, ll = 0.f;
                for (int k = i; k < z; k++)
                    if (seg_job[k] >= 0) mm = fmaxf(mm, at(k)[R * PAD + r]);
                const float ms = mm == -INFINITY ? 0.f : mm;
                for (int k = i; k < z; k++)
                    if (seg_job[k] >= 0) NN = fmaxf(NN, at(k)[R * PAD + r] - ms + at(k)[R * PAD + 2 * R + r]);
                float2 v = make_float2(0.f, 0.f);
                for (int k = i; k < z; k++)
                    if (seg_job[k] >= 0) {
                        const float *ml = at(k) + R * PAD + r;
                        const float2 w = *reinterpret_cast<const float2 *>(at(k) + r * PAD + d);
                        const float c = ml[2 * R] == -INFINITY ? 0.f : ex2(ml[0] - ms + ml[2 * R] - NN);
                        v.x += c * w.x, v.y += c * w.y;
                        ll += ml[R] * (ml[0] == -INFINITY ? 1.f : ex2(ml[0] - ms));
                    }
                *reinterpret_cast<float2 *>(mine_p + r * PAD + d) = v;
                if (d == 0) mine_p[R * PAD + r] = mm, mine_p[R * PAD + R + r] = ll, mine_p[R * PAD + 2 * R + r] = NN;
            }
            __threadfence();
            __syncthreads();
            if (tid == 0) {
                const uint32_t seen = atomicAdd(f.tickets + fc, 1);
                s_last = seen == (uint32_t)(ec - fc);
                if (s_last) f.tickets[fc] = 0;
                __threadfence();
            }
            __syncthreads();
            finish = s_last != 0;
            n_parts = ec - fc + 1;
        }
        if (finish) {
            for (int x = tid; x < rows * (D / 2); x += W * 32) {
                const int r = x / (D / 2), d = 2 * (x % (D / 2)), rr = jj.rt * kRows + r;
                const int head = jj.h * f.G + rr % f.G;
                float mm = -INFINITY, NN = -INFINITY, ll = 0.f;
                float2 v = make_float2(0.f, 0.f);
                auto src = [&](int k) -> const float * {
                    return inside ? at(k) : f.parts + ((size_t)(fc + k) * 2 + (k == 0 ? 1 : 0)) * PF;
                };
                auto get = [&](const float *p) { return inside ? *p : __ldcg(p); };
                const int k0 = inside ? i : 0, k1 = inside ? z : n_parts;
                for (int k = k0; k < k1; k++)
                    if (!inside || seg_job[k] >= 0) mm = fmaxf(mm, get(src(k) + R * PAD + r));
                const float ms = mm == -INFINITY ? 0.f : mm;
                for (int k = k0; k < k1; k++)
                    if (!inside || seg_job[k] >= 0)
                        NN = fmaxf(NN, get(src(k) + R * PAD + r) - ms + get(src(k) + R * PAD + 2 * R + r));
                for (int k = k0; k < k1; k++)
                    if (!inside || seg_job[k] >= 0) {
                        const float *ml = src(k) + R * PAD + r;
                        const float pm = get(ml), plv = get(ml + R), pN = get(ml + 2 * R);
                        const float2 *wp = reinterpret_cast<const float2 *>(src(k) + r * PAD + d);
                        const float2 w = inside ? *wp : __ldcg(wp);
                        const float c = pN == -INFINITY ? 0.f : ex2(pm - ms + pN - NN);
                        v.x += c * w.x, v.y += c * w.y;
                        ll += plv * (pm == -INFINITY ? 1.f : ex2(pm - ms));
                    }
                float den = ll, top = mm;
                if (a.sinks) {
                    const float sk = a.sinks[head] * kLog2e;
                    top = fmaxf(top, sk);
                    den = top == -INFINITY ? 0.f : (mm == -INFINITY ? ll : ll * ex2(mm - top)) + ex2(sk - top);
                }
                const float k = den == 0.f || NN == -INFINITY ? 0.f : ex2(NN - 15.f + (mm - top)) / den;
                *reinterpret_cast<__nv_bfloat162 *>(a.out + (long long)(row0 + rr / f.G) * a.o_stride + head * D + d) =
                    __floats2bfloat162_rn(v.x * k, v.y * k);
            }
        }
        __syncthreads();   // s_last is written again by the next job
        i = z;
    }
}

template <int D, int P, bool TOP>
cudaError_t few_launch(FewArgs f, int ctas, cudaStream_t st) {
    constexpr int W = Few<D, TOP>::kWarps;
    f.rows8 = TOP ? 16 : 8;
    const size_t fixed = (size_t)W * partial_floats(f.rows8, D) * 4 + (size_t)f.a.n_seqs * 12;
    f.stages = (int)std::min<size_t>(4, ((size_t)230000 - fixed) / ((size_t)W * Few<D, TOP>::kStage));
    const size_t smem = fixed + (size_t)f.stages * W * Few<D, TOP>::kStage;
    static PerDevice<bool> opted;
    cudaError_t e = smem_optin_once(moe_kv8_few_kernel<D, P, TOP>, opted);
    if (e != cudaSuccess) return e;
    return launch_pdl(moe_kv8_few_kernel<D, P, TOP>, dim3(ctas), dim3(W * 32), smem, st, f);
}
template <int D, int P>
cudaError_t few_rows(const FewArgs &f, bool top, int ctas, cudaStream_t st) {
    return top ? few_launch<D, P, true>(f, ctas, st) : few_launch<D, P, false>(f, ctas, st);
}
template <int D>
cudaError_t few_page(const FewArgs &f, bool top, int ctas, cudaStream_t st) {
    return f.a.c.P == 16 ? few_rows<D, 16>(f, top, ctas, st) : f.a.c.P == 32 ? few_rows<D, 32>(f, top, ctas, st)
                                                                             : few_rows<D, 64>(f, top, ctas, st);
}

cudaError_t sm_count(int *n) {
    static PerDevice<int> sms;
    int dev = 0;
    cudaError_t e = current_device_slot(&dev);
    if (e == cudaSuccess && !sms.v[dev]) e = cudaDeviceGetAttribute(&sms.v[dev], cudaDevAttrMultiProcessorCount, dev);
    *n = sms.v[dev];
    return e;
}

}  // namespace

size_t kv8_workspace_bytes(int D) { return kKv8ClearBytes + (size_t)kMaxCtas * 2 * partial_floats(kRows, D) * 4; }

cudaError_t launch_kv8_attend(const Kv8Attend &a, unsigned char *ws, cudaStream_t st) {
    const int G = a.QH / a.c.KVH;
    if (a.max_new * G <= 64) {
        FewArgs f{};
        f.a = a, f.G = G;
        f.status = reinterpret_cast<int32_t *>(ws);
        f.tickets = reinterpret_cast<uint32_t *>(ws + 64);
        f.parts = reinterpret_cast<float *>(ws + kKv8ClearBytes);
        int ctas = 0;
        const cudaError_t e = sm_count(&ctas);
        if (e != cudaSuccess) return e;
        ctas = std::min(ctas, kMaxCtas);
        const bool top = a.max_new * G > 8;
        return a.c.D == 64 ? few_page<64>(f, top, ctas, st) : few_page<128>(f, top, ctas, st);
    }
    const dim3 grid(a.QH, a.max_new, a.n_seqs);
    if (a.c.D == 64) return launch_pdl(moe_kv8_attend_kernel<64>, grid, dim3(128), 0, st, a);
    return launch_pdl(moe_kv8_attend_kernel<128>, grid, dim3(128), 0, st, a);
}
