// moe_kv8_attend.cu -- attention over the 8-bit paged key/value cache for a few
// new tokens a sequence (decode steps), and the choice between this kernel and
// that for prompts (moe_kv8_prompt.cu).
#include "moe_kv_few.cuh"

#include <algorithm>

namespace {

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
// 11 bits, where a sum takes fp32 weights in the plain form: one product instead
// of two, and results still 1.6e-3 from those in 64 bits (relative, over an
// output), as is a form in fp32 that is rounded to bf16 at its end.
// q is scaled per row by a power of two into fp16's range: exact for a bf16
// row's values down to 2^-28 of its largest.
constexpr int kRows = 16;   // rows of a unit

// Measured: 16 x 4096 tokens of 8 heads of 64 (67 MB) 23.8 us: lengths and
// table 1.4, the first pages 2.8, units 8.0 (HBM's rate), joins 4.7, the launch
// the rest; 96 ragged sequences of up to 12 K, 4 heads of 128 (612 MB), 110 us:
// 0.82 of a copy's rate; one sequence of 131 tokens 7.3 us.
// Warps, and units in each one's ring.  What bounds the kernel is latency at
// the instructions of a unit, so as many warps as registers and the 227 KB of
// shared memory allow come before a deeper ring: a warp's own copies are in
// flight while the others compute (8 rows of D = 64, 16 x 1024 tokens: 16
// warps with one unit each 17.3 us, 11 with two 23.4; 32 x 16384 tokens, the
// only side where the ring gained: 101 and 96).
template <int D, bool TOP>
struct Few {
    static constexpr int kWarps = D == 64 ? (TOP ? 10 : 16) : (TOP ? 8 : 10);
    static constexpr int kStages = D == 64 ? (TOP ? 2 : 1) : 1;
    static constexpr int kStage = 2 * kTile * D;   // bytes of one unit: keys, values
    static constexpr int kPad = D + 8;             // floats of a partial's row: 64-bit stores on distinct banks
};
// A partial: acc [rows][D + 8], then m, l, N [rows] each.
__host__ __device__ constexpr int partial_floats(int rows, int D) { return rows * (D + 8 + 3); }

template <int D, bool TOP>
__host__ __device__ constexpr int few_smem() {   // without the sequences
    return Few<D, TOP>::kWarps * (Few<D, TOP>::kStages * Few<D, TOP>::kStage + partial_floats(TOP ? 16 : 8, D) * 4);
}

struct FewArgs {
    Kv8Attend a;
    int G;                     // query heads per kv head
    int32_t *status;           // [2]
    uint32_t *tickets;         // [kMaxCtas], zero between calls
    float *parts;              // [kMaxCtas][2][partial_floats]
    int *seqs;                 // [3][n_seqs], or null: in shared memory
};

__device__ __forceinline__ float quad_max(float v) {
    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
    return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
}
__device__ __forceinline__ float quad_sum(float v) {
    v += __shfl_xor_sync(0xffffffffu, v, 1);
    return v + __shfl_xor_sync(0xffffffffu, v, 2);
}

// What turns a row's accumulator into its output (sink: the head's logit in
// units of log2, -inf without one): two factors, as their product may be below
// 2^-126 where the output is not.
__device__ __forceinline__ float2 row_factor(float m, float l, float N, float sink) {
    const float top = fmaxf(m, sink);
    const float den = top == -INFINITY ? l : (m == -INFINITY ? l : l * ex2(m - top)) + ex2(sink - top);
    const float half = ex2(0.5f * (N - 15.f + (m - top)));
    return den == 0.f || N == -INFINITY ? make_float2(0.f, 0.f) : make_float2(half, half / den);   // an empty row: 0; NaN stays NaN
}

// One warp's place in its units: where the next unit's pages come from.
template <int D, int P, bool TOP>
__global__ void __launch_bounds__(Few<D, TOP>::kWarps * 32, 1) moe_kv8_few_kernel(const __grid_constant__ FewArgs f) {
    constexpr int W = Few<D, TOP>::kWarps, NP = kTile / P, HP = P == 16 ? 2 : 1, NC = D / 16, ST = Few<D, TOP>::kStage, PAD = Few<D, TOP>::kPad;
    constexpr int S = Few<D, TOP>::kStages, R = TOP ? 16 : 8, PF = partial_floats(R, D);
    static_assert(PF * 4 <= S * ST && few_smem<D, TOP>() + kSmemSeqs * 12 <= 230000, "shared memory");
    extern __shared__ __align__(128) unsigned char smem_raw[];
    __shared__ __align__(8) uint64_t bars[W][S];
    __shared__ uint32_t meta[W][S][NP];           // per stage and page: key exponent byte, value's, 1 if it is there
    __shared__ int scan[W];
    __shared__ Seg segs[2 * W];                   // head and tail of each warp
    __shared__ int list[2 * W], group_at[2 * W + 1], group_seg[2 * W], shared_seg[2], s_first[2], s_count[2];
    const Kv8Attend &a = f.a;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t4 = lane & 3;
    unsigned char *ring = smem_raw + (size_t)warp * S * ST;
    float *part = reinterpret_cast<float *>(smem_raw + (size_t)W * S * ST);   // [W] head partials; tails go over the rings
    // per sequence: units of those before it (a kv head), index of its first unit in it, tokens that can be seen; of
    // many sequences in the workspace, where every CTA writes the same
    int *seq_s = reinterpret_cast<int *>(part + (size_t)W * PF);
    auto seq = [&](int what, int b) { return f.seqs ? f.seqs[what * a.n_seqs + b] : seq_s[what * a.n_seqs + b]; };
    if (lane == 0)
        for (int s = 0; s < S; s++) asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(smem_u32(&bars[warp][s])));
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");

    // every sequence's units: contiguous shares of sequences per thread, one block scan
    const int per_thr = (a.n_seqs + W * 32 - 1) / (W * 32), sb0 = min(tid * per_thr, a.n_seqs), sb1 = min(sb0 + per_thr, a.n_seqs);
    auto seq_units = [&](int b, int &first, int &seen) {
        int row0, n, pos0;
        kv8_rows(a, b, row0, n, pos0);
        seen = (int)max(0ll, min((long long)a.lens[b], (long long)a.width * P));
        first = kv8_first(pos0, a.window) / kTile;
        return n > 0 ? max(1, (seen + kTile - 1) / kTile - first) * ((n * f.G + kRows - 1) / kRows) : 0;
    };
    int mine = 0, first, seen_b;
    for (int b = sb0; b < sb1; b++) mine += seq_units(b, first, seen_b);
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
    int *seq_w = f.seqs ? f.seqs : seq_s;
    for (int b = sb0; b < sb1; b++) {   // only these final values are ever written
        const int cnt = per_thr == 1 ? mine : seq_units(b, first, seen_b);
        seq_w[b] = base, seq_w[a.n_seqs + b] = first, seq_w[2 * a.n_seqs + b] = seen_b;
        base += cnt;
    }
    if (tid < 2 * W) segs[tid].u0 = -1;
    if (tid < 2) shared_seg[tid] = -1;
    __syncthreads();
    const int units = total * a.c.KVH, ctas = min((int)gridDim.x, (units + 3) / 4);
    if ((int)blockIdx.x >= ctas) return;
    // the job of unit u (0 <= u < units)
    auto job_of = [&](int u) {
        Job j;
        int lo = 0, hi = a.n_seqs;   // the last sequence with KVH * units before it <= u
        const int uk = (unsigned)u / (unsigned)a.c.KVH;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (seq(0, mid) <= uk) lo = mid;
            else hi = mid;
        }
        const int before = seq(0, lo) * a.c.KVH;
        j.b = lo;
        j.nt = max(1, (seq(2, lo) + kTile - 1) / kTile - seq(1, lo));
        const unsigned tile = (unsigned)(u - before) / (unsigned)j.nt;
        if (TOP) {
            const unsigned n_rt = ((lo + 1 < a.n_seqs ? seq(0, lo + 1) : total) - seq(0, lo)) / j.nt;
            j.h = tile / n_rt;
            j.rt = tile % n_rt;
        } else {
            j.h = tile, j.rt = 0;    // one row tile: at most 8 rows
        }
        j.u0 = before + tile * j.nt;
        return j;
    };
    // The CTA's share: the even cuts, each moved down to its job's first unit
    // where the job is at most 8 units long (a job that one CTA can take at
    // once is not worth joining across two).
    int cut = (int)((long long)units * (blockIdx.x + (lane & 1)) / ctas);
    if (cut > 0 && cut < units) {
        const Job j = job_of(cut);
        if (j.nt <= 8) cut = j.u0;
    }
    const int c0 = __shfl_sync(0xffffffffu, cut, 0), c1 = __shfl_sync(0xffffffffu, cut, 1);
    const int u0 = c0 + (c1 - c0) * warp / W, u1 = c0 + (c1 - c0) * (warp + 1) / W;   // c1 - c0 < 2^31 / 16 (host)

    // the issuing side: place of the next unit to copy, its pages read one unit ahead
    Job ij = {0, 0, 0, 1, 0}, ji = ij;   // of unit iu, and of the one issued last
    int iu = u0;
    int pg = -1;
    auto fetch_page = [&]() {   // lane p < NP: page of the unit iu
        pg = -1;
        if (iu < u1 && lane < NP) {
            const int tile = seq(1, ij.b) + iu - ij.u0;
            const int t0 = tile * kTile + lane * P;
            if (t0 < seq(2, ij.b)) pg = __ldg(a.table + (size_t)ij.b * a.width + t0 / P);
        }
    };
    uint32_t pend_k = 0, pend_v = 0, pend_there = 0;   // put together only when they are stored: nothing waits for them here
    int pend_stage = -1;
    auto flush = [&]() {
        if (pend_stage >= 0 && lane < NP) meta[warp][pend_stage][lane] = pend_k | pend_v << 8 | pend_there;
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
        pend_k = pend_v = pend_there = 0;
        if (ok) {
            const size_t ph = (size_t)pg * a.c.KVH + ij.h;
            const uint32_t dst = smem_u32(ring + stage * ST) + lane * (P * D);
            bulk_copy(dst, a.c.k + ph * (P * D), P * D, bar);
            bulk_copy(dst + kTile * D, a.c.v + ph * (P * D), P * D, bar);
            pend_k = __ldg(a.c.ks + ph), pend_v = __ldg(a.c.vs + ph), pend_there = 1u << 16;
        }
        pend_stage = stage;
        ji = ij;
        iu++;
        if (iu < u1 && iu == ij.u0 + ij.nt) ij = job_of(iu);
        fetch_page();
    };
    if (u0 < u1) {
        ij = job_of(u0);
        fetch_page();
    }
    auto fill = [&](int u) {
#pragma unroll 1
        while (iu < u1 && iu < u + S) issue((iu - u0) % S);
    };
    bool fine = true;

    // the computing side
    // values: up to 8 rows transposed (16 dims x 8 rows a tile: dims g, g + 8 of rows 2 t4, 2 t4 + 1), else 16
    // rows x 8 dims (rows g, g + 8, dims 2 t4, 2 t4 + 1)
    constexpr int NA = TOP ? D / 8 : D / 16;
    float acc[NA][4], m[2], l[2], N[2];
    const float sc = a.scale * kLog2e;
    int up[2] = {0, 0};   // the rows' queries carry 2^up
    uint32_t qf[NC][4];
    float sink[2] = {-INFINITY, -INFINITY};
    Job j = ij;
    bool begun = false;
    int pos[2] = {0, 0}, pmin = 0, pmax = 0;
    int seg0 = u0;           // first unit of the running segment
    static_assert(S <= 2, "the job of a unit that is issued and not begun is ji");
    for (int u = u0; u < u1 && fine; u++) {
        const int i = u - u0, stage = i % S;
        // a new job: its rows' queries, on their way while the unit's pages are
        // (with dims of 128 after the pages: registers)
        const bool fresh = !begun;
        uint2 w[TOP ? 2 : 1][NC];
        if (fresh) j = iu > u ? ji : ij;
        if (D == 128) fill(u);
        if (fresh) {
            begun = true, seg0 = u;
            int row0, n, pos0;
            kv8_rows(a, j.b, row0, n, pos0);
            pmin = pos0 + j.rt * kRows / f.G;
            pmax = pos0 + min(n * f.G - 1, j.rt * kRows + kRows - 1) / f.G;
#pragma unroll
            for (int r = 0; r < (TOP ? 2 : 1); r++) {
                const int rr = j.rt * kRows + g + 8 * r, i2 = rr / f.G, head = j.h * f.G + rr - i2 * f.G;
                const bool on = rr < n * f.G;
                pos[r] = on ? pos0 + i2 : -1;
                const uint16_t *q = a.q + (long long)(row0 + i2) * a.q_stride + head * D + 4 * t4;
#pragma unroll
                for (int c = 0; c < NC; c++) w[r][c] = on ? __ldg(reinterpret_cast<const uint2 *>(q + 16 * c)) : make_uint2(0, 0);
                sink[r] = on && a.sinks ? a.sinks[head] * kLog2e : -INFINITY;
            }
        }
        if (D == 64) fill(u);
        if (fresh) {
            // each row scaled: its largest magnitude to [2^14, 2^15) (exponent field e means 2^(e - 127))
#pragma unroll
            for (int r = 0; r < (TOP ? 2 : 1); r++) {
                uint32_t am = 0;
#pragma unroll
                for (int c = 0; c < NC; c++)
                    am = max(am, max(max(w[r][c].x & 0x7FFFu, (w[r][c].x >> 16) & 0x7FFFu), max(w[r][c].y & 0x7FFFu, (w[r][c].y >> 16) & 0x7FFFu)));
                am = max(am, __shfl_xor_sync(0xffffffffu, am, 1));
                am = max(am, __shfl_xor_sync(0xffffffffu, am, 2));
                up[r] = min(141 - (int)(am >> 7), 127);
                const float mul = pow2i(up[r]);
                m[r] = -INFINITY, l[r] = 0.f, N[r] = -INFINITY;
#pragma unroll
                for (int c = 0; c < NC; c++) {
                    qf[c][r] = pack_f16(__uint_as_float(w[r][c].x << 16) * mul, __uint_as_float(w[r][c].x & 0xFFFF0000u) * mul);
                    qf[c][2 + r] = pack_f16(__uint_as_float(w[r][c].y << 16) * mul, __uint_as_float(w[r][c].y & 0xFFFF0000u) * mul);
                    if (!TOP) qf[c][1] = qf[c][3] = 0u;
                }
            }
#pragma unroll
            for (int d = 0; d < NA; d++) acc[d][0] = acc[d][1] = acc[d][2] = acc[d][3] = 0.f;
        }
        if (pend_stage == stage) flush();
        __syncwarp();
        fine = bar_wait(smem_u32(&bars[warp][stage]), (uint32_t)(i / S) & 1, f.status, 90);
        fine = __all_sync(0xffffffffu, fine);
        if (!fine) break;
        const int seen = seq(2, j.b), u_at = (seq(1, j.b) + u - j.u0) * kTile;
        // 32 tokens at a time
#pragma unroll 1
        for (int hf = 0; hf < 2; hf++) {
            const int t0 = u_at + 32 * hf;
            uint32_t mt[HP];
            bool whole = t0 + 32 <= seen && t0 + 31 <= pmin && (a.window == 0 || t0 > pmax - a.window);
#pragma unroll
            for (int p = 0; p < HP; p++) {
                mt[p] = meta[warp][stage][P == 64 ? 0 : hf * HP + p];
                whole = whole && (mt[p] >> 16);
            }
            // where this half's tokens begin in the unit: pages hold keys [D / 16][P][16], values [P / 16][D][16]
            const uint32_t kb = smem_u32(ring + stage * ST) + (P == 64 ? hf * 512 : hf * 32 * D);
            const uint32_t vb = smem_u32(ring + stage * ST) + kTile * D + hf * 32 * D;
            // scores: 4 token octets x (rows g: c0, c1; rows g + 8: c2, c3)
            float s[4][4];
#pragma unroll
            for (int n = 0; n < 4; n++) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
#pragma unroll
            for (int c = 0; c < NC; c++) {
                uint32_t w[4];
                ldsm4(w, kb + (lane / P) * (P * D) + c * (P * 16) + (lane % P) * 16);
#pragma unroll
                for (int n = 0; n < 4; n++) {
                    uint32_t b0, b1;
                    e4m3x4_to_f16(w[n], b0, b1);
                    mma_f16(s[n], qf[c], b0, b1);
                }
            }
            // byte 2 (n & 1) + e of a thread's value word is token 8 (n & 1) + 2 t4 + e of its 16
            auto sees = [&](int t, int p) { return t <= p && (a.window == 0 || t > p - a.window); };
            auto there = [&](int n, int t) { return t < seen && (mt[n * HP / 4] >> 16); };
            bool odd = false;
            if (!whole) {
                uint32_t keep[2] = {0, 0};   // value bytes that some row sees
#pragma unroll
                for (int n = 0; n < 4; n++)
#pragma unroll
                    for (int e = 0; e < 2; e++) {
                        const int t = t0 + 8 * n + 2 * t4 + e;
#pragma unroll
                        for (int r = 0; r < (TOP ? 2 : 1); r++)
                            if (!(there(n, t) && sees(t, pos[r]))) s[n][2 * r + e] = -INFINITY;
                        if (there(n, t) && t <= pmax && t >= kv8_first(pmin, a.window)) keep[n / 2] |= 0xFFu << (16 * (n & 1) + 8 * e);
                    }
                // values that no row sees to zero: nothing they hold may meet a weight of 0
                uint32_t nan = 0;
                for (int x = lane; x < 8 * D; x += 32) {   // words of [2][D][16]: word x & 3 is that of the lanes t4 = x & 3
                    const uint32_t at = vb + 4 * x, k = x >= 4 * D ? keep[1] : keep[0];
                    uint32_t w;
                    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w) : "r"(at) : "memory");
                    w &= k;
                    nan |= ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
                    asm volatile("st.shared.b32 [%0], %1;" ::"r"(at), "r"(w) : "memory");
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // before the next copy into the stage
                __syncwarp();                                                  // and before other lanes read the values
                // a NaN that only some rows see: those rows' values apart (below)
                odd = __any_sync(0xffffffffu, nan != 0 && pmin != pmax);
            }
            bool moved = false;
            float corr[2] = {1.f, 1.f};
#pragma unroll
            for (int r = 0; r < (TOP ? 2 : 1); r++) {
                float mx = -INFINITY, pmx[HP], ks[HP];   // ks > 0: a hidden token's -inf stays
#pragma unroll
                for (int p = 0; p < HP; p++) {
                    ks[p] = fmaxf(pow2i((int)(mt[p] & 255u) - 127 - up[r]) * sc, 1e-37f);
                    float pm = -INFINITY;
#pragma unroll
                    for (int n = p * (4 / HP); n < (p + 1) * (4 / HP); n++) pm = fmaxf(pm, fmaxf(s[n][2 * r], s[n][2 * r + 1]));
                    pmx[p] = pm * ks[p], mx = fmaxf(mx, pmx[p]);
                }
                mx = quad_max(mx);
                const float mn = fmaxf(m[r], mx), ms = mn == -INFINITY ? 0.f : mn;
                const float was = N[r] + (m[r] - ms);    // the old reference, over the new m
                float mv = -INFINITY;                    // over the new m, as scores may be too large for an exponent beside them
#pragma unroll
                for (int p = 0; p < HP; p++) mv = fmaxf(mv, pmx[p] - ms + (float)((int)((mt[p] >> 8) & 255u) - 127));
                if (HP > 1) mv = quad_max(mv);
                else mv = mx - ms + (float)((int)((mt[0] >> 8) & 255u) - 127);
                const float Nn = fmaxf(was, mv), Ns = Nn == -INFINITY ? 0.f : Nn;
                l[r] *= ex2(m[r] - ms);
                corr[r] = ex2(was - Ns);
                moved |= Nn != was;
                m[r] = mn, N[r] = Nn;
                float sum = 0.f;
#pragma unroll
                for (int n = 0; n < 4; n++) {
                    const int p = n * HP / 4;
                    const float fac = ex2(fminf((float)((int)((mt[p] >> 8) & 255u) - 112) - Ns, 126.f));
#pragma unroll
                    for (int e = 0; e < 2; e++) {
                        // the product rounded as the maximum was: a score past 2^24 is off by more than 1 otherwise
                        const float w = ex2(__fsub_rn(__fmul_rn(s[n][2 * r + e], ks[p]), ms));
                        sum += w;
                        s[n][2 * r + e] = w * fac;
                    }
                }
                l[r] += sum;
            }
            if (__any_sync(0xffffffffu, moved)) {
                const float c0 = TOP ? corr[0] : __shfl_sync(0xffffffffu, corr[0], 8 * t4);
                const float c1 = TOP ? c0 : __shfl_sync(0xffffffffu, corr[0], 8 * t4 + 4);
#pragma unroll
                for (int d = 0; d < NA; d++) {
                    acc[d][0] *= c0, acc[d][1] *= c1;
                    acc[d][2] *= TOP ? corr[1] : c0, acc[d][3] *= TOP ? corr[1] : c1;
                }
            }
            uint32_t pf[2][TOP ? 4 : 2];   // weights: rows as an A fragment, or as a B fragment
#pragma unroll
            for (int kk = 0; kk < 2; kk++)
#pragma unroll
                for (int x = 0; x < (TOP ? 4 : 2); x++) {
                    const float *sp = TOP ? s[2 * kk + (x >> 1)] + 2 * (x & 1) : s[2 * kk + x];
                    pf[kk][x] = pack_f16(sp[0], sp[1]);
                }
            // value words wl, wh of dims g, g + 8 of a 16-dim tile
            auto times = [&](int kk, uint32_t wl, uint32_t wh, float (&lo)[4], float (&hi)[4]) {
                uint32_t v[4];
                e4m3x4_to_f16(wl, v[0], v[2]);
                e4m3x4_to_f16(wh, v[1], v[3]);
                if constexpr (TOP) {
                    mma_f16(lo, pf[kk], v[0], v[2]);
                    mma_f16(hi, pf[kk], v[1], v[3]);
                } else {
                    mma_f16(lo, v, pf[kk][0], pf[kk][1]);
                }
            };
            if (!odd) {
#pragma unroll
                for (int kk = 0; kk < 2; kk++)
#pragma unroll
                    for (int q = 0; q < D / 32; q++) {
                        uint32_t w[4];
                        ldsm4(w, vb + kk * (16 * D) + (32 * q + lane) * 16);
#pragma unroll
                        for (int n = 0; n < 2; n++) {
                            constexpr int F = TOP ? 2 : 1;
                            times(kk, w[2 * n], w[2 * n + 1], acc[F * (2 * q + n)], acc[F * (2 * q + n) + F - 1]);
                        }
                    }
            } else {
                // one position's rows at a time, with only the values that they see
#pragma unroll 1
                for (int p = pmin; p <= pmax; p++) {
                    uint32_t keep[2] = {0, 0};
#pragma unroll
                    for (int n = 0; n < 4; n++)
#pragma unroll
                        for (int e = 0; e < 2; e++)
                            if (sees(t0 + 8 * n + 2 * t4 + e, p)) keep[n / 2] |= 0xFFu << (16 * (n & 1) + 8 * e);
                    // rows of the accumulator's columns (transposed: 2 t4, 2 t4 + 1; else g, g + 8)
                    const int p0 = TOP ? pos[0] : __shfl_sync(0xffffffffu, pos[0], 8 * t4);
                    const int p1 = TOP ? pos[1] : __shfl_sync(0xffffffffu, pos[0], 8 * t4 + 4);
#pragma unroll
                    for (int q = 0; q < D / 16; q++) {
                        float x[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
                        for (int kk = 0; kk < 2; kk++) {
                            uint32_t w[2];
#pragma unroll
                            for (int y = 0; y < 2; y++) {
                                asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w[y]) : "r"(vb + kk * (16 * D) + (16 * q + 8 * y + g) * 16 + 4 * t4) : "memory");
                                w[y] &= keep[kk];
                            }
                            times(kk, w[0], w[1], x[0], x[1]);
                        }
#pragma unroll
                        for (int y = 0; y < (TOP ? 2 : 1); y++)
#pragma unroll
                            for (int e = 0; e < 4; e++)
                                if ((TOP ? (e >> 1 ? p1 : p0) : (e & 1 ? p1 : p0)) == p) acc[(TOP ? 2 : 1) * q + y][e] += x[y][e];
                    }
                }
            }
        }
        __syncwarp();   // the stage is read: the next iteration fills it
        if (u + 1 == j.u0 + j.nt || u + 1 == u1) {
            begun = false;
            const bool begins = seg0 == j.u0, ends = u + 1 == j.u0 + j.nt;
            if (begins && ends) {
                // the whole job was this warp's
                int row0, n, pos0;
                kv8_rows(a, j.b, row0, n, pos0);
#pragma unroll
                for (int r = 0; r < 2; r++) {
                    float2 k = row_factor(m[TOP ? r : 0], quad_sum(l[TOP ? r : 0]), N[TOP ? r : 0], sink[TOP ? r : 0]);
                    if (!TOP) k = make_float2(__shfl_sync(0xffffffffu, k.x, 8 * t4 + 4 * r), __shfl_sync(0xffffffffu, k.y, 8 * t4 + 4 * r));
                    const int rr = j.rt * kRows + (TOP ? g + 8 * r : 2 * t4 + r);
                    if (rr >= n * f.G) continue;
                    __nv_bfloat16 *o = reinterpret_cast<__nv_bfloat16 *>(a.out) + (long long)(row0 + rr / f.G) * a.o_stride +
                                       (j.h * f.G + rr % f.G) * D + (TOP ? 2 * t4 : g);
#pragma unroll
                    for (int d = 0; d < NA; d++) {
                        if (TOP) {
                            *reinterpret_cast<__nv_bfloat162 *>(o + 8 * d) = __floats2bfloat162_rn(acc[d][2 * r] * k.x * k.y, acc[d][2 * r + 1] * k.x * k.y);
                        } else {
                            o[16 * d] = __float2bfloat16_rn(acc[d][r] * k.x * k.y);
                            o[16 * d + 8] = __float2bfloat16_rn(acc[d][2 + r] * k.x * k.y);
                        }
                    }
                }
            } else {
                // a head of more to come goes to its own place, the last segment over
                // the ring, whose copies have all landed and been read
                const bool last = u + 1 == u1;
                float *to = last ? reinterpret_cast<float *>(ring) : part + (size_t)warp * PF;
#pragma unroll
                for (int r = 0; r < 2; r++) {
                    float *row = to + (TOP ? g + 8 * r : 2 * t4 + r) * PAD + (TOP ? 2 * t4 : g);
#pragma unroll
                    for (int d = 0; d < NA; d++) {
                        if (TOP) *reinterpret_cast<float2 *>(row + 8 * d) = make_float2(acc[d][2 * r], acc[d][2 * r + 1]);
                        else row[16 * d] = acc[d][r], row[16 * d + 8] = acc[d][2 + r];
                    }
                }
#pragma unroll
                for (int r = 0; r < (TOP ? 2 : 1); r++) {
                    const float ls = quad_sum(l[r]);
                    float *ml = to + R * PAD + g + 8 * r;
                    if (t4 == 0) ml[0] = m[r], ml[R] = ls, ml[2 * R] = N[r];
                }
                if (lane == 0) segs[2 * warp + last] = {j.u0, j.nt, j.b, j.h, j.rt};
            }
        }
    }
    if (!fine)   // copies may still be in flight: each stage's last phase, with a limit
        for (int s = 0; s < S; s++)
            if (s < iu - u0) bar_wait(smem_u32(&bars[warp][s]), (uint32_t)((iu - u0 - 1 - s) / S) & 1, f.status, 91);
    __syncthreads();

    // Joining: the CTA's segments in order, those of one job a group (they are
    // neighbours); then, of the jobs that other CTAs share (at most the first
    // and the last), those whose other partials are all there.  Either time all
    // groups at once: the partials' m, l and N side by side in shared memory,
    // then a thread for each group, row and pair of dims (16 x 4096 tokens: 23.7
    // us, 26.3 with the groups one after the other).
    auto scal = [&](int k) {   // 3 R floats, behind the tails in the rings
        return reinterpret_cast<float *>(smem_raw + (size_t)(k % W) * S * ST) + PF + k / W * (3 * R);
    };
    static_assert((PF + (kMaxCtas + W) / W * 3 * R) * 4 <= S * ST, "room for the scalars of a join: kMaxCtas + 1 partials at most");
    auto scalars = [&](int k, const float *from) {
        for (int y = lane; y < 3 * R; y += 32) scal(k)[y] = *(volatile const float *)(from + R * PAD + y);
    };
    // partials k0 .. k0 + n - 1 (at(k)) of segment sg's job: row r, dims d, d + 1
    auto join = [&](const Seg &sg, int k0, int n, auto at, bool done, int r, int d) {
        int row0, nr, pos0;
        kv8_rows(a, sg.b, row0, nr, pos0);
        if (r >= min(kRows, nr * f.G - sg.rt * kRows)) return;
        float mm = -INFINITY, NN = -INFINITY, ll = 0.f;
#pragma unroll 4
        for (int k = k0; k < k0 + n; k++) mm = fmaxf(mm, scal(k)[r]);
        const float ms = mm == -INFINITY ? 0.f : mm;
#pragma unroll 4
        for (int k = k0; k < k0 + n; k++) NN = fmaxf(NN, scal(k)[r] - ms + scal(k)[2 * R + r]);
        const float Ns = NN == -INFINITY ? 0.f : NN;
        float2 v = make_float2(0.f, 0.f);
#pragma unroll 8
        for (int k = k0; k < k0 + n; k++) {
            const float km = scal(k)[r], kl = scal(k)[R + r], kn = scal(k)[2 * R + r];
            const float c = ex2(km - ms + kn - Ns);   // no tokens: 2^-inf
            volatile const float *p = at(k) + r * PAD + d;
            v.x = fmaf(c, p[0], v.x), v.y = fmaf(c, p[1], v.y);
            ll += kl * (km == -INFINITY ? 1.f : ex2(km - ms));   // the l of NaN scores has no maximum
        }
        if (done) {
            const int rr = sg.rt * kRows + r, i2 = rr / f.G, head = sg.h * f.G + rr - i2 * f.G;
            const float2 k = row_factor(mm, ll, NN, a.sinks ? a.sinks[head] * kLog2e : -INFINITY);
            *reinterpret_cast<__nv_bfloat162 *>(a.out + (long long)(row0 + i2) * a.o_stride + head * D + d) =
                __floats2bfloat162_rn(v.x * k.x * k.y, v.y * k.x * k.y);
        } else {
            float *mine_p = f.parts + ((size_t)blockIdx.x * 2 + (sg.u0 >= c0 ? 1 : 0)) * PF;
            *reinterpret_cast<float2 *>(mine_p + r * PAD + d) = v;
            if (d == 0) mine_p[R * PAD + r] = mm, mine_p[R * PAD + R + r] = ll, mine_p[R * PAD + 2 * R + r] = NN;
        }
    };
    constexpr int kCell = R * (D / 2);   // threads of a group
    const int my_seg = lane < 2 * W ? segs[lane].u0 : -1;
    const unsigned valid = __ballot_sync(0xffffffffu, my_seg >= 0), lower = valid & ((1u << lane) - 1);
    const int before = __shfl_sync(0xffffffffu, my_seg, lower ? 31 - __clz(lower) : 0);
    const bool leads = my_seg >= 0 && (!lower || before != my_seg);
    const unsigned leaders = __ballot_sync(0xffffffffu, leads);
    const int groups = __popc(leaders), partials = __popc(valid);
    auto whole_job = [&](const Seg &sg) { return sg.u0 >= c0 && sg.u0 + sg.nt <= c1; };
    // every warp writes the same
    if (my_seg >= 0) list[__popc(lower)] = lane;
    if (leads) {
        const int gi = __popc(leaders & ((1u << lane) - 1));
        group_at[gi] = __popc(lower), group_seg[gi] = lane;
        if (!whole_job(segs[lane])) shared_seg[my_seg >= c0 ? 1 : 0] = lane;
    }
    if (lane == 0) group_at[groups] = partials;
    __syncwarp();
    auto here = [&](int k) -> const float * {
        const int x = list[k];
        return x & 1 ? reinterpret_cast<const float *>(smem_raw + (size_t)(x >> 1) * S * ST) : part + (size_t)(x >> 1) * PF;
    };
    for (int k = warp; k < partials; k += W) scalars(k, here(k));
    __syncthreads();
    for (int x = tid; x < groups * kCell; x += W * 32) {
        const int gi = x / kCell, k0 = group_at[gi];
        const Seg sg = segs[group_seg[gi]];
        join(sg, k0, group_at[gi + 1] - k0, here, whole_job(sg), x % kCell / (D / 2), 2 * (x % (D / 2)));
    }
    if (shared_seg[0] < 0 && shared_seg[1] < 0) return;   // the same for the whole CTA

    __threadfence();
    __syncthreads();
    if (tid < 2) {
        s_count[tid] = 0;
        if (shared_seg[tid] >= 0) {
            // the CTAs that share the job, by the even cuts (no cut inside it was moved)
            const Seg x = segs[shared_seg[tid]];
            const int c_first = (int)(((long long)(x.u0 + 1) * ctas - 1) / units), c_last = (int)(((long long)(x.u0 + x.nt) * ctas - 1) / units);
            if (atomicAdd(f.tickets + c_first, 1) == (uint32_t)(c_last - c_first)) {
                f.tickets[c_first] = 0;   // as the next call finds it
                s_first[tid] = c_first, s_count[tid] = c_last - c_first + 1;
            }
        }
        __threadfence();
    }
    __syncthreads();
    const int n0 = s_count[0], n1 = s_count[1];
    auto there_at = [&](int k) -> const float * {
        const int i = k >= n0, kk = k - (i ? n0 : 0);
        return f.parts + ((size_t)(s_first[i] + kk) * 2 + (kk == 0 ? 1 : 0)) * PF;
    };
    for (int k = warp; k < n0 + n1; k += W) scalars(k, there_at(k));
    __syncthreads();
    for (int x = tid; x < 2 * kCell; x += W * 32) {
        const int i = x / kCell, n = i ? n1 : n0;
        if (n) join(segs[shared_seg[i]], i ? n0 : 0, n, there_at, true, x % kCell / (D / 2), 2 * (x % (D / 2)));
    }
}

constexpr size_t kPartOffset = kKv8ClearBytes + (size_t)kKv8MaxSeqs * 12;

template <int D, int P, bool TOP>
cudaError_t few_launch(FewArgs f, int ctas, cudaStream_t st) {
    constexpr int W = Few<D, TOP>::kWarps;
    if (f.a.n_seqs <= kSmemSeqs) f.seqs = nullptr;
    const size_t smem = few_smem<D, TOP>() + (f.seqs ? 0 : (size_t)f.a.n_seqs * 12);
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

}  // namespace

size_t kv8_workspace_bytes(int D) { return kPartOffset + (size_t)kMaxCtas * 2 * partial_floats(kRows, D) * 4; }

cudaError_t launch_kv8_attend(const Kv8Attend &a, unsigned char *ws, cudaStream_t st) {
    // Up to 64 rows of a kv head the streaming kernel: its work grows by the row
    // tile of 16, that of the kernel for prompts, 256 rows a CTA, does not.  us at
    // 32, 64, 128 rows, 8 kv heads of 64, streaming and prompts: 32 sequences of
    // 4096 tokens 76 and 113, 133 and 110, 243 and 111; 8 of them 33 and 57, 46
    // and 55, 75 and 56.  Not so where the prompts' CTAs are few, as they walk all
    // keys: one sequence of 32 K tokens 36 and 415, 50 and 402, 73 and 403.
    const int G = a.QH / a.c.KVH;
    if (a.max_new * G <= 64) {
        FewArgs f{};
        f.a = a, f.G = G;
        f.status = reinterpret_cast<int32_t *>(ws);
        f.tickets = reinterpret_cast<uint32_t *>(ws + 64);
        f.seqs = reinterpret_cast<int *>(ws + kKv8ClearBytes);
        f.parts = reinterpret_cast<float *>(ws + kPartOffset);
        int ctas = 0;
        const cudaError_t e = sm_count(&ctas);
        if (e != cudaSuccess) return e;
        ctas = std::min(ctas, kMaxCtas);
        const bool top = a.max_new * G > 8;
        return a.c.D == 64 ? few_page<64>(f, top, ctas, st) : few_page<128>(f, top, ctas, st);
    }
    return launch_kv8_prompt(a, reinterpret_cast<int32_t *>(ws), st);
}
