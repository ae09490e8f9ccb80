// moe_kv4_attend.cu -- attention over the 4-bit paged key/value cache for a few
// new tokens a sequence (decode steps, drafted tokens).
#include "moe_kv_few.cuh"
#include "moe_kv4.cuh"

#include <algorithm>

namespace {

// ---- few new tokens a sequence: keys and values streamed once ----
//
// The work is cut, shared out and joined as in the kernel for the 8-bit cache
// (moe_kv8_attend.cu): units of 64 tokens, one kv head and 16 rows (new tokens x
// the kv head's query heads) in order of (sequence, kv head, row tile, tokens),
// a contiguous share of them for each CTA and each of its warps; what a share
// cuts apart is joined in a fixed order.
//
// A unit's pages are one bulk copy each, codes and scales together.  Codes
// become fp16 by the hardware's conversion, unscaled (E2M1 is exact in it); the
// blocks' scales meet fp32 numbers instead, of which there are fewer: a score is
// the sum over blocks of 32 dims of the key's scale times the block's product,
// and a token's weight is multiplied by the scale of each value block before it
// becomes that block's fp16 operand.  Keys are read by ldmatrix, a thread 8 dims
// of a token (the queries are loaded in that order); values by its transposing
// form, a thread 4 dims of two tokens, whose nibbles two masks bring side by
// side.
//
// Scales are turned into floats once for a warp's 32 tokens, through shared
// memory: a lane a word, then 16 bytes a thread and block.  (Each thread its own:
// 128 of the 430 instructions of the integer pipe that 32 tokens of D = 128 take,
// and that pipe bounds the kernel.)
//
// Softmax, per row, in units of log2: m at least every score so far, moved (to 4
// above the largest) only when one passes it, so that the common step has no
// exchange between lanes; l the sum of the weights w = 2^(s - m) <= 1.  The
// accumulator of a block of values holds sum w 2^(15 + e - E) code over tokens
// with scale 2^e, E the largest e so far, for all rows the same.  Where the e of
// 32 tokens are all within 4 of E, w 2^(15 + e - E) is the fp16 operand: the row's
// largest is then at least 2^6 and the others keep 11 bits down to 2^-20 of it.
// Where they are not, tokens are multiplied in classes of e within 4 of one
// another, each with its own reference, and added in fp32.
// q is scaled per row by a power of two into fp16's range: exact for a bf16
// row's values down to 2^-28 of its largest.

// Warps, and units in each one's ring: as many warps as registers and shared
// memory allow (a multiple of 4: registers are given to four at a time).
template <int D, bool TOP>
struct Few {
    static constexpr int kWarps = D == 64 ? (TOP ? 12 : 16) : (TOP ? 8 : 12);
    static constexpr int kStages = D == 128 ? 1 : 2;
    static constexpr int kStage = kTile * D / 16 * 17;   // bytes of one unit
    static constexpr int kPad = D + 8;                   // floats of a partial's row
    static constexpr int kRowsHeld = TOP ? 16 : 8;
    // a partial: acc [rows][D + 8], then m, l [rows], the accumulator's exponent [blocks][rows]
    static constexpr int kScalars = kRowsHeld * (2 + D / 32);
    static constexpr int kPartial = kRowsHeld * kPad + kScalars;
    // a warp's own: the ring, scales, queries; the last partial goes over them, and behind it the scalars of a join
    static constexpr int kScales = kStages * kStage, kQueries = kScales + D / 32 * 2 * 32 * 4;
    static constexpr int kHeld = kQueries + kRowsHeld / 8 * (D / 32) * 512;
    static constexpr int kJoin = (kPartial + (kMaxCtas + kWarps) / kWarps * kScalars) * 4;   // kMaxCtas + 1 partials at most
    static constexpr int kRing = ((kHeld > kJoin ? kHeld : kJoin) + 127) / 128 * 128;
    static constexpr int kSmem = kWarps * (kRing + kPartial * 4);   // without the sequences
};

struct FewArgs {
    Kv4Attend a;
    int G;                     // query heads per kv head
    int32_t *status;           // [2]
    uint32_t *tickets;         // [kMaxCtas], zero between calls
    float *parts;              // [kMaxCtas][2][partial_floats]
    int *seqs;                 // [3][n_seqs], or null: in shared memory
};

__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void mma_f16_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
                 : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ uint32_t lds32(uint32_t at) {
    uint32_t w;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w) : "r"(at) : "memory");
    return w;
}
__device__ __forceinline__ void sts128(uint32_t at, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
__device__ __forceinline__ void lds128(uint32_t at, uint32_t (&v)[4]) {
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "r"(at) : "memory");
}
__device__ __forceinline__ void lds256(uint32_t at, float (&v)[8]) {
    asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]) : "r"(at) : "memory");
    asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]) : "r"(at + 16) : "memory");
}
// Byte i of w, in the exponent's place.
__device__ __forceinline__ uint32_t byte_exp(uint32_t w, int i) { return (i == 3 ? w >> 1 : w << (23 - 8 * i)) & 0x7F800000u; }

// What turns a row's accumulator into its output (N: of the block, the exponent of its unit; sink: the
// head's logit in units of log2, -inf without one): two factors, as their
// product may be below 2^-126 where the output is not.
__device__ __forceinline__ float2 row_factor(float m, float l, float N, float sink) {
    const float top = fmaxf(m, sink);
    const float den = top == -INFINITY ? l : (m == -INFINITY ? l : l * ex2(m - top)) + ex2(sink - top);
    const float half = ex2(0.5f * (N + (m - top)));
    return den == 0.f || m == -INFINITY ? make_float2(0.f, 0.f) : make_float2(half, half / den);   // an empty row: 0; NaN stays NaN
}

template <int D, int P, bool TOP>
__global__ void __launch_bounds__(Few<D, TOP>::kWarps * 32, 1) moe_kv4_few_kernel(const __grid_constant__ FewArgs f) {
    constexpr int W = Few<D, TOP>::kWarps, NP = kTile / P, HP = P == 16 ? 2 : 1, NB = D / 32, ST = Few<D, TOP>::kStage, PAD = Few<D, TOP>::kPad;
    constexpr int S = Few<D, TOP>::kStages, R = TOP ? 16 : 8, RR = TOP ? 2 : 1, PF = Few<D, TOP>::kPartial, PB = kv4_page_bytes(P, D);
    constexpr int SC = Few<D, TOP>::kScalars, RING = Few<D, TOP>::kRing;
    static_assert(Few<D, TOP>::kSmem + kSmemSeqs * 12 <= 230000, "shared memory");
    extern __shared__ __align__(128) unsigned char smem_raw[];
    __shared__ __align__(8) uint64_t bars[W][S];
    __shared__ int scan[W];
    __shared__ Job jobs[W];                       // each warp's running job
    __shared__ Seg segs[2 * W];                   // head and tail of each warp
    __shared__ int list[2 * W], group_at[2 * W + 1], group_seg[2 * W], shared_seg[2], s_first[2], s_count[2];
    const Kv4Attend &a = f.a;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t4 = lane & 3;
    unsigned char *ring = smem_raw + (size_t)warp * RING;
    float *part = reinterpret_cast<float *>(smem_raw + (size_t)W * RING);   // [W] head partials; tails go over the rings
    // per sequence: units of those before it (a kv head), index of its first unit in it, tokens that can be seen; of
    // many sequences in the workspace, where every CTA writes the same
    const uint32_t scratch = smem_u32(ring) + Few<D, TOP>::kScales;    // floats [keys, values][block][t4][8]
    const uint32_t queries = smem_u32(ring) + Few<D, TOP>::kQueries;   // fp16 [block][row / 8][lane][8]
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
    unsigned pages_at[S];   // per stage: the pages that are there
#pragma unroll
    for (int s = 0; s < S; s++) pages_at[s] = 0;
    auto fetch_page = [&]() {   // lane p < NP: page of the unit iu
        pg = -1;
        if (iu < u1 && lane < NP) {
            const int tile = seq(1, ij.b) + iu - ij.u0;
            const int t0 = tile * kTile + lane * P;
            if (t0 < seq(2, ij.b)) pg = __ldg(a.table + (size_t)ij.b * a.width + t0 / P);
        }
    };
    auto issue = [&](int stage) {
        const bool ok = lane < NP && pg >= 0 && pg < a.c.n_pages;
        const unsigned okm = __ballot_sync(0xffffffffu, ok);
        const uint32_t bar = smem_u32(&bars[warp][stage]);
        if (lane == 0)
            asm volatile("{ .reg .b64 st; mbarrier.arrive.expect_tx.shared::cta.b64 st, [%0], %1; }" ::"r"(bar),
                         "r"((uint32_t)(__popc(okm) * PB)) : "memory");
        __syncwarp();
        if (ok) bulk_copy(smem_u32(ring + stage * ST) + lane * PB, a.c.c + ((size_t)pg * a.c.KVH + ij.h) * PB, PB, bar);
#pragma unroll
        for (int s = 0; s < S; s++)
            if (s == stage) pages_at[s] = okm;
        if (S > 1) ji = ij;
        iu++;
        if (iu < u1 && iu == ij.u0 + ij.nt) ij = job_of(iu);
        fetch_page();
    };
    if (u0 < u1) {
        ij = job_of(u0);
        fetch_page();
    }
    bool fine = true;

    // the computing side
    // values: up to 8 rows transposed (dims 32 b + 4 g + e of rows 2 t4, 2 t4 + 1: tile 2 b + (e & 1), number e & 2 and
    // the one after it), else 16 rows (rows g, g + 8, dims 32 b + 8 t4 + 4 x + j: tile 4 b + j, number x)
    constexpr int NT = TOP ? 4 : 2, NA = NB * NT;   // tiles of a block, all
    float acc[NA][4], m[RR], l[RR];
    // E of block vb, as a scale byte: where the lane's group of 8 has value scales (D = 64: lanes 16 ..)
    const int vb = D == 64 ? (lane >> 3) & 1 : lane >> 3;
    int E = 0;
    auto of_block = [&](auto x, int b) { return __shfl_sync(0xffffffffu, x, 8 * b + (D == 64 ? 16 : 0)); };
    const float sc = a.scale * kLog2e;
    float rs[RR];     // turns a row's products into scores
    float sink[RR];
    bool begun = false;
    int pos[RR], pmin = 0, pmax = 0, seen = 0, at0 = 0, job_end = 0;   // the job's tokens, place of unit 0 in it, unit behind its last
    int seg0 = u0;           // first unit of the running segment
    static_assert(S <= 2, "the job of a unit that is issued and not begun is ji");
#pragma unroll
    for (int r = 0; r < RR; r++) sink[r] = -INFINITY, pos[r] = 0, rs[r] = 0.f;
    for (int u = u0; u < u1 && fine; u++) {
        const int i = u - u0, stage = i % S;
        const bool fresh = !begun;
        const Job j = S > 1 && iu > u ? ji : ij;   // the unit's, where it begins one
#pragma unroll 1
        while (iu < u1 && iu < u + S) issue((iu - u0) % S);
        if (fresh) {
            // a new job: its rows' queries, while the unit's pages are on their way
            if (lane == 0) jobs[warp] = j;
            seen = seq(2, j.b), at0 = seq(1, j.b) - j.u0, job_end = j.u0 + j.nt;
            begun = true, seg0 = u;
            int row0, n, pos0;
            kv8_rows(a, j.b, row0, n, pos0);
            pmin = pos0 + j.rt * kRows / f.G;
            pmax = pos0 + min(n * f.G - 1, j.rt * kRows + kRows - 1) / f.G;
#pragma unroll
            for (int r = 0; r < RR; r++) {
                const int rr = j.rt * kRows + g + 8 * r, i2 = rr / f.G, head = j.h * f.G + rr - i2 * f.G;
                const bool on = rr < n * f.G;
                pos[r] = on ? pos0 + i2 : -1;
                sink[r] = on && a.sinks ? a.sinks[head] * kLog2e : -INFINITY;
                const uint16_t *q = a.q + (long long)(row0 + i2) * a.q_stride + head * D + 8 * t4;
                uint4 w[NB];
#pragma unroll
                for (int b = 0; b < NB; b++) w[b] = on ? __ldg(reinterpret_cast<const uint4 *>(q + 32 * b)) : make_uint4(0, 0, 0, 0);
                // the row scaled: its largest magnitude to [2^14, 2^15) (exponent field e means 2^(e - 127))
                uint32_t am = 0;
#pragma unroll
                for (int b = 0; b < NB; b++) {
                    const uint32_t x[4] = {w[b].x, w[b].y, w[b].z, w[b].w};
#pragma unroll
                    for (int e = 0; e < 4; e++) am = max(am, max(x[e] & 0x7FFFu, (x[e] >> 16) & 0x7FFFu));
                }
                am = max(am, __shfl_xor_sync(0xffffffffu, am, 1));
                am = max(am, __shfl_xor_sync(0xffffffffu, am, 2));
                const int up = min(141 - (int)(am >> 7), 127);
                const float mul = pow2i(up);
                rs[r] = fmaxf(pow2i(-up) * sc, 1e-37f);   // > 0: a hidden token's -inf stays
                m[r] = -INFINITY, l[r] = 0.f;
#pragma unroll
                for (int b = 0; b < NB; b++) {
                    const uint32_t x[4] = {w[b].x, w[b].y, w[b].z, w[b].w};
                    uint32_t y[4];   // dims 8 t4 + 2 e, + 1
#pragma unroll
                    for (int e = 0; e < 4; e++) y[e] = pack_f16(__uint_as_float(x[e] << 16) * mul, __uint_as_float(x[e] & 0xFFFF0000u) * mul);
                    sts128(queries + (b * RR + r) * 512 + 16 * lane, y[0], y[1], y[2], y[3]);
                }
            }
            E = 0;
#pragma unroll
            for (int d = 0; d < NA; d++) acc[d][0] = acc[d][1] = acc[d][2] = acc[d][3] = 0.f;
        }
        __syncwarp();
        fine = bar_wait(smem_u32(&bars[warp][stage]), (uint32_t)(i / S) & 1, f.status, 95);
        fine = __all_sync(0xffffffffu, fine);
        if (!fine) break;
        const int u_at = (at0 + u) * kTile;
        const unsigned here = S == 1 || stage == 0 ? pages_at[0] : pages_at[S - 1];
        // 32 tokens at a time: octets 0 .. 3, of which a thread has tokens 8 n + 2 t4 + e
#pragma unroll 1
        for (int hf = 0; hf < 2; hf++) {
            const int t0 = u_at + 32 * hf;
            const unsigned pages = P == 64 ? here : here >> (hf * HP);   // bit p: of this half
            const bool whole = t0 + 32 <= seen && t0 + 31 <= pmin && (a.window == 0 || t0 > pmax - a.window) && (pages & ((1u << HP) - 1)) == (1u << HP) - 1;
            // this half's codes: a token's row of key block b
            const uint32_t page = smem_u32(ring + stage * ST) + (P == 64 ? 0 : hf * HP * PB);
            const uint32_t rows_at = page + (P == 16 ? (lane >> 4) * PB + (lane & 15) * 16 : P == 32 ? lane * 16 : hf * 512 + lane * 16);
            // its scales: a lane the four tokens of a word, octets 2 kk and 2 kk + 1, of block vb
            uint32_t vs;
            {
                const int kk = (lane >> 2) & 1;
                const uint32_t at = page + P * D + 4 * t4 + (P == 64 ? hf * 32 : 0) + (P == 16 ? kk * PB : kk * 16) + vb * P;
                const uint32_t ks = lds32(at + (D == 64 && lane >= 16 ? NB * P : 0));
                vs = D == 64 ? ks : lds32(at + NB * P);
                if (D == 128 || lane < 16) sts128(scratch + 16 * (lane & ~7) + 32 * t4 + 16 * kk, byte_exp(ks, 0), byte_exp(ks, 1), byte_exp(ks, 2), byte_exp(ks, 3));
                if (!whole) {
                    uint32_t keep = 0;   // values that some row sees
#pragma unroll
                    for (int e = 0; e < 4; e++) {
                        const int n = 2 * kk + (e >> 1), t = t0 + 8 * n + 2 * t4 + (e & 1);
                        if (t < seen && (pages >> (n * HP / 4) & 1) && t <= pmax && t >= kv8_first(pmin, a.window)) keep |= 0xFFu << (8 * e);
                    }
                    vs &= keep;
                }
                if (D == 64 && lane < 16) vs = 0;
            }
            // the largest and (as 256 less it) the smallest value scale of each block
            const uint32_t lo2 = vs & 0x00FF00FFu, hi2 = vs >> 8 & 0x00FF00FFu;
            const uint32_t most = __vmaxu2(lo2, hi2), least = __vmaxu2((0x01000100u - lo2) & 0x00FF00FFu, (0x01000100u - hi2) & 0x00FF00FFu);
            uint32_t ends = __vmaxu2(__byte_perm(most, least, 0x5410), __byte_perm(most, least, 0x7632));
#pragma unroll
            for (int o = 1; o < 8; o <<= 1) ends = __vmaxu2(ends, __shfl_xor_sync(0xffffffffu, ends, o));
            const int E1 = max(E, (int)(ends & 0xFFFFu));
            const bool wild = __any_sync(0xffffffffu, ends && E1 - 256 + (int)(ends >> 16) > 4);
            if (__any_sync(0xffffffffu, E1 > E)) {
                const float k = ex2((float)(E - E1));
#pragma unroll
                for (int b = 0; b < NB; b++) {
                    const float kb = of_block(k, b);
#pragma unroll
                    for (int d = b * NT; d < (b + 1) * NT; d++) acc[d][0] *= kb, acc[d][1] *= kb, acc[d][2] *= kb, acc[d][3] *= kb;
                }
                E = E1;
            }
            // values' scales over 2^(E - 15), where that is all (see below for the others); nothing for what is not seen
            auto scale_values = [&](uint32_t w, int E) {
                uint32_t x[4];
#pragma unroll
                for (int e = 0; e < 4; e++) x[e] = w >> (8 * e) & 255u ? byte_exp(w, e) + ((uint32_t)(142 - E) << 23) : 0u;
                if (D == 128 || lane >= 16) sts128(scratch + NB * 128 + 128 * vb + 32 * t4 + 4 * (lane & 4), x[0], x[1], x[2], x[3]);
            };
            if (!wild) scale_values(vs, E);
            __syncwarp();
            // scores: 4 token octets x (rows g: c0, c1; rows g + 8: c2, c3)
            float s[4][2 * RR];
#pragma unroll
            for (int n = 0; n < 4; n++)
#pragma unroll
                for (int e = 0; e < 2 * RR; e++) s[n][e] = 0.f;
#pragma unroll 1
            for (int b = 0; b < NB; b++) {
                uint32_t kw[4];
                ldsm4(kw, rows_at + b * (P * 16));
                uint32_t x0[4], x1[4];
                lds128(queries + b * RR * 512 + 16 * lane, x0);
                if (TOP) lds128(queries + (b * RR + RR - 1) * 512 + 16 * lane, x1);
                const uint32_t q0[4] = {x0[0], TOP ? x1[0] : 0u, x0[1], TOP ? x1[1] : 0u}, q1[4] = {x0[2], TOP ? x1[2] : 0u, x0[3], TOP ? x1[3] : 0u};
                float ks[8];   // of octet n and token e: 2 n + e
                lds256(scratch + 128 * b + 32 * t4, ks);
#pragma unroll
                for (int n = 0; n < 4; n++) {
                    uint32_t h[4];
                    float x[4];
                    e2m1x8_to_f16(kw[n], h);
                    mma_f16_first(x, q0, h[0], h[1]);
                    mma_f16(x, q1, h[2], h[3]);
#pragma unroll
                    for (int e = 0; e < 2 * RR; e++) s[n][e] = fmaf(x[e], ks[2 * n + (e & 1)], s[n][e]);
                }
            }
#pragma unroll
            for (int n = 0; n < 4; n++)
#pragma unroll
                for (int e = 0; e < 2 * RR; e++) s[n][e] *= rs[e >> 1];
            if (!whole) {
#pragma unroll
                for (int n = 0; n < 4; n++)
#pragma unroll
                    for (int e = 0; e < 2; e++) {
                        const int t = t0 + 8 * n + 2 * t4 + e;
                        const bool there = t < seen && (pages >> (n * HP / 4) & 1);
#pragma unroll
                        for (int r = 0; r < RR; r++)
                            if (!(there && t <= pos[r] && (a.window == 0 || t > pos[r] - a.window))) s[n][2 * r + e] = -INFINITY;
                    }
            }
            // a score above m: m moves
            float mx[RR];
            bool above = false;
#pragma unroll
            for (int r = 0; r < RR; r++) {
                mx[r] = fmaxf(fmaxf(fmaxf(s[0][2 * r], s[0][2 * r + 1]), fmaxf(s[1][2 * r], s[1][2 * r + 1])),
                              fmaxf(fmaxf(s[2][2 * r], s[2][2 * r + 1]), fmaxf(s[3][2 * r], s[3][2 * r + 1])));
                above |= mx[r] > m[r];
            }
            if (__any_sync(0xffffffffu, above)) {
                float corr[RR];
#pragma unroll
                for (int r = 0; r < RR; r++) {
                    const float q = quad_max(mx[r]), to = q > m[r] ? q + 4.f : m[r];
                    corr[r] = q > m[r] ? ex2(m[r] - to) : 1.f;
                    l[r] *= corr[r], m[r] = to;
                }
                // rows in the accumulator's columns (transposed: rows 2 t4, 2 t4 + 1; else g, g + 8)
                const float k0 = TOP ? corr[0] : __shfl_sync(0xffffffffu, corr[0], 8 * t4);
                const float k1 = TOP ? corr[RR - 1] : __shfl_sync(0xffffffffu, corr[0], 8 * t4 + 4);
#pragma unroll
                for (int d = 0; d < NA; d++) {
                    acc[d][0] *= k0, acc[d][1] *= TOP ? k0 : k1;
                    acc[d][2] *= TOP ? k1 : k0, acc[d][3] *= k1;
                }
            }
#pragma unroll
            for (int r = 0; r < RR; r++) {
                const float ms = m[r] == -INFINITY ? 0.f : m[r];
                float sum = 0.f;
#pragma unroll
                for (int n = 0; n < 4; n++)
#pragma unroll
                    for (int e = 0; e < 2; e++) sum += s[n][2 * r + e] = ex2(s[n][2 * r + e] - ms);
                l[r] += sum;
            }
            // block b's values times the weights, times(tile, operands)
            auto values = [&](int b, auto times) {
                float vsc[8];
                lds256(scratch + NB * 128 + 128 * b + 32 * t4, vsc);
                uint32_t vw[4];
                ldsm4t(vw, rows_at + P * D / 2 + b * (P * 16));
#pragma unroll
                for (int kk = 0; kk < 2; kk++) {
                    // tokens of a word's halves side by side: dims 4 g and 4 g + 2 of two octets, 4 g + 1 and 4 g + 3
                    const uint32_t lo = __byte_perm(vw[2 * kk], vw[2 * kk + 1], 0x5410), hi = __byte_perm(vw[2 * kk], vw[2 * kk + 1], 0x7632);
                    uint32_t h0[4], h1[4], p[RR][2];
                    e2m1x8_to_f16((lo & 0x0F0F0F0Fu) | (hi << 4 & 0xF0F0F0F0u), h0);
                    e2m1x8_to_f16((lo >> 4 & 0x0F0F0F0Fu) | (hi & 0xF0F0F0F0u), h1);
#pragma unroll
                    for (int r = 0; r < RR; r++)
#pragma unroll
                        for (int x = 0; x < 2; x++) {
                            const int n = 2 * kk + x;
                            p[r][x] = pack_f16(s[n][2 * r] * vsc[2 * n], s[n][2 * r + 1] * vsc[2 * n + 1]);
                        }
                    times(kk, h0, h1, p);
                }
            };
            auto product = [&](float (*to)[4], const uint32_t (&h0)[4], const uint32_t (&h1)[4], const uint32_t (&p)[RR][2]) {
                if constexpr (TOP) {
                    const uint32_t pf[4] = {p[0][0], p[RR - 1][0], p[0][1], p[RR - 1][1]};
                    mma_f16(to[0], pf, h0[0], h0[2]);
                    mma_f16(to[1], pf, h1[0], h1[2]);
                    mma_f16(to[2], pf, h0[1], h0[3]);
                    mma_f16(to[3], pf, h1[1], h1[3]);
                } else {
                    mma_f16(to[0], h0, p[0][0], p[0][1]);
                    mma_f16(to[1], h1, p[0][0], p[0][1]);
                }
            };
            if (!wild) {
#pragma unroll
                for (int b = 0; b < NB; b++)
                    values(b, [&](int, const uint32_t (&h0)[4], const uint32_t (&h1)[4], const uint32_t (&p)[RR][2]) { product(acc + NT * b, h0, h1, p); });
            } else {
                // classes of scales, the largest first; each one's products apart
                uint32_t left = vs;
#pragma unroll 1
                while (__any_sync(0xffffffffu, left)) {
                    int top = 0;
#pragma unroll
                    for (int e = 0; e < 4; e++) top = max(top, (int)(left >> (8 * e) & 255u));
#pragma unroll
                    for (int o = 1; o < 8; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
                    uint32_t in = 0;
#pragma unroll
                    for (int e = 0; e < 4; e++)
                        if ((int)(left >> (8 * e) & 255u) >= max(top - 4, 1)) in |= 0xFFu << (8 * e);
                    __syncwarp();   // the scales before are read
                    scale_values(left & in, top);
                    left &= ~in;
                    __syncwarp();
                    const float k = pow2i(top - E);
#pragma unroll
                    for (int b = 0; b < NB; b++) {
                        float part_acc[NT][4];
                        const float kb = of_block(k, b);
#pragma unroll
                        for (int d = 0; d < NT; d++) part_acc[d][0] = part_acc[d][1] = part_acc[d][2] = part_acc[d][3] = 0.f;
                        values(b, [&](int, const uint32_t (&h0)[4], const uint32_t (&h1)[4], const uint32_t (&p)[RR][2]) { product(part_acc, h0, h1, p); });
#pragma unroll
                        for (int d = 0; d < NT; d++)
#pragma unroll
                            for (int e = 0; e < 4; e++) acc[NT * b + d][e] = fmaf(part_acc[d][e], kb, acc[NT * b + d][e]);
                    }
                }
            }
            __syncwarp();   // the scales are read
        }
        __syncwarp();   // the stage is read: the next iteration fills it
        if (u + 1 == job_end || u + 1 == u1) {
            const Job j = jobs[warp];
            begun = false;
            const bool begins = seg0 == j.u0, ends = u + 1 == j.u0 + j.nt;
            float ls[RR];
#pragma unroll
            for (int r = 0; r < RR; r++) ls[r] = quad_sum(l[r]);
            float N[NB];   // the accumulator's unit: 2^N
#pragma unroll
            for (int b = 0; b < NB; b++) N[b] = (float)(of_block(E, b) - 142);
            if (begins && ends) {
                // the whole job was this warp's
                int row0, n, pos0;
                kv8_rows(a, j.b, row0, n, pos0);
#pragma unroll
                for (int r = 0; r < 2; r++) {
                    const int rr = j.rt * kRows + (TOP ? g + 8 * r : 2 * t4 + r);
                    __nv_bfloat16 *o = reinterpret_cast<__nv_bfloat16 *>(a.out) + (long long)(row0 + rr / f.G) * a.o_stride +
                                       (j.h * f.G + rr % f.G) * D + (TOP ? 8 * t4 : 4 * g);
#pragma unroll
                    for (int b = 0; b < NB; b++) {
                        float2 k = row_factor(m[TOP ? r : 0], ls[TOP ? r : 0], N[b], sink[TOP ? r : 0]);
                        if (!TOP) k = make_float2(__shfl_sync(0xffffffffu, k.x, 8 * t4 + 4 * r), __shfl_sync(0xffffffffu, k.y, 8 * t4 + 4 * r));
                        if (rr >= n * f.G) continue;
                        auto put = [&](float x, float y) {
                            const __nv_bfloat162 v = __floats2bfloat162_rn(x * k.x * k.y, y * k.x * k.y);
                            return *reinterpret_cast<const uint32_t *>(&v);
                        };
                        const float (*t)[4] = acc + NT * b;
                        if constexpr (TOP)
                            *reinterpret_cast<uint4 *>(o + 32 * b) = make_uint4(put(t[0][2 * r], t[1][2 * r]), put(t[2][2 * r], t[3][2 * r]),
                                                                                put(t[0][2 * r + 1], t[1][2 * r + 1]), put(t[2][2 * r + 1], t[3][2 * r + 1]));
                        else
                            *reinterpret_cast<uint2 *>(o + 32 * b) = make_uint2(put(t[0][r], t[1][r]), put(t[0][2 + r], t[1][2 + r]));
                    }
                }
            } else {
                // a head of more to come goes to its own place, the last segment over
                // the ring, whose copies have all landed and been read
                const bool last = u + 1 == u1;
                float *to = last ? reinterpret_cast<float *>(ring) : part + (size_t)warp * PF;
#pragma unroll
                for (int r = 0; r < 2; r++) {
                    float *row = to + (TOP ? g + 8 * r : 2 * t4 + r) * PAD + (TOP ? 8 * t4 : 4 * g);
#pragma unroll
                    for (int b = 0; b < NB; b++) {
                        const float (*t)[4] = acc + NT * b;
                        if constexpr (TOP) {
                            *reinterpret_cast<float4 *>(row + 32 * b) = make_float4(t[0][2 * r], t[1][2 * r], t[2][2 * r], t[3][2 * r]);
                            *reinterpret_cast<float4 *>(row + 32 * b + 4) = make_float4(t[0][2 * r + 1], t[1][2 * r + 1], t[2][2 * r + 1], t[3][2 * r + 1]);
                        } else {
                            *reinterpret_cast<float4 *>(row + 32 * b) = make_float4(t[0][r], t[1][r], t[0][2 + r], t[1][2 + r]);
                        }
                    }
                }
#pragma unroll
                for (int r = 0; r < RR; r++) {
                    float *ml = to + R * PAD + g + 8 * r;
                    if (t4 == 0) {
                        ml[0] = m[r], ml[R] = ls[r];
#pragma unroll
                        for (int b = 0; b < NB; b++) ml[(2 + b) * R] = N[b];
                    }
                }
                if (lane == 0) segs[2 * warp + last] = {j.u0, j.nt, j.b, j.h, j.rt};
            }
        }
    }
    if (!fine)   // copies may still be in flight: each stage's last phase, with a limit
        for (int s = 0; s < S; s++)
            if (s < iu - u0) bar_wait(smem_u32(&bars[warp][s]), (uint32_t)((iu - u0 - 1 - s) / S) & 1, f.status, 96);
    __syncthreads();

    // Joining: the CTA's segments in order, those of one job a group (they are
    // neighbours); then, of the jobs that other CTAs share (at most the first
    // and the last), those whose other partials are all there.  Either time all
    // groups at once: the partials' m, l and N side by side in shared memory,
    // then a thread for each group, row and pair of dims.
    auto scal = [&](int k) {   // SC floats, behind the tails in the rings
        return reinterpret_cast<float *>(smem_raw + (size_t)(k % W) * RING) + PF + k / W * SC;
    };
    auto scalars = [&](int k, const float *from) {
        for (int y = lane; y < SC; y += 32) scal(k)[y] = *(volatile const float *)(from + R * PAD + y);
    };
    // partials k0 .. k0 + n - 1 (at(k)) of segment sg's job: row r, dims d, d + 1
    auto join = [&](const Seg &sg, int k0, int n, auto at, bool done, int r, int d) {
        int row0, nr, pos0;
        kv8_rows(a, sg.b, row0, nr, pos0);
        if (r >= min(kRows, nr * f.G - sg.rt * kRows)) return;
        const int nb = (2 + d / 32) * R + r;   // where a partial's N of the block is
        float mm = -INFINITY, NN = -INFINITY, ll = 0.f;
#pragma unroll 4
        for (int k = k0; k < k0 + n; k++) mm = fmaxf(mm, scal(k)[r]);
        const float ms = mm == -INFINITY ? 0.f : mm;
#pragma unroll 4
        for (int k = k0; k < k0 + n; k++) NN = fmaxf(NN, scal(k)[r] - ms + scal(k)[nb]);
        const float Ns = NN == -INFINITY ? 0.f : NN;
        float2 v = make_float2(0.f, 0.f);
#pragma unroll 8
        for (int k = k0; k < k0 + n; k++) {
            const float km = scal(k)[r], kl = scal(k)[R + r], kn = scal(k)[nb];
            const float c = ex2(km - ms + kn - Ns);   // no tokens: 2^-inf
            volatile const float *p = at(k) + r * PAD + d;
            v.x = fmaf(c, p[0], v.x), v.y = fmaf(c, p[1], v.y);
            ll += kl * (km == -INFINITY ? 1.f : ex2(km - ms));   // the l of NaN scores has no maximum
        }
        if (done) {
            const int rr = sg.rt * kRows + r, i2 = rr / f.G, head = sg.h * f.G + rr - i2 * f.G;
            const float2 k = row_factor(mm, ll, Ns, a.sinks ? a.sinks[head] * kLog2e : -INFINITY);
            *reinterpret_cast<__nv_bfloat162 *>(a.out + (long long)(row0 + i2) * a.o_stride + head * D + d) =
                __floats2bfloat162_rn(v.x * k.x * k.y, v.y * k.x * k.y);
        } else {
            float *mine_p = f.parts + ((size_t)blockIdx.x * 2 + (sg.u0 >= c0 ? 1 : 0)) * PF;
            *reinterpret_cast<float2 *>(mine_p + r * PAD + d) = v;
            if (d == 0) mine_p[R * PAD + r] = mm, mine_p[R * PAD + R + r] = ll;
            if (d % 32 == 0) mine_p[R * PAD + nb] = Ns;
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
        return x & 1 ? reinterpret_cast<const float *>(smem_raw + (size_t)(x >> 1) * RING) : part + (size_t)(x >> 1) * PF;
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

// A CTA of 128 threads a row and query head, 128 keys at a time.
__global__ void __launch_bounds__(128) moe_kv4_attend_kernel(const Kv4Attend a) {
    __shared__ float qs[128], p[128], red[128];
    __shared__ const uint8_t *vat[128];
    __shared__ const uint8_t *vsc[128];
    const int tid = threadIdx.x, D = a.c.D, P = a.c.P, NB = D / 32;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int b = blockIdx.x / a.max_new, i = blockIdx.x % a.max_new, head = blockIdx.y, h = head / (a.QH / a.c.KVH);
    int row0, n, pos0;
    kv8_rows(a, b, row0, n, pos0);
    if (i >= n) return;
    const int pos = pos0 + i, row = row0 + i;
    const int last = (int)min((long long)pos, (long long)a.width * P - 1), first = kv8_first(pos, a.window);
    if (tid < D) qs[tid] = bf16_to_f32(a.q[(long long)row * a.q_stride + head * D + tid]) * a.scale;
    __syncthreads();
    float m = -INFINITY, l = 0.f, acc = 0.f;
    const int dim = tid % D, part = tid / D, parts = 128 / D;
    for (int k0 = first; k0 <= last; k0 += 128) {
        const int t = k0 + tid;
        float s = -INFINITY;
        vat[tid] = nullptr;
        if (t <= last) {
            const int page = a.table[(size_t)b * a.width + t / P], off = t % P;
            if (page >= 0 && page < a.c.n_pages) {
                const uint8_t *base = a.c.c + ((size_t)page * a.c.KVH + h) * kv4_page_bytes(P, D);
                const uint8_t *sc = base + P * D + (off & ~15) + kv4_scale_byte(off & 15);
                float dot = 0.f;
                for (int x = 0; x < NB; x++) {
                    float part_dot = 0.f;
                    for (int c = 0; c < 4; c++) {
                        uint32_t hh[4];
                        e2m1x8_to_f16(*reinterpret_cast<const uint32_t *>(base + (x * P + off) * 16 + 4 * c), hh);
                        for (int e = 0; e < 4; e++) {
                            const float2 y = __half22float2(*reinterpret_cast<const __half2 *>(&hh[e]));
                            part_dot += y.x * qs[32 * x + 8 * c + 2 * e] + y.y * qs[32 * x + 8 * c + 2 * e + 1];
                        }
                    }
                    dot += part_dot * kv4_scale(sc[x * P]);
                }
                s = dot;
                vat[tid] = base + P * D / 2 + off * 16;
                vsc[tid] = sc + P * NB;
            }
        }
        red[tid] = s;
        __syncthreads();
        float mn = m;
        for (int j = 0; j < 128; j++) mn = fmaxf(mn, red[j]);
        const float f = mn == -INFINITY ? 1.f : expf(m - mn);
        p[tid] = vat[tid] ? expf(s - (mn == -INFINITY ? 0.f : mn)) : 0.f;
        __syncthreads();
        acc *= f, l *= f, m = mn;
        for (int j = part; j < 128; j += parts)
            if (vat[j]) {
                uint32_t hh[4];
                e2m1x8_to_f16(vat[j][(dim / 32) * P * 16 + dim % 32 / 2] >> (4 * (dim & 1)) & 15, hh);
                acc += p[j] * (kv4_scale(vsc[j][(dim / 32) * P]) * __half22float2(*reinterpret_cast<const __half2 *>(&hh[0])).x);
            }
        for (int j = 0; j < 128; j++) l += p[j];
        __syncthreads();
    }
    if (parts == 2) {
        p[tid] = acc;
        __syncthreads();
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

constexpr size_t kPartOffset = kKv8ClearBytes + (size_t)kKv8MaxSeqs * 12;

template <int D, int P, bool TOP>
cudaError_t few_launch(FewArgs f, int ctas, cudaStream_t st) {
    constexpr int W = Few<D, TOP>::kWarps;
    if (f.a.n_seqs <= kSmemSeqs) f.seqs = nullptr;
    const size_t smem = Few<D, TOP>::kSmem + (f.seqs ? 0 : (size_t)f.a.n_seqs * 12);
    static PerDevice<bool> opted;
    cudaError_t e = smem_optin_once(moe_kv4_few_kernel<D, P, TOP>, opted);
    if (e != cudaSuccess) return e;
    return launch_pdl(moe_kv4_few_kernel<D, P, TOP>, dim3(ctas), dim3(W * 32), smem, st, f);
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

size_t kv4_workspace_bytes(int D) { return kPartOffset + (size_t)kMaxCtas * 2 * (D == 64 ? Few<64, true>::kPartial : Few<128, true>::kPartial) * 4; }

cudaError_t launch_kv4_attend(const Kv4Attend &a, unsigned char *ws, cudaStream_t st) {
    const int G = a.QH / a.c.KVH;
    if ((long long)a.max_new * G <= 64) {
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
    return launch_pdl(moe_kv4_attend_kernel, dim3((unsigned)((long long)a.n_seqs * a.max_new), a.QH), dim3(128), 0, st, a);
}
