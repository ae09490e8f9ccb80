// moe_kv4_attend.cu -- attention over the 4-bit paged key/value cache for a few
// new tokens a sequence (decode steps, drafted tokens).
#include "moe_kv_few.cuh"
#include "moe_kv4.cuh"

#include <algorithm>
#include <climits>
#include <cmath>

namespace {

// ---- few new tokens a sequence: keys and values streamed once ----
//
// The work is cut, shared out and joined as in the kernel for the 8-bit cache
// (moe_kv8_attend.cu): units of 64 tokens, one kv head and 8 or 16 rows (new
// tokens x the kv head's query heads) in order of (sequence, kv head, row tile,
// tokens), a contiguous share of them for each CTA and each of its warps; what a
// share cuts apart is joined in a fixed order.
//
// A unit's pages are one bulk copy each, codes and scales together.  Long calls are
// bound by no one pipe: issue slots, the integer pipe, which turns codes into fp16
// (two cycles a pair, by the hardware's conversion), and HBM are about half busy
// each, and 16 warps an SM wait for instructions of fixed latency and for loads
// most.  So instructions are spared: 96 ragged sequences, 598 K tokens, 20 / 4 heads
// of 128 take 89 us, 49 at HBM's rate.  Short ones are latencies: of 16 x 4096
// tokens, 64 / 8 heads of 64, the bytes are 5 us of 23.5.
//  * Both products have the cache's side as their 16-row operand, keys [tokens]
//    [dims] and values [dims][tokens], and eight rows of queries or weights as
//    the other, so that nothing is multiplied that is no row; a unit may have
//    several such eights, for which its codes are converted once.
//  * Codes stay unscaled (E2M1 is exact in fp16).  A score is the sum over blocks
//    of 32 dims of the key's scale, in fp32, times the block's product; a weight
//    is multiplied by its token's value scale, a power of two, in fp16.
//  * Scales are turned into numbers once for a warp's 32 tokens, a lane a word,
//    and handed round through shared memory.
// Keys are read by ldmatrix, a thread 8 dims of a token (the queries are loaded
// in that order); values by its transposing form, a thread 4 dims of two tokens,
// whose nibbles two masks bring side by side.  Weights come out of the scores'
// layout by movmatrix.
//
// Softmax, per row, in units of log2: weights w = 2^(s - m) <= 2^15, l their sum.
// m moves (to 11 below the largest score) only when a score is more than 15 above
// it, so that the common step has no exchange between lanes.  The accumulator of a
// block of values holds sum w 2^(e - E) code over tokens with scale 2^e, E the
// largest e so far that any row sees, for all rows the same, but 25 at most: a row
// that sees none of the largest scales keeps its sum in fp32 (a row's largest
// weight is at least 2^7, so values down to 2^-84 keep 24 bits of it; an exponent
// of their own for each row's sums made decode steps 4 to 5 % slower).  Where the e of 32 tokens are all within
// 4 of E, w 2^(e - E) is the fp16 operand: the row's largest is then at least 2^7
// and the others keep 11 bits down to 2^-21 of it, some down to 2^-31.
// Where they are not, or above E, tokens are multiplied in classes of e within 4 of one
// another, each with its own reference, and added in fp32.
// q is scaled per row by a power of two into fp16's range: exact for a bf16
// row's values down to 2^-28 of its largest.

// RT: eights of rows of a unit; three or four, with the 8 warps that registers
// then allow, were slower than two units of two.  Warps, and units in each one's
// ring: as many warps as registers and shared memory allow (a multiple of 4:
// registers are given to four at a time; the ragged sequences above: 12 warps 99
// us, 16 94, and with both halves of a unit computed together 89).
template <int D, int P, int RT>
struct Few {
    static constexpr int kWarps = D == 64 ? (RT == 2 && P == 16 ? 12 : 16) : RT == 2 ? 8 : P == 32 ? 16 : 12;
    static constexpr int kStages = D == 128 ? 1 : 2;
    static constexpr int kStage = kTile * D / 16 * 17;   // bytes of one unit
    static constexpr int kPad = D + 8;                   // floats of a partial's row
    static constexpr int kUnitRows = 8 * RT;
    static constexpr int kHalves = RT == 1 ? 2 : 1;      // halves of a unit that are computed together
    // a partial: acc [rows][D + 8], then m, l [rows], the accumulator's exponent [blocks][rows]
    static constexpr int kPartial = kUnitRows * (kPad + 2 + D / 32);
    // a warp's own: the ring, scales, queries; the last partial goes over them, and behind it the scalars of a join
    static constexpr int kScales = kStages * kStage, kQueries = kScales + kHalves * (D / 32) * (128 + 64);
    static constexpr int kHeld = kQueries + RT * (D / 32) * 512;
    static constexpr int kJoin = (kPartial + (kMaxCtas + kWarps) / kWarps * 8 * (2 + D / 32)) * 4;   // kMaxCtas + 1 partials at most
    static constexpr int kRing = ((kHeld > kJoin ? kHeld : kJoin) + 127) / 128 * 128;
    static constexpr int kSmem = kWarps * kRing;   // without the sequences
};

constexpr int kMaxWarps = 16;
constexpr int kMostE = 127 + 25;   // as a scale byte: a step's products with the largest scales, 2^100 units, are below 2^123

// Of a unit's rows: their first and last position, the tokens that can be seen,
// and the unit's index from which the job is counted.
struct Span {
    int pmin, pmax, seen, seg0;
};

struct FewArgs {
    Kv4Attend a;
    int G;                     // query heads per kv head
    int most_up;               // powers of two that a row is scaled by, at most
    int32_t *status;           // [2]
    uint32_t *tickets;         // [kMaxCtas], zero between calls
    float *parts, *heads;      // [kMaxCtas][2] and [kMaxCtas][kMaxWarps] partials
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
__device__ __forceinline__ void sts64(uint32_t at, uint32_t x, uint32_t y) {
    asm volatile("st.shared.v2.b32 [%0], {%1,%2};" ::"r"(at), "r"(x), "r"(y) : "memory");
}
__device__ __forceinline__ void sts128(uint32_t at, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
__device__ __forceinline__ void lds128(uint32_t at, uint32_t (&v)[4]) {
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "r"(at) : "memory");
}
// An 8 x 8 matrix of 16-bit numbers, a lane two of a row, turned.
__device__ __forceinline__ uint32_t turn8(uint32_t x) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}
__device__ __forceinline__ uint32_t mul_f16(uint32_t x, uint32_t y) {
    const __half2 r = __hmul2(*reinterpret_cast<const __half2 *>(&x), *reinterpret_cast<const __half2 *>(&y));
    return *reinterpret_cast<const uint32_t *>(&r);
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

template <int D, int P, int RT>
__global__ void __launch_bounds__(Few<D, P, RT>::kWarps * 32, 1) moe_kv4_few_kernel(const __grid_constant__ FewArgs f) {
    typedef Few<D, P, RT> F;
    constexpr int W = F::kWarps, NP = kTile / P, HP = P == 16 ? 2 : 1, NB = D / 32, ST = F::kStage, PAD = F::kPad, S = F::kStages;
    constexpr int HV = F::kHalves, R = F::kUnitRows, PF = F::kPartial, PB = kv4_page_bytes(P, D), RING = F::kRing, SC = 8 * (2 + NB);   // (scalars of eight rows)
    static_assert(F::kSmem + kSmemSeqs * 12 <= 230000, "shared memory");
    extern __shared__ __align__(128) unsigned char smem_raw[];
    __shared__ __align__(8) uint64_t bars[W][S];
    __shared__ int scan[W];
    __shared__ Span spans[W];                     // what each warp's rows see
    __shared__ int row_pos[W][R], share[3];       // their positions; the CTA's first unit, the one behind its last; units of a kv head
    __shared__ unsigned pages_at[W][S];           // the pages that are there, of each stage
    __shared__ Job next_job[W], jobs[W][S];       // each warp's of the unit to be copied next, and of the stages
    __shared__ Seg segs[2 * W];                   // head and tail of each warp
    __shared__ int list[2 * W], group_at[2 * W + 1], group_seg[2 * W], shared_seg[2], s_first[2], s_count[2];
    const Kv4Attend &a = f.a;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t4 = lane & 3;
    unsigned char *ring = smem_raw + (size_t)warp * RING;
    float *part = f.heads + (size_t)blockIdx.x * (kMaxWarps * PF);   // [W] head partials (in memory, as few warps have one); tails go over the rings
    // per sequence: units of those before it (a kv head), index of its first unit in it, tokens that can be seen; of
    // many sequences in the workspace, where every CTA writes the same
    const uint32_t scratch = smem_u32(ring) + F::kScales;    // keys, floats [block][g][4]; values, fp16 pairs [block][t4][4]
    const uint32_t queries = smem_u32(ring) + F::kQueries;   // fp16 [block][row / 8][lane][8]
    int *seq_s = reinterpret_cast<int *>(smem_raw + (size_t)W * RING);
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
        return n > 0 ? max(1, (seen + kTile - 1) / kTile - first) * ((n * f.G + R - 1) / R) : 0;
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
    if (tid == 0) share[2] = total;
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
        const unsigned n_rt = ((lo + 1 < a.n_seqs ? seq(0, lo + 1) : share[2]) - seq(0, lo)) / j.nt;
        j.h = tile / n_rt;
        j.rt = tile % n_rt;
        j.u0 = before + tile * j.nt;
        return j;
    };
    // The CTA's share: the even cuts, each moved down to its job's first unit
    // where the job is at most 8 units long (a job that one CTA can take at
    // once is not worth joining across two).
    __syncthreads();   // share[2]
    int cut = (int)((long long)units * (blockIdx.x + (lane & 1)) / ctas);
    if (cut > 0 && cut < units) {
        const Job j = job_of(cut);
        if (j.nt <= 8) cut = j.u0;
    }
    if (tid < 2) share[tid] = cut;
    const int cta0 = __shfl_sync(0xffffffffu, cut, 0), cta1 = __shfl_sync(0xffffffffu, cut, 1);
    const int u0 = cta0 + (cta1 - cta0) * warp / W, u1 = cta0 + (cta1 - cta0) * (warp + 1) / W;   // c1 - c0 < 2^31 / 16 (host)

    // the issuing side: the next unit to copy, its pages read one unit ahead
    int iu = u0;
    int pg = -1;
    auto find_job = [&] {
        const Job j = job_of(iu);
        __syncwarp();
        if (lane == 0) next_job[warp] = j;
        __syncwarp();
    };
    auto fetch_page = [&]() {   // lane p < NP: page of the unit iu
        pg = -1;
        if (iu < u1 && lane < NP) {
            const int b = next_job[warp].b, tile = seq(1, b) + iu - next_job[warp].u0;
            const int t0 = tile * kTile + lane * P;
            if (t0 < seq(2, b)) pg = __ldg(a.table + (size_t)b * a.width + t0 / P);
        }
    };
    auto issue = [&](int stage) {
        const bool ok = lane < NP && pg >= 0 && pg < a.c.n_pages;
        const unsigned okm = __ballot_sync(0xffffffffu, ok);
        const uint32_t bar = smem_u32(&bars[warp][stage]);
        if (lane == 0) {
            jobs[warp][stage] = next_job[warp], pages_at[warp][stage] = okm;
            asm volatile("{ .reg .b64 st; mbarrier.arrive.expect_tx.shared::cta.b64 st, [%0], %1; }" ::"r"(bar),
                         "r"((uint32_t)(__popc(okm) * PB)) : "memory");
        }
        __syncwarp();
        if (ok) bulk_copy(smem_u32(ring + stage * ST) + lane * PB, a.c.c + ((size_t)pg * a.c.KVH + next_job[warp].h) * PB, PB, bar);
        iu++;
        if (iu < u1 && iu == next_job[warp].u0 + next_job[warp].nt) find_job();
        fetch_page();
    };
    if (u0 < u1) {
        find_job();
        fetch_page();
    }
    bool fine = true;

    // the computing side: a thread has rows 8 x + 2 t4 + c (c < 2); of values the dims 32 b + 4 g + 2 d + y of them, in number
    // 2 d + c of the tile [b][y][x]
    float acc[NB][2][RT][4], m[RT][2], l[RT][2];
    float rs[RT][2];       // turn a row's products into scores
    bool large = false;    // of scores: products are rounded to scores first, as they are when compared
    // E of block vb, as a scale byte: where the lane's group of 8 has value scales (D = 64: lanes 16 ..)
    const int vb = D == 64 ? (lane >> 3) & 1 : lane >> 3;
    int E = 0;
    auto of_block = [&](auto x, int b) { return __shfl_sync(0xffffffffu, x, 8 * b + (D == 64 ? 16 : 0)); };
    const float sc = a.scale * kLog2e;
    bool begun = false;
    int at0 = 0, seg_end = 0, all_from = 0, all_to = 0;   // place of unit 0 in the job, unit behind the segment's last, tokens that all rows see
    for (int u = u0; u < u1 && fine; u++) {
        const int i = u - u0, stage = i % S;
        const bool fresh = !begun;
#pragma unroll 1
        while (iu < u1 && iu < u + S) issue((iu - u0) % S);
        if (fresh) {
            // a new job: its rows' queries, while the unit's pages are on their way
            const Job j = jobs[warp][stage];
            at0 = seq(1, j.b) - j.u0, seg_end = min(j.u0 + j.nt, u1);
            begun = true;
            int row0, n, pos0;
            kv8_rows(a, j.b, row0, n, pos0);
            {
                // (rows far before the sequence are as near as the last of those: token - position stays in 32 bits)
                const int pmin = max(pos0 + j.rt * R / f.G, -1), pmax = max(pos0 + min(n * f.G - 1, j.rt * R + R - 1) / f.G, -1), seen = seq(2, j.b);
                all_from = a.window ? max(pmax - a.window + 1, 0) : 0, all_to = min(seen - 1, pmin);
                if (lane == 0) spans[warp] = {pmin, pmax, seen, u};
                for (int r = lane; r < R; r += 32) row_pos[warp][r] = j.rt * R + r < n * f.G ? max(pos0 + (j.rt * R + r) / f.G, -1) : -1;
            }
#pragma unroll
            for (int x = 0; x < RT; x++) {
                const int rr = j.rt * R + 8 * x + g, i2 = rr / f.G, head = j.h * f.G + rr - i2 * f.G;
                const uint16_t *q = a.q + (long long)(row0 + i2) * a.q_stride + head * D + 8 * t4;
                uint4 w[NB];
#pragma unroll
                for (int b = 0; b < NB; b++) w[b] = rr < n * f.G ? __ldg(reinterpret_cast<const uint4 *>(q + 32 * b)) : make_uint4(0, 0, 0, 0);
                // the row scaled: its largest magnitude to [2^14, 2^15) (exponent field e means 2^(e - 127))
                uint32_t am = 0;
#pragma unroll
                for (int b = 0; b < NB; b++) {
                    const uint32_t y[4] = {w[b].x, w[b].y, w[b].z, w[b].w};
#pragma unroll
                    for (int e = 0; e < 4; e++) am = max(am, max(y[e] & 0x7FFFu, (y[e] >> 16) & 0x7FFFu));
                }
                am = max(am, __shfl_xor_sync(0xffffffffu, am, 1));
                am = max(am, __shfl_xor_sync(0xffffffffu, am, 2));
                // (not so far that what undoes it is below 2^-120: a factor of 0 or less bits would make scores wrong)
                const int up = min(141 - (int)(am >> 7), f.most_up);
                const float mul = pow2i(up), back = pow2i(-up) * sc;
#pragma unroll
                for (int b = 0; b < NB; b++) {
                    const uint32_t y[4] = {w[b].x, w[b].y, w[b].z, w[b].w};
                    uint32_t z[4];   // dims 8 t4 + 2 e, + 1
#pragma unroll
                    for (int e = 0; e < 4; e++) z[e] = pack_f16(__uint_as_float(y[e] << 16) * mul, __uint_as_float(y[e] & 0xFFFF0000u) * mul);
                    sts128(queries + (b * RT + x) * 512 + 16 * lane, z[0], z[1], z[2], z[3]);
                }
#pragma unroll
                for (int c = 0; c < 2; c++) {
                    rs[x][c] = __shfl_sync(0xffffffffu, back, 8 * t4 + 4 * c);
                    m[x][c] = -INFINITY, l[x][c] = 0.f;
                }
            }
            E = 0, large = false;
#pragma unroll
            for (int i = 0; i < NB * 2 * RT * 4; i++) (&acc[0][0][0][0])[i] = 0.f;
        }
        __syncwarp();
        fine = bar_wait(smem_u32(&bars[warp][stage]), (uint32_t)(i / S) & 1, f.status, 95);
        fine = __all_sync(0xffffffffu, fine);
        if (!fine) break;
        const int u_at = (at0 + u) * kTile;
        const unsigned here = pages_at[warp][stage];
        // HV halves of 32 tokens at a time
#pragma unroll 1
        for (int h0 = 0; h0 < 2; h0 += HV) {
            const int t0 = u_at + 32 * h0;
            constexpr int PV = HV * HP < NP ? HV * HP : NP;              // their pages
            const unsigned pages = P == 64 ? here : here >> (h0 * HP);   // bit p: of these
            const bool whole = t0 >= all_from && t0 + 32 * HV - 1 <= all_to && (pages & ((1u << PV) - 1)) == (1u << PV) - 1;
            auto there = [&](int v, int n) { return pages >> ((4 * v + n) * PV / (4 * HV)) & 1; };   // of octet n of half v
            // the codes of half v: a token's row of key block b; its scales: a lane the four tokens of a word, octets 2 kk and
            // 2 kk + 1, of block vb
            const uint32_t page = smem_u32(ring + stage * ST) + (P == 64 ? 0 : h0 * HP * PB);
            const uint32_t rows_at = page + (P == 16 ? (lane >> 4) * PB + (lane & 15) * 16 : lane * 16) + (P == 64 ? h0 * 512 : 0);
            constexpr int kRowsOn = P == 64 ? 512 : HP * PB;   // from half to half
            uint32_t vs[HV], ends = 0;
#pragma unroll
            for (int v = 0; v < HV; v++) {
                const int kk = (lane >> 2) & 1;
                const uint32_t at = page + P * D + 4 * t4 + (P == 64 ? (h0 + v) * 32 : v * HP * PB) + (P == 16 ? kk * PB : kk * 16) + vb * P;
                const uint32_t ks = lds32(at + (D == 64 && lane >= 16 ? NB * P : 0));
                vs[v] = D == 64 ? ks : lds32(at + NB * P);
                if (D == 128 || lane < 16) {   // tokens 2 t4 and 2 t4 + 1 of the octets
                    const uint32_t to = scratch + v * (NB * 192) + 128 * vb + 32 * t4 + 8 * kk;
                    sts64(to, byte_exp(ks, 0), byte_exp(ks, 2));
                    sts64(to + 16, byte_exp(ks, 1), byte_exp(ks, 3));
                }
                if (!whole) {
                    const Span sp = spans[warp];
                    uint32_t keep = 0;   // values that some row sees
#pragma unroll
                    for (int e = 0; e < 4; e++) {
                        const int n = 2 * kk + (e >> 1), t = t0 + 32 * v + 8 * n + 2 * t4 + (e & 1);
                        if (t < sp.seen && there(v, n) && t <= sp.pmax && t >= kv8_first(sp.pmin, a.window)) keep |= 0xFFu << (8 * e);
                    }
                    vs[v] &= keep;
                }
                if (D == 64 && lane < 16) vs[v] = 0;
                // the largest and (as 256 less it) the smallest value scale of each block
                const uint32_t lo2 = vs[v] & 0x00FF00FFu, hi2 = vs[v] >> 8 & 0x00FF00FFu;
                const uint32_t most = __vmaxu2(lo2, hi2), least = __vmaxu2((0x01000100u - lo2) & 0x00FF00FFu, (0x01000100u - hi2) & 0x00FF00FFu);
                ends = __vmaxu2(ends, __vmaxu2(__byte_perm(most, least, 0x5410), __byte_perm(most, least, 0x7632)));
            }
#pragma unroll
            for (int o = 1; o < 8; o <<= 1) ends = __vmaxu2(ends, __shfl_xor_sync(0xffffffffu, ends, o));
            int E1 = max(E, (int)(ends & 0xFFFFu));
            bool wild = __any_sync(0xffffffffu, ends && E1 - 256 + (int)(ends >> 16) > 4);
            if (__any_sync(0xffffffffu, E1 > E)) {
                wild = wild || __any_sync(0xffffffffu, E1 > kMostE);
                E1 = min(E1, kMostE);
#pragma unroll
                for (int v = 0; v < HV; v++) vs[v] = __vminu4(vs[v], kKv4MaxByte * 0x01010101u);   // (bytes that no append writes)
                const float k = ex2((float)(E - E1));
#pragma unroll
                for (int b = 0; b < NB; b++) {
                    const float kb = of_block(k, b);
#pragma unroll
                    for (int i = 0; i < 2 * RT * 4; i++) (&acc[b][0][0][0])[i] *= kb;
                }
                E = E1;
            }
            // the value scales w of half v, all within 4 of E: 2^(e - E) in fp16; nothing for what is not seen
            auto scale_values = [&](int v, uint32_t w, int E) {
                const uint32_t some = (w | (w & 0x7F7F7F7Fu) + 0x7F7F7F7Fu) & 0x80808080u, keep = (some >> 7) * 255u;
                const uint32_t by = (uint32_t)(15 - E) * 0x10001u;
                w |= (uint32_t)E * 0x01010101u & ~keep;   // (no borrow from the neighbour)
                const uint32_t x = (__byte_perm(w, 0, 0x4140) + by) << 10 & __byte_perm(keep, 0, 0x1100);
                const uint32_t y = (__byte_perm(w, 0, 0x4342) + by) << 10 & __byte_perm(keep, 0, 0x3322);
                if (D == 128 || lane >= 16) sts64(scratch + v * (NB * 192) + NB * 128 + 64 * vb + 16 * t4 + 2 * (lane & 4), x, y);
            };
            if (!wild) {
#pragma unroll
                for (int v = 0; v < HV; v++) scale_values(v, vs[v], E);
            }
            __syncwarp();
            // products: tokens 32 v + 8 n + g, rows 2 t4 + c of the eights
            float s[RT][4 * HV][2];
#pragma unroll
            for (int i = 0; i < RT * 8 * HV; i++) (&s[0][0][0])[i] = 0.f;
#pragma unroll 1
            for (int b = 0; b < NB; b++) {
                uint32_t q[RT][4];
#pragma unroll
                for (int x = 0; x < RT; x++) lds128(queries + (b * RT + x) * 512 + 16 * lane, q[x]);
#pragma unroll
                for (int v = 0; v < HV; v++) {
                    uint32_t kw[4], ks[4], k0[2][4], k1[2][4];   // of two octets: dims 8 t4 .. + 3, + 4 .. + 7
                    ldsm4(kw, rows_at + v * kRowsOn + b * (P * 16));
                    lds128(scratch + v * (NB * 192) + 128 * b + 16 * g, ks);
#pragma unroll
                    for (int n = 0; n < 4; n++) {
                        uint32_t h[4];
                        e2m1x8_to_f16(kw[n], h);
                        k0[n >> 1][n & 1] = h[0], k0[n >> 1][2 + (n & 1)] = h[1];
                        k1[n >> 1][n & 1] = h[2], k1[n >> 1][2 + (n & 1)] = h[3];
                    }
#pragma unroll
                    for (int x = 0; x < RT; x++)
#pragma unroll
                        for (int h = 0; h < 2; h++) {
                            float y[4];
                            mma_f16_first(y, k0[h], q[x][0], q[x][1]);
                            mma_f16(y, k1[h], q[x][2], q[x][3]);
#pragma unroll
                            for (int e = 0; e < 4; e++) {
                                float &to = s[x][4 * v + 2 * h + (e >> 1)][e & 1];
                                to = fmaf(y[e], __uint_as_float(ks[2 * h + (e >> 1)]), to);
                            }
                        }
                }
            }
            if (!whole) {
#pragma unroll
                for (int x = 0; x < RT; x++)
#pragma unroll
                    for (int c = 0; c < 2; c++) {
                        // tokens from .. to of the thread's first one on
                        const int pos = row_pos[warp][8 * x + 2 * t4 + c], from = (a.window ? max(pos - a.window + 1, 0) : 0) - t0 - g, to = min(spans[warp].seen - 1, pos) - t0 - g;
#pragma unroll
                        for (int n = 0; n < 4 * HV; n++)
                            if (8 * n < from || 8 * n > to || !there(n / 4, n % 4)) s[x][n][c] = -INFINITY;
                    }
            }
            auto to_scores = [&] {
#pragma unroll
                for (int x = 0; x < RT; x++)
#pragma unroll
                    for (int i = 0; i < 8 * HV; i++) s[x][i >> 1][i & 1] = __fmul_rn(s[x][i >> 1][i & 1], rs[x][i & 1]);
            };
            if (large) to_scores();
            // a score too far above m: m moves
            float mx[RT][2];
            bool above = false;
#pragma unroll
            for (int x = 0; x < RT; x++)
#pragma unroll
                for (int c = 0; c < 2; c++) {
                    mx[x][c] = fmaxf(fmaxf(s[x][0][c], s[x][1][c]), fmaxf(s[x][2][c], s[x][3][c]));
                    if (HV == 2) mx[x][c] = fmaxf(mx[x][c], fmaxf(fmaxf(s[x][4 * HV - 4][c], s[x][4 * HV - 3][c]), fmaxf(s[x][4 * HV - 2][c], s[x][4 * HV - 1][c])));
                    if (!large) mx[x][c] = __fmul_rn(mx[x][c], rs[x][c]);
                    above |= mx[x][c] - m[x][c] > 15.f;   // (-inf less -inf is not)
                }
            if (__any_sync(0xffffffffu, above)) {
                bool far = false;
#pragma unroll
                for (int x = 0; x < RT; x++)
#pragma unroll
                    for (int c = 0; c < 2; c++) {
                        float q = mx[x][c];
                        q = fmaxf(q, __shfl_xor_sync(0xffffffffu, q, 4));
                        q = fmaxf(q, __shfl_xor_sync(0xffffffffu, q, 8));
                        q = fmaxf(q, __shfl_xor_sync(0xffffffffu, q, 16));
                        if (q - m[x][c] > 15.f) {
                            const float near = q - 11.f, to = q - near > 15.f ? q : near;   // (where its rounding is 16)
                            const float corr = ex2(m[x][c] - to);
                            l[x][c] *= corr, m[x][c] = to;
#pragma unroll
                            for (int b = 0; b < NB; b++)
#pragma unroll
                                for (int y = 0; y < 2; y++) acc[b][y][x][c] *= corr, acc[b][y][x][2 + c] *= corr;
                        }
                        far |= m[x][c] >= 0x1p17f || (m[x][c] <= -0x1p17f && m[x][c] > -INFINITY);
                    }
                if (!large && __any_sync(0xffffffffu, far)) {
                    large = true;
                    to_scores();
                }
            }
            uint32_t p[RT][4 * HV];   // weights, of row g: tokens 8 n + 2 t4, + 1
#pragma unroll
            for (int x = 0; x < RT; x++) {
                float w[4 * HV][2];
#pragma unroll
                for (int c = 0; c < 2; c++) {
                    const float k = large ? 1.f : rs[x][c], ms = m[x][c] == -INFINITY ? 0.f : m[x][c];
                    float sum = 0.f;
#pragma unroll
                    for (int n = 0; n < 4 * HV; n++) sum += w[n][c] = ex2(fmaf(s[x][n][c], k, -ms));
                    l[x][c] += sum;
                }
#pragma unroll
                for (int n = 0; n < 4 * HV; n++) p[x][n] = turn8(pack_f16(w[n][0], w[n][1]));
            }
            // block b's values of half v times the weights, added to `to`
            auto values = [&](int v, int b, float (&to)[2][RT][4]) {
                uint32_t sv[4], vw[4];
                lds128(scratch + v * (NB * 192) + NB * 128 + 64 * b + 16 * t4, sv);
                ldsm4t(vw, rows_at + v * kRowsOn + P * D / 2 + b * (P * 16));
#pragma unroll
                for (int kk = 0; kk < 2; kk++) {
                    // tokens of a word's halves side by side: dims 4 g and 4 g + 2 of two octets, 4 g + 1 and 4 g + 3
                    const uint32_t lo = __byte_perm(vw[2 * kk], vw[2 * kk + 1], 0x5410), hi = __byte_perm(vw[2 * kk], vw[2 * kk + 1], 0x7632);
                    uint32_t h0[4], h1[4];
                    e2m1x8_to_f16((lo & 0x0F0F0F0Fu) | (hi << 4 & 0xF0F0F0F0u), h0);
                    e2m1x8_to_f16((lo >> 4 & 0x0F0F0F0Fu) | (hi & 0xF0F0F0F0u), h1);
#pragma unroll
                    for (int x = 0; x < RT; x++) {
                        const uint32_t p0 = mul_f16(p[x][4 * v + 2 * kk], sv[2 * kk]), p1 = mul_f16(p[x][4 * v + 2 * kk + 1], sv[2 * kk + 1]);
                        mma_f16(to[0][x], h0, p0, p1);
                        mma_f16(to[1][x], h1, p0, p1);
                    }
                }
            };
            if (!wild) {
#pragma unroll
                for (int b = 0; b < NB; b++)
#pragma unroll
                    for (int v = 0; v < HV; v++) values(v, b, acc[b]);
            } else {
                // classes of scales, the largest first; each one's products apart
#pragma unroll
                for (int v = 0; v < HV; v++) {
                    uint32_t left = vs[v];
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
                        scale_values(v, left & in, top);
                        left &= ~in;
                        __syncwarp();
                        const float k = pow2i(top - E);
#pragma unroll
                        for (int b = 0; b < NB; b++) {
                            float apart[2][RT][4];
                            const float kb = of_block(k, b);
#pragma unroll
                            for (int i = 0; i < 2 * RT * 4; i++) (&apart[0][0][0])[i] = 0.f;
                            values(v, b, apart);
#pragma unroll
                            for (int i = 0; i < 2 * RT * 4; i++) (&acc[b][0][0][0])[i] = fmaf((&apart[0][0][0])[i], kb, (&acc[b][0][0][0])[i]);
                        }
                    }
                }
            }
            __syncwarp();   // the scales are read
        }
        __syncwarp();   // the stage is read: the next iteration fills it
        if (u + 1 == seg_end) {
            const Job j = jobs[warp][stage];
            begun = false;
            const bool begins = spans[warp].seg0 == j.u0, ends = u + 1 == j.u0 + j.nt;
#pragma unroll
            for (int x = 0; x < RT; x++)
#pragma unroll
                for (int c = 0; c < 2; c++) {
                    l[x][c] += __shfl_xor_sync(0xffffffffu, l[x][c], 4);
                    l[x][c] += __shfl_xor_sync(0xffffffffu, l[x][c], 8);
                    l[x][c] += __shfl_xor_sync(0xffffffffu, l[x][c], 16);
                }
            float N[NB];   // the accumulator's unit over that of l: 2^N
#pragma unroll
            for (int b = 0; b < NB; b++) N[b] = (float)(of_block(E, b) - 127);
            if (begins && ends) {
                // the whole job was this warp's
                int row0, n, pos0;
                kv8_rows(a, j.b, row0, n, pos0);
#pragma unroll
                for (int x = 0; x < RT; x++)
#pragma unroll
                    for (int c = 0; c < 2; c++) {
                        const int rr = j.rt * R + 8 * x + 2 * t4 + c;
                        if (rr >= n * f.G) continue;
                        const int head = j.h * f.G + rr % f.G;
                        const float sink = a.sinks ? a.sinks[head] * kLog2e : -INFINITY;
                        uint16_t *o = a.out + (long long)(row0 + rr / f.G) * a.o_stride + head * D + 4 * g;
#pragma unroll
                        for (int b = 0; b < NB; b++) {
                            const float2 k = row_factor(m[x][c], l[x][c], N[b], sink);
                            auto put = [&](float y, float z) {
                                const __nv_bfloat162 v = __floats2bfloat162_rn(y * k.x * k.y, z * k.x * k.y);
                                return *reinterpret_cast<const uint32_t *>(&v);
                            };
                            *reinterpret_cast<uint2 *>(o + 32 * b) = make_uint2(put(acc[b][0][x][c], acc[b][1][x][c]), put(acc[b][0][x][2 + c], acc[b][1][x][2 + c]));
                        }
                    }
            } else {
                // a head of more to come goes to its own place, the last segment over
                // the ring, whose copies have all landed and been read
                const bool last = u + 1 == u1;
                float *to = last ? reinterpret_cast<float *>(ring) : part + (size_t)warp * PF;
#pragma unroll
                for (int x = 0; x < RT; x++)
#pragma unroll
                    for (int c = 0; c < 2; c++) {
                        const int r = 8 * x + 2 * t4 + c;
#pragma unroll
                        for (int b = 0; b < NB; b++)
                            *reinterpret_cast<float4 *>(to + r * PAD + 32 * b + 4 * g) = make_float4(acc[b][0][x][c], acc[b][1][x][c], acc[b][0][x][2 + c], acc[b][1][x][2 + c]);
                        float *ml = to + R * PAD + r;
                        if (g == 0) {
                            ml[0] = m[x][c], ml[R] = l[x][c];
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

    const int c0 = share[0], c1 = share[1], all_units = share[2] * a.c.KVH, all_ctas = min((int)gridDim.x, (all_units + 3) / 4);   // (as above)

    // Joining: the CTA's segments in order, those of one job a group (they are
    // neighbours); then, of the jobs that other CTAs share (at most the first
    // and the last), those whose other partials are all there.  Either time all
    // groups at once, for eight rows after the others: the partials' m, l and N
    // side by side in shared memory, then a thread for each group, row and pair
    // of dims.
    auto scal = [&](int k) {   // SC floats, behind the tails in the rings
        return reinterpret_cast<float *>(smem_raw + (size_t)(k % W) * RING) + PF + k / W * SC;
    };
    auto scalars = [&](int k, const float *from, int x) {
        for (int y = lane; y < SC; y += 32) scal(k)[y] = *(volatile const float *)(from + R * PAD + y / 8 * R + 8 * x + y % 8);
    };
    // partials k0 .. k0 + n - 1 (at(k)) of segment sg's job: row r (8 x + r8), dims d, d + 1
    auto join = [&](const Seg &sg, int k0, int n, auto at, bool done, int x, int r8, int d) {
        const int r = 8 * x + r8;
        int row0, nr, pos0;
        kv8_rows(a, sg.b, row0, nr, pos0);
        if (r >= min(R, nr * f.G - sg.rt * R)) return;
        const int nb = (2 + d / 32) * 8 + r8;   // where a partial's N of the block is
        float mm = -INFINITY, NN = -INFINITY, ll = 0.f;
#pragma unroll 4
        for (int k = k0; k < k0 + n; k++) mm = fmaxf(mm, scal(k)[r8]);
        const float ms = mm == -INFINITY ? 0.f : mm;
#pragma unroll 4
        for (int k = k0; k < k0 + n; k++) NN = fmaxf(NN, scal(k)[r8] - ms + scal(k)[nb]);
        const float Ns = NN == -INFINITY ? 0.f : NN;
        float2 v = make_float2(0.f, 0.f);
#pragma unroll 8
        for (int k = k0; k < k0 + n; k++) {
            const float km = scal(k)[r8], kl = scal(k)[8 + r8], kn = scal(k)[nb];
            const float c = ex2(km - ms + kn - Ns);   // no tokens: 2^-inf
            volatile const float *p = at(k) + r * PAD + d;
            v.x = fmaf(c, p[0], v.x), v.y = fmaf(c, p[1], v.y);
            ll += kl * (km == -INFINITY ? 1.f : ex2(km - ms));   // the l of NaN scores has no maximum
        }
        if (done) {
            const int rr = sg.rt * R + r, i2 = rr / f.G, head = sg.h * f.G + rr - i2 * f.G;
            const float2 k = row_factor(mm, ll, Ns, a.sinks ? a.sinks[head] * kLog2e : -INFINITY);
            *reinterpret_cast<__nv_bfloat162 *>(a.out + (long long)(row0 + i2) * a.o_stride + head * D + d) =
                __floats2bfloat162_rn(v.x * k.x * k.y, v.y * k.x * k.y);
        } else {
            float *mine_p = f.parts + ((size_t)blockIdx.x * 2 + (sg.u0 >= c0 ? 1 : 0)) * PF;
            *reinterpret_cast<float2 *>(mine_p + r * PAD + d) = v;
            if (d == 0) mine_p[R * PAD + r] = mm, mine_p[R * PAD + R + r] = ll;
            if (d % 32 == 0) mine_p[R * PAD + (2 + d / 32) * R + r] = Ns;
        }
    };
    constexpr int kCell = 8 * (D / 2);   // threads of a group
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
#pragma unroll 1
    for (int x8 = 0; x8 < RT; x8++) {
        if (x8) __syncthreads();   // the scalars before are read
        for (int k = warp; k < partials; k += W) scalars(k, here(k), x8);
        __syncthreads();
        for (int x = tid; x < groups * kCell; x += W * 32) {
            const int gi = x / kCell, k0 = group_at[gi];
            const Seg sg = segs[group_seg[gi]];
            join(sg, k0, group_at[gi + 1] - k0, here, whole_job(sg), x8, x % kCell / (D / 2), 2 * (x % (D / 2)));
        }
    }
    if (shared_seg[0] < 0 && shared_seg[1] < 0) return;   // the same for the whole CTA

    __threadfence();
    __syncthreads();
    if (tid < 2) {
        s_count[tid] = 0;
        if (shared_seg[tid] >= 0) {
            // the CTAs that share the job, by the even cuts (no cut inside it was moved)
            const Seg x = segs[shared_seg[tid]];
            const int c_first = (int)(((long long)(x.u0 + 1) * all_ctas - 1) / all_units), c_last = (int)(((long long)(x.u0 + x.nt) * all_ctas - 1) / all_units);
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
#pragma unroll 1
    for (int x8 = 0; x8 < RT; x8++) {
        if (x8) __syncthreads();
        for (int k = warp; k < n0 + n1; k += W) scalars(k, there_at(k), x8);
        __syncthreads();
        for (int x = tid; x < 2 * kCell; x += W * 32) {
            const int i = x / kCell, n = i ? n1 : n0;
            if (n) join(segs[shared_seg[i]], i ? n0 : 0, n, there_at, true, x8, x % kCell / (D / 2), 2 * (x % (D / 2)));
        }
    }
}

constexpr size_t kPartOffset = kKv8ClearBytes + (size_t)kKv8MaxSeqs * 12;

template <int D, int P, int RT>
cudaError_t few_launch(FewArgs f, int ctas, cudaStream_t st) {
    if (f.a.n_seqs <= kSmemSeqs) f.seqs = nullptr;
    const size_t smem = Few<D, P, RT>::kSmem + (f.seqs ? 0 : (size_t)f.a.n_seqs * 12);
    static PerDevice<bool> opted;
    cudaError_t e = smem_optin_once(moe_kv4_few_kernel<D, P, RT>, opted);
    if (e != cudaSuccess) return e;
    return launch_pdl(moe_kv4_few_kernel<D, P, RT>, dim3(ctas), dim3(Few<D, P, RT>::kWarps * 32), smem, st, f);
}
constexpr int kMostEights = 2;   // of a unit's rows
template <int D, int P>
cudaError_t few_rows(const FewArgs &f, int rows, int ctas, cudaStream_t st) {
    return rows <= 8 ? few_launch<D, P, 1>(f, ctas, st) : few_launch<D, P, kMostEights>(f, ctas, st);
}
template <int D>
cudaError_t few_page(const FewArgs &f, int rows, int ctas, cudaStream_t st) {
    return f.a.c.P == 16 ? few_rows<D, 16>(f, rows, ctas, st) : f.a.c.P == 32 ? few_rows<D, 32>(f, rows, ctas, st)
                                                                              : few_rows<D, 64>(f, rows, ctas, st);
}

}  // namespace

// Partials of a call: two a CTA, and one a warp.
static size_t partial_bytes(int D) { return (size_t)(D == 64 ? Few<64, 16, kMostEights>::kPartial : Few<128, 16, kMostEights>::kPartial) * 4; }

size_t kv4_workspace_bytes(int D) { return kPartOffset + (size_t)kMaxCtas * (2 + kMaxWarps) * partial_bytes(D); }

cudaError_t launch_kv4_attend(const Kv4Attend &a, unsigned char *ws, cudaStream_t st) {
    // The streaming kernel's work grows by the unit of 16 rows, that of the kernel
    // for prompts by 256 rows a CTA, which walks all keys.  Per 64 tokens of a
    // kv head the first takes 0.23 us of an SM a unit (dims of 64; 0.44 with 128),
    // the second 0.67 to 0.8 (0.95 to 1.05) a CTA of up to 128, 256 rows, in as many
    // waves as its CTAs take; some 10 us are the joins'.  us with the first and the
    // second, 8 kv heads of 64: one sequence of 32 K tokens, 128 rows 65 and 344,
    // 512 rows 198 and 414; 4 of 8 K, 256 rows 112 and 110, 512 rows 205 and 109; 32
    // of 4 K, 48 rows 93 and 102, 64 rows 116 and 97.  Of 128: one of 32 K, 512
    // rows 377 and 549; 8 of 4 K, 40 rows 67 and 66, 64 rows 80 and 66.
    int sms = 0;
    const cudaError_t e = sm_count(&sms);
    if (e != cudaSuccess) return e;
    const int G = a.QH / a.c.KVH;
    const long long rows = (long long)a.max_new * G, heads = (long long)a.n_seqs * a.c.KVH, tiles = (rows + 15) / 16;
    const long long waves = (heads * ((rows + 255) / 256) + sms - 1) / sms;
    const int tenths = a.c.D == 64 ? (rows <= 128 ? 30 : 40) : (rows <= 128 ? 16 : 21);
    const bool countable = ((long long)a.width * a.c.P / kTile + 2) * tiles * heads <= INT_MAX;   // the first's units
    if (rows <= 16 || (countable && 10 * heads * tiles < waves * sms * tenths)) {
        FewArgs f{};
        f.a = a, f.G = G, f.most_up = std::min(126, 120 + std::ilogb(a.scale * kLog2e));
        f.status = reinterpret_cast<int32_t *>(ws);
        f.tickets = reinterpret_cast<uint32_t *>(ws + 64);
        f.seqs = reinterpret_cast<int *>(ws + kKv8ClearBytes);
        f.parts = reinterpret_cast<float *>(ws + kPartOffset);
        f.heads = reinterpret_cast<float *>(ws + kPartOffset + (size_t)kMaxCtas * 2 * partial_bytes(a.c.D));
        const int ctas = std::min(sms, kMaxCtas), r = (int)std::min(rows, (long long)16);
        return a.c.D == 64 ? few_page<64>(f, r, ctas, st) : few_page<128>(f, r, ctas, st);
    }
    return launch_kv4_prompt(a, reinterpret_cast<int32_t *>(ws), st);
}
