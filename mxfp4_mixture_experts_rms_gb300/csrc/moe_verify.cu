// moe_verify.cu -- drafted tokens against the target model's logits.
//
// With p_j the distribution from which moe_sample would draw at row j of a
// sequence and q_j the one that its drafted token x_j was drawn from, x_j is
// accepted where u_j q_j(x_j) < p_j(x_j), and the first row whose token is not
// draws from max(p - q, 0): then each token has the probability that p gives
// it.  Two kernels: the first (moe_sample.cu) finds the limits of what every
// row keeps and its weight, the second, a cluster a sequence, looks at the
// drafted tokens' logits alone, and reads one row, that of the draw, twice: for
// the sums of each warp's part, and in the part that holds the chosen token.
// q is read at kept tokens only.
//
// Sums are whole numbers of units of 2^-52, at least one where there is anything:
// of a lane's tokens, summed in two fp32 parts.  Where that comes to less than
// 2^36 units (q is p but for last bits) the row is summed again in smaller ones.
// (64-bit floats are the GPU's slowest numbers: with sums and quotients in them the
// second kernel took 76 us at 64 sequences, 282 rows of 128 K logits, in place of
// 38; the first takes 100, as moe_sample would.)
#include "moe_sample.cuh"
#include "../../include/moe.h"

#include <cooperative_groups.h>

#include <algorithm>
#include <climits>

namespace cg = cooperative_groups;

namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;

struct VerifyArgs {
    SampleArgs s;
    const int32_t *drafts;   // [rows]
    const float *probs;      // rows of probs_stride, or null: a drafted token was certain
    long long probs_stride;
    const float *u, *draws;  // [rows], [n_seqs]
    int32_t *ids, *accepted;
};

typedef unsigned long long u64;
__device__ __forceinline__ u64 warp_sum(u64 v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
// x (0 .. 1 and a little more) in units of 2^-(52 + up), at least one of them if it is not 0.
__device__ __forceinline__ u64 units(float x, int up) {
    const uint32_t b = __float_as_uint(x);
    const int s = (int)(b >> 23) - 98 + up;   // mantissa times 2^(exponent - 150)
    const u64 m = (b & 0x7FFFFFu) | 0x800000u;
    return x > 0.f ? max(s >= 0 ? m << min(s, 38) : m >> min(-s, 63), (u64)1) : 0;
}
// u (0 .. 1 - 2^-24; NaN: 0) in units of 2^-64.
__device__ __forceinline__ u64 fraction(float u) {
    const uint32_t b = __float_as_uint(fminf(fmaxf(u, 0.f), 0.99999994f));
    const int s = (int)(b >> 23) - 86;
    const u64 m = (b & 0x7FFFFFu) | 0x800000u;
    return s >= 0 ? m << s : m >> min(-s, 63);
}
__device__ __forceinline__ float used_prob(float q) { return fminf(fmaxf(q, 0.f), 1.f); }   // NaN: 0

// A cluster a sequence; of the row of the draw each CTA has a part, each of its
// warps one of that.
template <bool BF16>
__global__ void __launch_bounds__(kThreads, 2) moe_verify_kernel(const VerifyArgs a) {
    typedef Row<BF16, false, kThreads> R;
    constexpr int VE = R::VE, U = BF16 ? 2 : 4;   // logits of a vector; vectors that a lane loads at once
    __shared__ u64 parts[2][kMaxCluster], sums[kWarps];
    __shared__ int s_row;
    cg::cluster_group cl = cg::this_cluster();
    const int rank = (int)cl.block_rank(), C = (int)cl.num_blocks();
    const int b = blockIdx.x / C, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    asm volatile("barrier.cluster.arrive.relaxed.aligned;");
    asm volatile("griddepcontrol.launch_dependents;");
    // What the first kernel does not write is read before it has ended: it lets
    // this one start only when all before it are done.
    const int s0 = min(max(a.s.starts[b], 0), a.s.rows), s1 = min(max(a.s.starts[b + 1], s0), a.s.rows);
    const float t = used_temperature(a.s.temperature ? a.s.temperature[b] : 1.f);
    const float mp = a.s.min_p ? used_min_p(a.s.min_p[b]) : 0.f;
    const int n = s1 - s0;
    const float draw = n > 0 ? a.draws[b] : 0.f;
    // of row s0 + j: the drafted token (-1: none, or not in the vocabulary), its logit and probability, the random number
    struct Draft {
        int x;
        float l, q, u;
    };
    auto draft = [&](int j) {
        Draft d{-1, 0.f, 0.f, 0.f};
        if (j < n - 1) {
            const int row = s0 + j;
            d.x = a.drafts[row], d.u = a.u[row];
            if (d.x < 0 || d.x >= a.s.V) d.x = -1;
            if (d.x >= 0) {
                const long long at = row * a.s.stride + d.x;
                d.l = BF16 ? bf16_to_f32(__ldg(reinterpret_cast<const uint16_t *>(a.s.x) + at)) : __ldg(reinterpret_cast<const float *>(a.s.x) + at);
                d.q = a.probs ? used_prob(__ldg(a.probs + row * a.probs_stride + d.x)) : 1.f;
            }
        }
        return d;
    };
    Draft d{-1, 0.f, 0.f, 0.f};
    if (warp == 0) d = draft(lane);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");   // every CTA of the sequence runs
    if (n == 0) {
        if (rank == 0 && tid == 0) a.accepted[b] = 0;
        return;
    }
    // the first row whose token is not accepted, 32 rows at a time
    if (warp == 0) {
        for (int j = 0;; j += 32, d = draft(j + lane)) {
            bool ok = false;
            if (d.x >= 0) {
                const SampleLimits lim = a.s.limits[s0 + j + lane];
                const uint32_t key = order_key(d.l);
                if (lim.top) {
                    const Weight<true> weight(key_logit(lim.top), t);
                    const float w = weight(d.l), uq = d.u * d.q;
                    const bool in = (key > lim.T || (key == lim.T && d.x < lim.cut)) && key && w > 0.f && (mp < 1.f ? w >= lim.least : key == lim.top);
                    ok = in && fmaf(w, lim.inv, -uq) + fmaf(w, lim.inv_lo, -fmaf(d.u, d.q, -uq)) > 0.f;   // u q < w inv
                }
            }
            const unsigned stop = __ballot_sync(0xffffffffu, !ok);
            if (stop) {
                if (lane == 0) s_row = j + __ffs(stop) - 1;
                break;
            }
        }
    }
    __syncthreads();
    const int j0 = s_row;

    // the draw at row j0 (at most n - 1)
    const int row = s0 + j0;
    const SampleLimits lim = a.s.limits[row];
    R r;
    {
        const uintptr_t at = (uintptr_t)a.s.x + (size_t)row * a.s.stride * (BF16 ? 2 : 4);
        r.g = reinterpret_cast<const uint4 *>(at & ~(uintptr_t)15);
        r.off = (int)(at & 15) / (BF16 ? 2 : 4);
        r.V = a.s.V, r.s = nullptr;
        const int vecs = (r.off + r.V + VE - 1) / VE, each = (vecs + C - 1) / C;
        const int c0 = min(rank * each, vecs), c1 = min(c0 + each, vecs), per = (c1 - c0 + kWarps - 1) / kWarps;
        r.c0 = c0, r.v0 = min(c0 + warp * per, c1), r.v1 = min(r.v0 + per, c1);
    }
    if (rank == 0) {
        for (int j = tid; j < n; j += kThreads)
            if (j != j0 || !lim.top) a.ids[s0 + j] = j < j0 ? a.drafts[s0 + j] : -1;
        if (tid == 0) a.accepted[b] = j0;
    }
    if (!lim.top) return;   // nothing to draw
    const Weight<true> weight(key_logit(lim.top), t);
    const float xT = lim.T ? key_logit(lim.T) : -INFINITY;
    const int cut = lim.T ? lim.cut : 0;   // (of logits of -inf none)
    const int x0 = j0 < n - 1 ? a.drafts[row] : -1;
    const float *probs = a.probs + row * a.probs_stride;
    bool minus = j0 < n - 1;   // less what the draft's probabilities are
    const bool whole = a.probs && ((uintptr_t)(probs - r.off) & 15u) == 0;   // a vector's probabilities are vectors
    // the draft's probabilities of a vector's tokens, the first being i
    auto drafted_q = [&](int i, float (&q)[VE]) {
        if (whole && i >= 0 && i + VE <= r.V) {
#pragma unroll
            for (int e = 0; e < VE; e += 4) {
                const float4 f = __ldg(reinterpret_cast<const float4 *>(probs + i + e));
                q[e] = f.x, q[e + 1] = f.y, q[e + 2] = f.z, q[e + 3] = f.w;
            }
        } else {
#pragma unroll
            for (int e = 0; e < VE; e++) q[e] = i + e >= 0 && i + e < r.V ? __ldg(probs + i + e) : 0.f;
        }
    };
    // U vectors a lane at a time: f(index of the first token, what its tokens add, and their sum)
    auto walk = [&](auto f) {
        for (int v = r.v0; v < r.v1; v += 32 * U) {
            uint4 w[U];
            float q[U][VE];
            bool some[U];   // are there tokens that may be kept?
#pragma unroll
            for (int u = 0; u < U; u++) w[u] = v + 32 * u + lane < r.v1 ? r.fetch(v + 32 * u + lane) : BF16 ? make_uint4(0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u)
                                                                                                             : make_uint4(0xFF800000u, 0xFF800000u, 0xFF800000u, 0xFF800000u);
#pragma unroll
            for (int u = 0; u < U; u++) {
                float x[VE], top = -INFINITY;
                R::values(w[u], x);
#pragma unroll
                for (int e = 0; e < VE; e++) top = fmaxf(top, x[e]);   // NaN passes over
                some[u] = top > -INFINITY && top >= xT;
                const int i = (v + 32 * u + lane) * VE - r.off;
#pragma unroll
                for (int e = 0; e < VE; e++) q[u][e] = minus && i + e == x0 && !a.probs ? 1.f : 0.f;
                if (some[u] && minus && a.probs) drafted_q(i, q[u]);
            }
#pragma unroll
            for (int u = 0; u < U; u++) {
                const int i = (v + 32 * u + lane) * VE - r.off;
                float x[VE], y[VE], sum = 0.f;
                R::values(w[u], x);
#pragma unroll
                for (int e = 0; e < VE; e++) {
                    y[e] = 0.f;
                    if (some[u] && (x[e] > xT || (x[e] == xT && i + e < cut))) {
                        const float w = weight(x[e]);
                        // (what p and q have in common goes first, so that inv_lo still shows in what is left)
                        if (mp < 1.f ? w >= lim.least : x[e] == weight.top) y[e] = fmaxf(fmaf(w, lim.inv_lo, fmaf(w, lim.inv, -used_prob(q[u][e]))), 0.f);
                    }
                    sum += y[e];
                }
                if (f(i, y, sum)) return;
            }
        }
    };
    int up = 0;   // of the units
    for (int turn = 0; turn < 2; turn++) {
        float hi = 0.f, lo = 0.f;
        walk([&](int, const float (&)[VE], float sum) {
            const float s = hi + sum, z = s - hi;
            lo += (hi - (s - z)) + (sum - z);
            hi = s;
            return false;
        });
        // (lo is a correction of either sign, below half a unit in hi's last place)
        const u64 mine = warp_sum(lo >= 0.f ? units(hi, up) + (lo > 0.f ? units(lo, up) : 0) : max(units(hi, up) - min(units(-lo, up), units(hi, up)), (u64)1));
        if (lane == 0) sums[warp] = mine;
        __syncthreads();
        u64 at = 0, all = 0;
        for (int w = 0; w < kWarps; w++) {
            if (w < warp) at += sums[w];
            all += sums[w];
        }
        if (tid < C) *cl.map_shared_rank(&parts[turn][rank], tid) = all;
        cl.sync();
        u64 total = 0;
        for (int c = 0; c < C; c++) {
            if (c < rank) at += parts[turn][c];
            total += parts[turn][c];
        }
        if (total < 1ull << 36 && minus && turn == 0) {
            if (total == 0) minus = false;   // p is nowhere above q: from p
            else up = __clzll((long long)total) - 2;   // a sum below 2^62
            continue;
        }
        if (total == 0) {
            if (rank == 0 && tid == 0) a.ids[row] = -1;
            return;
        }
        const u64 target = __umul64hi(total, fraction(draw));   // below the total
        if (target < at || target >= at + mine) return;
        int last = -1, id = -1;
        walk([&](int i, const float (&y)[VE], float sum) {
            if (!__any_sync(0xffffffffu, sum > 0.f)) return false;
            u64 s = 0;
#pragma unroll
            for (int e = 0; e < VE; e++) {
                s += units(y[e], up);
                if (y[e] > 0.f) last = i + e;
            }
            u64 inc = s;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const u64 z = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += z;
            }
            u64 run = at + inc - s;
            const bool hit = target >= run && target < run + s;
            if (hit)
#pragma unroll
                for (int e = 0; e < VE; e++) {
                    const u64 one = units(y[e], up);
                    if (target >= run && target < run + one) id = i + e;
                    run += one;
                }
            const unsigned who = __ballot_sync(0xffffffffu, hit);
            at += __shfl_sync(0xffffffffu, inc, 31);
            if (who) id = __shfl_sync(0xffffffffu, id, __ffs(who) - 1);
            return who != 0;
        });
        if (id < 0) id = __reduce_max_sync(0xffffffffu, last);   // (the parts' sums were rounded otherwise)
        if (lane == 0) a.ids[row] = id;
        return;
    }
}

template <bool BF16>
cudaError_t verify_launch(const VerifyArgs &a, cudaStream_t st) {
    const long long vecs = ((long long)a.s.V + (BF16 ? 7 : 3)) / (BF16 ? 8 : 4) + 1;
    int sms = 0, C = kMaxCluster;
    const cudaError_t e = sm_count(&sms);
    if (e != cudaSuccess) return e;
    while (C > 1 && ((long long)a.s.n_seqs * C > 2 * sms || vecs / C < 256)) C /= 2;   // (two CTAs an SM)
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)a.s.n_seqs * C);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = C, attr[1].val.clusterDim.y = 1, attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, moe_verify_kernel<BF16>, a);
}

}  // namespace

extern "C" {

size_t moe_verify_workspace_bytes(int n_rows) { return n_rows > 0 ? (size_t)n_rows * sizeof(SampleLimits) : 0; }

int moe_verify(const void *logits, int is_bf16, int n_rows, int vocab, long long row_stride, const int32_t *drafts,
               const float *draft_probs, long long probs_stride, const int32_t *starts, int n_seqs, const float *temperature,
               const int32_t *top_k, const float *top_p, const float *min_p, const float *u, const float *draws, int32_t *ids,
               int32_t *accepted, void *workspace, size_t workspace_bytes, void *stream) {
    if (n_rows < 0 || n_rows > (1 << 24) || vocab < 1 || vocab > (1 << 22) || n_seqs < 0 || n_seqs > 65536)
        return moe_fail_status(MOE_EINVAL, "n_rows must be 0..2^24, vocab 1..2^22 and n_seqs 0..65536");
    if (is_bf16 != 0 && is_bf16 != 1) return moe_fail_status(MOE_EINVAL, "is_bf16 must be 0 or 1");
    if (n_seqs == 0) return MOE_OK;
    if (!starts || !accepted || (n_rows && (!logits || !drafts || !u || !draws || !ids || !workspace)))
        return moe_fail_status(MOE_EINVAL, "NULL logits, drafts, starts, u, draws, ids, accepted or workspace");
    if (row_stride < vocab || (draft_probs && probs_stride < vocab))
        return moe_fail_status(MOE_EINVAL, "row_stride and probs_stride must be at least vocab");
    if ((uintptr_t)logits & (is_bf16 ? 1u : 3u)) return moe_fail_status(MOE_EINVAL, "misaligned logits");
    if (((uintptr_t)drafts | (uintptr_t)draft_probs | (uintptr_t)starts | (uintptr_t)temperature | (uintptr_t)top_k | (uintptr_t)top_p |
         (uintptr_t)min_p | (uintptr_t)u | (uintptr_t)draws | (uintptr_t)ids | (uintptr_t)accepted) & 3u)
        return moe_fail_status(MOE_EINVAL, "pointers must be 4-byte aligned");
    if ((uintptr_t)workspace & 15u) return moe_fail_status(MOE_EINVAL, "the workspace must be 16-byte aligned");
    if (workspace_bytes < moe_verify_workspace_bytes(n_rows))
        return moe_fail_status(MOE_ENOMEM, "workspace of %zu bytes, %zu needed", workspace_bytes, moe_verify_workspace_bytes(n_rows));
    // what one row's or sequence's CTAs write others may still have to read
    struct Array {
        const void *p;
        long long row, stride, n;   // bytes of a row, from row to row; rows
    };
    auto clash = [](const Array &x, const Array &y) {   // y: one row
        if (!x.p || !y.p || x.n <= 0 || y.n <= 0 || !y.row) return false;
        const uintptr_t xa = (uintptr_t)x.p, ya = (uintptr_t)y.p;
        if (ya + y.row <= xa || xa + (x.n - 1) * x.stride + x.row <= ya) return false;
        const long long at = ya < xa ? 0 : (long long)((ya - xa) % x.stride);   // in a row, or behind its end
        return at < x.row || at + y.row > x.stride;
    };
    auto flat = [](const void *p, long long n) { return Array{p, 4 * n, 4 * n, n > 0}; };
    const long long size = is_bf16 ? 2 : 4;
    const Array out[] = {flat(ids, n_rows), flat(accepted, n_seqs), {workspace, (long long)moe_verify_workspace_bytes(n_rows), 1, n_rows > 0}};
    const Array in[] = {flat(drafts, n_rows), flat(u, n_rows), flat(starts, n_seqs + 1), flat(draws, n_seqs), flat(temperature, n_seqs),
                        flat(top_k, n_seqs), flat(top_p, n_seqs), flat(min_p, n_seqs), {logits, vocab * size, row_stride * size, n_rows},
                        {draft_probs, vocab * 4ll, probs_stride * 4, n_rows}};
    for (int o = 0; o < 3; o++) {
        for (int i = 0; i < o; i++)
            if (clash(out[i], out[o])) return moe_fail_status(MOE_EINVAL, "ids, accepted and the workspace must not overlap");
        for (const Array &x : in)
            if (clash(x, out[o])) return moe_fail_status(MOE_EINVAL, "ids, accepted and the workspace must not overlap an input");
    }
    VerifyArgs a{};
    a.s.x = logits, a.s.rows = n_rows, a.s.V = vocab, a.s.stride = row_stride;
    a.s.temperature = temperature, a.s.top_k = top_k, a.s.top_p = top_p, a.s.min_p = min_p;
    a.s.starts = starts, a.s.n_seqs = n_seqs, a.s.limits = static_cast<SampleLimits *>(workspace);
    a.drafts = drafts, a.probs = draft_probs, a.probs_stride = probs_stride, a.u = u, a.draws = draws, a.ids = ids, a.accepted = accepted;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e = n_rows ? launch_sample_limits(a.s, is_bf16, st) : cudaSuccess;
    if (e == cudaSuccess) e = is_bf16 ? verify_launch<true>(a, st) : verify_launch<false>(a, st);
    return e == cudaSuccess ? MOE_OK : moe_fail_status(MOE_ECUDA, "moe_verify: %s", cudaGetErrorString(e));
}

}  // extern "C"
