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
// Sums are exact to about 2^-45 of the total: fp32 over the tokens that a lane
// reads at once, those in two fp32 parts, a lane's and a warp's in 64 bits.
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

struct Part {
    double sum;
    long long ties;
};

__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
__device__ __forceinline__ float used_prob(float q) { return fminf(fmaxf(q, 0.f), 1.f); }   // NaN: 0

// Rows of a cluster's CTAs in 16-byte vectors, each warp's side by side.
template <bool BF16>
__global__ void __launch_bounds__(kThreads) moe_verify_kernel(const VerifyArgs a) {
    typedef Row<BF16, false, kThreads> R;
    constexpr int VE = R::VE;
    __shared__ Part parts[2][kMaxCluster];
    __shared__ double sums[kWarps];
    __shared__ int ties[kWarps], s_count;
    cg::cluster_group cl = cg::this_cluster();
    const int rank = (int)cl.block_rank(), C = (int)cl.num_blocks();
    const int b = blockIdx.x / C, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    asm volatile("barrier.cluster.arrive.relaxed.aligned;");
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int s0 = min(max(a.s.starts[b], 0), a.s.rows), s1 = min(max(a.s.starts[b + 1], s0), a.s.rows);
    const float t = used_temperature(a.s.temperature ? a.s.temperature[b] : 1.f);
    const float mp = a.s.min_p ? used_min_p(a.s.min_p[b]) : 0.f;
    const int n = s1 - s0;
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");   // every CTA of the sequence runs
    if (n == 0) {
        if (rank == 0 && tid == 0) a.accepted[b] = 0;
        return;
    }
    auto logit = [&](int row, int i) {
        const long long at = row * a.s.stride + i;
        return BF16 ? bf16_to_f32(__ldg(reinterpret_cast<const uint16_t *>(a.s.x) + at)) : __ldg(reinterpret_cast<const float *>(a.s.x) + at);
    };
    auto row_of = [&](int row) {
        R d;
        const uintptr_t at = (uintptr_t)a.s.x + (size_t)row * a.s.stride * (BF16 ? 2 : 4);
        d.g = reinterpret_cast<const uint4 *>(at & ~(uintptr_t)15);
        d.off = (int)(at & 15) / (BF16 ? 2 : 4);
        d.V = a.s.V, d.s = nullptr;
        return d;
    };

    // the drafted tokens, 32 rows at a time: accepted, not, or (2) among the tokens at T, of which some are left out
    int j0 = 0;
    for (bool more = true; more && j0 < n - 1;) {
        const int j = j0 + lane;
        int state = 0;
        if (j < n - 1) {
            const SampleLimits lim = a.s.limits[s0 + j];
            const int x = a.drafts[s0 + j];
            if (x >= 0 && x < a.s.V && lim.top) {
                const float l = logit(s0 + j, x);
                const uint32_t key = order_key(l);
                const Weight weight(key_logit(lim.top), t);
                const float w = weight(l), q = a.probs ? used_prob(__ldg(a.probs + (s0 + j) * a.probs_stride + x)) : 1.f;
                const bool in = key >= max(lim.T, 1u) && w > 0.f && (mp < 1.f ? w >= mp * weight(weight.top) : key == lim.top);
                if (in && (double)a.u[s0 + j] * q * lim.total < w) state = key == lim.T && lim.cut ? 2 : 1;
            }
        }
        const unsigned stop = __ballot_sync(0xffffffffu, state != 1);
        if (!stop) {
            j0 += 32;
            continue;
        }
        const int at = __ffs(stop) - 1;
        j0 += at;
        if (j0 >= n - 1 || __shfl_sync(0xffffffffu, state, at) == 0) break;
        // is it among the first r tokens at T?
        const SampleLimits lim = a.s.limits[s0 + j0];
        const int x = a.drafts[s0 + j0];
        const float xT = key_logit(lim.T);
        __syncthreads();
        if (tid == 0) s_count = 0;
        __syncthreads();
        R d = row_of(s0 + j0);
        int found = 0;
        for (int v = tid; v * VE - d.off < x; v += kThreads) {
            float y[VE];
            R::values(d.fetch(v), y);
#pragma unroll
            for (int e = 0; e < VE; e++) found += y[e] == xT && v * VE - d.off + e < x;
        }
        found = __reduce_add_sync(0xffffffffu, found);
        if (lane == 0) atomicAdd(&s_count, found);
        __syncthreads();
        more = s_count < lim.r;
        j0 += more;
    }
    j0 = min(j0, n - 1);

    // the draw at row j0
    const int row = s0 + j0;
    const SampleLimits lim = a.s.limits[row];
    R d = row_of(row);
    {
        const int vecs = (d.off + d.V + VE - 1) / VE, each = (vecs + C - 1) / C;
        const int c0 = min(rank * each, vecs), c1 = min(c0 + each, vecs), per = (c1 - c0 + kWarps - 1) / kWarps;
        d.c0 = c0, d.v0 = min(c0 + warp * per, c1), d.v1 = min(d.v0 + per, c1);
    }
    if (rank == 0) {
        for (int j = tid; j < n; j += kThreads)
            if (j != j0 || !lim.top) a.ids[s0 + j] = j < j0 ? a.drafts[s0 + j] : -1;
        if (tid == 0) a.accepted[b] = j0;
    }
    if (!lim.top) return;   // nothing to draw
    const Weight weight(key_logit(lim.top), t);
    const float xT = lim.T ? key_logit(lim.T) : -INFINITY, least = mp * weight(weight.top);
    const float per_weight = (float)(1. / lim.total);
    const int x0 = a.drafts[row];
    const float *probs = a.probs + row * a.probs_stride;
    int turn = 0;
    bool minus = j0 < n - 1;   // less what the draft's probabilities are
    // what token i with logit x adds; rank_T: tokens at T before it
    auto adds = [&](float x, int i, int &rank_T) {
        bool in = x > xT;
        if (x == xT && lim.T) in = rank_T++ < lim.r;
        if (!in) return 0.f;
        const float w = weight(x);
        if (!(mp < 1.f ? w >= least : x == weight.top)) return 0.f;
        const float q = !minus ? 0.f : a.probs ? used_prob(__ldg(probs + i)) : i == x0 ? 1.f : 0.f;
        return fmaxf(fmaf(w, per_weight, -q), 0.f);
    };
    int tie0 = 0;   // tokens at T before this warp's part, where that counts
    if (lim.cut) {
        int mine = 0;
        d.each([&](float (&x)[VE], int) {
#pragma unroll
            for (int e = 0; e < VE; e++) mine += x[e] == xT;
        });
        mine = __reduce_add_sync(0xffffffffu, mine);
        if (lane == 0) ties[warp] = mine;
        __syncthreads();
        int all = 0;
        for (int w = 0; w < kWarps; w++) {
            if (w < warp) tie0 += ties[w];
            all += ties[w];
        }
        if (tid < C) cl.map_shared_rank(&parts[turn][rank], tid)->ties = all;
        cl.sync();
        for (int c = 0; c < rank; c++) tie0 += (int)parts[turn][c].ties;
    }
    for (int attempt = 0; attempt < 2; attempt++) {
        // 32 vectors at a time, a lane a vector, f(the lane's sum, its tokens' shares)
        auto walk = [&](auto f) {
            int rank_T = tie0;
            for (int v = d.v0; v < d.v1; v += 32) {
                float x[VE], y[VE];
                if (v + lane < d.v1) {
                    R::values(d.fetch(v + lane), x);
                } else {
#pragma unroll
                    for (int e = 0; e < VE; e++) x[e] = -INFINITY;
                }
                int mine = 0;
                if (lim.cut) {
                    int at = 0;
#pragma unroll
                    for (int e = 0; e < VE; e++) at += x[e] == xT;
                    mine = rank_T;
                    if (__any_sync(0xffffffffu, at)) {
                        int inc = at;
#pragma unroll
                        for (int o = 1; o < 32; o <<= 1) {
                            const int z = __shfl_up_sync(0xffffffffu, inc, o);
                            if (lane >= o) inc += z;
                        }
                        mine += inc - at;
                        rank_T += __shfl_sync(0xffffffffu, inc, 31);
                    }
                }
                float sum = 0.f;
                const int i = (v + lane) * VE - d.off;
#pragma unroll
                for (int e = 0; e < VE; e++) y[e] = adds(x[e], i + e, mine), sum += y[e];
                if (f(sum, y, i)) return;
            }
        };
        float hi = 0.f, lo = 0.f;
        walk([&](float sum, const float (&)[VE], int) {
            const float s = hi + sum, z = s - hi;
            lo += (hi - (s - z)) + (sum - z);
            hi = s;
            return false;
        });
        const double mine = warp_sum((double)hi + lo);
        if (lane == 0) sums[warp] = mine;
        __syncthreads();
        turn ^= 1;
        // where the CTA's share of the running sum begins, and the warp's: sums in
        // one order, so that each ends where the next begins
        double at = 0., end = 0.;
        for (int w = 0; w < kWarps; w++) {
            if (w < warp) at += sums[w];
            end += sums[w];
        }
        if (tid < C) cl.map_shared_rank(&parts[turn][rank], tid)->sum = end;
        cl.sync();
        double total = 0., base = 0., next = 0.;
        for (int c = 0; c < C; c++) {
            if (c == rank) base = total;
            total += parts[turn][c].sum;
            if (c == rank) next = total;
        }
        if (!(total > 0.)) {
            if (minus) {   // p is nowhere above q: from p
                minus = false;
                continue;
            }
            if (rank == 0 && tid == 0) a.ids[row] = -1;
            return;
        }
        end = warp == kWarps - 1 ? next : base + (at + sums[warp]);
        at = base + at;
        const double target = (double)fminf(fmaxf(a.draws[b], 0.f), 0.99999994f) * total;   // below the total
        if (target < at || target >= end) return;
        int last = -1, id = -1;
        walk([&](float, const float (&y)[VE], int i) {
            double s = 0.;
#pragma unroll
            for (int e = 0; e < VE; e++) {
                s += y[e];
                if (y[e] > 0.f) last = i + e;
            }
            double inc = s;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const double z = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += z;
            }
            double run = at + inc - s;
            bool hit = false;
            if (target < at + inc && s > 0.)
#pragma unroll
                for (int e = 0; e < VE; e++) {
                    run += y[e];
                    if (!hit && y[e] > 0.f && target < run) hit = true, id = i + e;
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
    int C = kMaxCluster;
    while (C > 1 && ((long long)a.s.n_seqs * C > 2 * 152 || vecs / C < 256)) C /= 2;
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
