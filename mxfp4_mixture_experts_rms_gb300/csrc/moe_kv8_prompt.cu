// moe_kv8_prompt.cu -- attention over the 8-bit paged cache for many new
// tokens a sequence (prompts, or pieces of them): tensor-core products on
// tcgen05 with accumulators in tensor memory.
//
// One CTA per (sequence, kv head, 128 rows), a row being a new token and one of
// the kv head's query heads; 64 cached tokens a step.  Its warps:
//  * 4..7 read the step's pages (16-byte loads, the next step's on their way),
//    turn E4M3 codes into fp16 (exact) and write them as the K-major,
//    128-byte-swizzled operand tiles K [64 tokens][D] and V^T [D][64 tokens],
//    two stages;
//  * 8 (one lane) issues S = Q K^T (M 128, N 64) into one of two score buffers
//    one step ahead, and O += P V (N = D), fp32 in tensor memory;
//  * 0..3 are the softmax, a thread a row: scores by tcgen05.ld, no shuffles,
//    weights as fp16 into the P tile.
// Softmax references as in the kernel for a few tokens (m of the scores, N + m
// of score + value exponent), but moved only when a score passes one by more
// than 2^8, so that the accumulator in tensor memory is rarely rescaled:
// weights are 2^(7 + s + e - M) <= 2^15.  Two CTAs share an SM, one's softmax
// beside the other's products.  Bound by the softmax's instructions (about
// five a score) at head dims of 64.
//
// A NaN value that only some of a tile's rows see would reach the others as
// 0 * NaN: where the pages hold one in a step that not all rows see, the CTA's
// rows are computed once more, one at a time.
#include "moe_kv8.cuh"

#include <algorithm>

namespace {

constexpr int kM = 128;         // rows of a CTA
constexpr int kT = 64;          // tokens of a step
constexpr int kStages = 2;
constexpr int kThreads = 9 * 32;
constexpr uint64_t kWaitNs = 2000000000ull;
constexpr float kLog2e = 1.4426950408889634f;

template <int D>
struct Smem {   // offsets from a 1024-byte boundary
    static constexpr int kQ = 0;
    static constexpr int kP = kM * D * 2;
    static constexpr int kK = kP + kM * kT * 2;             // kStages x [64][D]
    static constexpr int kV = kK + kStages * kT * D * 2;    // kStages x [D][64]
    static constexpr int kBytes = kV + kStages * kT * D * 2;
};

__device__ __forceinline__ uint32_t smem_u32(const void *p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }
__device__ __forceinline__ uint64_t now_ns() {
    uint64_t t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}
__device__ __forceinline__ bool bar_try(uint64_t *b, uint32_t parity) {
    uint32_t ok;
    asm volatile("{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
                 : "=r"(ok) : "r"(smem_u32(b)), "r"(parity) : "memory");
    return ok != 0;
}
// Bounded wait: false (and the status word set) after about 2 s, or when a
// failure was reported elsewhere first; drain: only the time limit ends it.
__device__ bool bar_wait(uint64_t *b, uint32_t parity, int32_t *status, int where, bool drain = false) {
    if (bar_try(b, parity)) return true;
    const uint64_t t0 = now_ns();
    for (uint32_t i = 1;; i++) {
        if (bar_try(b, parity)) return true;
        if ((i & 63) == 0) {
            if (!drain && *(volatile int32_t *)status != 0) return false;
            if (now_ns() - t0 > kWaitNs) {
                set_device_error(status, MOE_DEV_WAIT_TIMEOUT, where);
                return false;
            }
        }
    }
}
__device__ __forceinline__ void bar_init(uint64_t *b, uint32_t n) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(b)), "r"(n));
}
__device__ __forceinline__ void bar_arrive(uint64_t *b) {
    asm volatile("{ .reg .b64 st; mbarrier.arrive.shared::cta.b64 st, [%0]; }" ::"r"(smem_u32(b)) : "memory");
}
__device__ __forceinline__ void commit(uint64_t *b) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(b)) : "memory");
}
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
// Operand tile: K-major, 128-byte swizzle, 8-row groups 1024 B apart.
__device__ __forceinline__ uint64_t tile_desc(uint32_t at) {
    return (uint64_t)((at >> 4) & 0x3FFFu) | (uint64_t)1 << 16 | (uint64_t)(1024 >> 4) << 32 | (uint64_t)1 << 46 | (uint64_t)2 << 61;
}
__device__ __forceinline__ uint32_t swizzled(int row, int chunk) { return (uint32_t)(row * 128 + ((chunk ^ (row & 7)) << 4)); }
// fp16 operands, fp32 accumulator, M = 128.
constexpr uint32_t inst_desc(int N) { return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(kM >> 4) << 24); }
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
    asm volatile("{ .reg .pred p; setp.ne.b32 p, %4, 0; tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p; }" ::"r"(d),
                 "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)acc));
}
// 32 consecutive columns of the thread's TMEM lane; wait_ld before their use.
__device__ __forceinline__ void tmem_ld32(uint32_t at, float (&v)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
        "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]), "=f"(v[9]),
          "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]), "=f"(v[17]), "=f"(v[18]),
          "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]), "=f"(v[25]), "=f"(v[26]), "=f"(v[27]),
          "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
        : "r"(at));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t at, const float (&v)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,"
        "%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(at),
        "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]), "f"(v[8]), "f"(v[9]), "f"(v[10]),
        "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]), "f"(v[15]), "f"(v[16]), "f"(v[17]), "f"(v[18]), "f"(v[19]), "f"(v[20]),
        "f"(v[21]), "f"(v[22]), "f"(v[23]), "f"(v[24]), "f"(v[25]), "f"(v[26]), "f"(v[27]), "f"(v[28]), "f"(v[29]), "f"(v[30]),
        "f"(v[31])
        : "memory");
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
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
__device__ __forceinline__ uint32_t bits_of(__nv_bfloat162 v) { return *reinterpret_cast<const uint32_t *>(&v); }

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
    const int last = (int)min((long long)pos, (long long)a.width * P - 1), first = a.window > 0 ? max(0, pos - a.window + 1) : 0;
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
__global__ void __launch_bounds__(kThreads, 2) moe_kv8_prompt_kernel(const __grid_constant__ PromptArgs f) {
    constexpr int NP = kT / P, KU = kT * (D / 16) / 128;   // pages of a step; 16-byte units of keys (and of values) a thread
    typedef Smem<D> L;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *smem = reinterpret_cast<unsigned char *>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    __shared__ __align__(8) uint64_t full[kStages], empty[kStages], s_full[2], q_full, p_full, o_done, drain;
    __shared__ uint32_t meta[kStages][NP];   // key exponent byte, value's, 1 if the page is there
    __shared__ uint32_t tmem_slot;
    __shared__ int job[2], odd;
    const Kv8Attend &a = f.a;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, kvh = blockIdx.y;
    if (tid == 0) {
        for (int s = 0; s < kStages; s++) bar_init(&full[s], 128), bar_init(&empty[s], 1), bar_init(&s_full[s], 1);
        bar_init(&q_full, 128), bar_init(&p_full, 128), bar_init(&o_done, 1), bar_init(&drain, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        odd = 0;
    }
    if (warp == 8) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 256;" ::"r"(smem_u32(&tmem_slot)));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (warp == 0) {
        // the blockIdx.x-th row tile: sequences in order, a sequence's last
        // (longest) tile first
        int x = blockIdx.x, found = -1, rt = 0;
        for (int b0 = 0; b0 < a.n_seqs && found < 0; b0 += 32) {
            int row0, n = 0, pos0;
            if (b0 + lane < a.n_seqs) kv8_rows(a, b0 + lane, row0, n, pos0);
            const int mine = (n * f.G + kM - 1) / kM;
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
                const int last = __shfl_sync(0xffffffffu, inc, at), cnt = __shfl_sync(0xffffffffu, mine, at);
                rt = cnt - 1 - (x - (last - cnt));
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
        const int r0 = job[1] * kM, rows = min(kM, n * f.G - r0);
        const int p_first = pos0 + r0 / f.G, p_last = pos0 + (r0 + rows - 1) / f.G;
        // tokens that any row sees, and the steps over them (aligned to 64)
        const int seen = (int)max(0ll, min((long long)p_last + 1, (long long)a.width * P));
        const int lo = a.window > 0 ? max(0, p_first - a.window + 1) : 0;
        const int step0 = lo / kT, steps = max(1, (seen + kT - 1) / kT - step0);
        int32_t *status = f.status;
        // does every row see all of the step's tokens (where their pages are)?
        auto whole = [&](int t0) { return t0 + kT <= seen && t0 + kT - 1 <= p_first && (a.window == 0 || t0 > p_last - a.window); };

        if (warp < 4) {
            // ---- the softmax ----
            const int r = tid, rr = r0 + r, i2 = rr / f.G, head = kvh * f.G + rr - i2 * f.G;
            const bool on = r < rows;
            const int pos = on ? pos0 + i2 : -1;
            int up;
            {
                // the row's queries, scaled by a power of two: largest magnitude in [2^14, 2^15)
                const uint4 *q = reinterpret_cast<const uint4 *>(a.q + (long long)(row0 + i2) * a.q_stride + head * D);
                uint32_t am = 0;
#pragma unroll
                for (int c = 0; c < D / 8; c++) {
                    const uint4 w = on ? __ldg(q + c) : make_uint4(0, 0, 0, 0);
                    const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int e = 0; e < 4; e++) am = max(am, max(x[e] & 0x7FFFu, (x[e] >> 16) & 0x7FFFu));
                }
                up = min(141 - (int)(am >> 7), 127);
                const float mul = pow2i(up);
#pragma unroll
                for (int c = 0; c < D / 8; c++) {
                    const uint4 w = on ? __ldg(q + c) : make_uint4(0, 0, 0, 0);
                    const uint32_t x[4] = {w.x, w.y, w.z, w.w};
                    uint32_t y[4];
#pragma unroll
                    for (int e = 0; e < 4; e++) y[e] = pack_f16(__uint_as_float(x[e] << 16) * mul, __uint_as_float(x[e] & 0xFFFF0000u) * mul);
                    *reinterpret_cast<uint4 *>(smem + L::kQ + (c / 8) * (kM * 128) + swizzled(r, c % 8)) = make_uint4(y[0], y[1], y[2], y[3]);
                }
                fence_async();
                bar_arrive(&q_full);
            }
            const float sc = a.scale * kLog2e;
            float m = -INFINITY, N = -INFINITY, l = 0.f;
            const uint32_t lanes = tmem + ((uint32_t)(32 * warp) << 16);
            bool ok = true;
            for (int j = 0; j < steps; j++) {
                const int st = j % kStages, t0 = (step0 + j) * kT;
                ok = bar_wait(&s_full[j & 1], (uint32_t)(j >> 1) & 1, status, 100);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                fence_after();
                uint32_t mt[NP];
                bool all = whole(t0);
#pragma unroll
                for (int p = 0; p < NP; p++) mt[p] = meta[st][p], all = all && (mt[p] >> 16);
                // 32 scores at a time, read twice: for the largest, and for the weights
                auto scores = [&](int hf, float (&s)[32]) {
                    tmem_ld32(lanes + (j & 1) * kT + 32 * hf, s);
                    if (!all)
#pragma unroll
                        for (int c = 0; c < 32; c++) {
                            const int t = t0 + 32 * hf + c;
                            if (!(t < seen && t <= pos && (a.window == 0 || t > pos - a.window) && (mt[(32 * hf + c) / P] >> 16))) s[c] = -INFINITY;
                        }
                };
                auto key_scale = [&](int p) { return fmaxf(pow2i((int)(mt[p] & 255u) - 127 - up) * sc, 1e-37f); };   // > 0: -inf stays
                float pm[NP], mx = -INFINITY, mv = -INFINITY;
#pragma unroll
                for (int p = 0; p < NP; p++) pm[p] = -INFINITY;
#pragma unroll
                for (int hf = 0; hf < 2; hf++) {
                    float s[32];
                    scores(hf, s);
#pragma unroll
                    for (int c = 0; c < 32; c++) pm[(32 * hf + c) / P] = fmaxf(pm[(32 * hf + c) / P], s[c]);
                }
                const float ms0 = m == -INFINITY ? 0.f : m;
#pragma unroll
                for (int p = 0; p < NP; p++) {
                    pm[p] *= key_scale(p);
                    mx = fmaxf(mx, pm[p]), mv = fmaxf(mv, pm[p] - ms0 + (float)((int)((mt[p] >> 8) & 255u) - 127));
                }
                // the references follow when passed by more than 2^8
                float corr = 1.f;
                const bool move = mx > m + 8.f || mv > N + 8.f;
                if (move) {
                    const float mn = fmaxf(m, mx), was = N + (m - mn);
                    float nn = was;
#pragma unroll
                    for (int p = 0; p < NP; p++) nn = fmaxf(nn, pm[p] - mn + (float)((int)((mt[p] >> 8) & 255u) - 127));
                    l *= ex2(m - mn);
                    corr = ex2(was - nn);
                    m = mn, N = nn;
                }
                const float ms = m == -INFINITY ? 0.f : m, Ns = N == -INFINITY ? 0.f : N;
                // weights; the products of the step before have read the P tile
                if (j > 0) {
                    ok = bar_wait(&o_done, (uint32_t)(j - 1) & 1, status, 101);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    fence_after();
                    if (__any_sync(0xffffffffu, move)) {
#pragma unroll 1
                        for (int c = 0; c < D; c += 32) {
                            float o[32];
                            tmem_ld32(lanes + 2 * kT + c, o);
#pragma unroll
                            for (int e = 0; e < 32; e++) o[e] *= corr;
                            tmem_st32(lanes + 2 * kT + c, o);
                        }
                    }
                }
                float sum = 0.f;
#pragma unroll
                for (int hf = 0; hf < 2; hf++) {
                    float s[32];
                    scores(hf, s);
#pragma unroll
                    for (int c8 = 0; c8 < 4; c8++) {
                        const int p = (32 * hf + 8 * c8) / P;
                        const float fac = ex2(fminf((float)((int)((mt[p] >> 8) & 255u) - 120) - Ns, 126.f)), ks = key_scale(p);
                        uint32_t y[4];
#pragma unroll
                        for (int e = 0; e < 4; e++) {
                            const float w0 = ex2(fmaf(s[8 * c8 + 2 * e], ks, -ms)), w1 = ex2(fmaf(s[8 * c8 + 2 * e + 1], ks, -ms));
                            sum += w0 + w1;
                            y[e] = pack_f16(w0 * fac, w1 * fac);
                        }
                        *reinterpret_cast<uint4 *>(smem + L::kP + swizzled(r, 4 * hf + c8)) = make_uint4(y[0], y[1], y[2], y[3]);
                    }
                }
                l += sum;
                fence_async();
                fence_before();
                bar_arrive(&p_full);
            }
            if (ok) ok = __all_sync(0xffffffffu, bar_wait(&o_done, (uint32_t)(steps - 1) & 1, status, 102));
            if (ok) {
                fence_after();
                const float sink = on && a.sinks ? a.sinks[head] * kLog2e : -INFINITY;
                const float top = fmaxf(m, sink);
                const float den = top == -INFINITY ? l : (m == -INFINITY ? l : l * ex2(m - top)) + ex2(sink - top);
                const float k = den == 0.f || N == -INFINITY ? 0.f : ex2(N - 7.f + (m - top)) / den;
                uint4 *o = reinterpret_cast<uint4 *>(a.out + (long long)(row0 + i2) * a.o_stride + head * D);
#pragma unroll 1
                for (int c = 0; c < D; c += 32) {
                    float v[32];
                    tmem_ld32(lanes + 2 * kT + c, v);
                    if (!on) continue;
#pragma unroll
                    for (int x = 0; x < 4; x++)
                        o[c / 8 + x] = make_uint4(bits_of(__floats2bfloat162_rn(v[8 * x] * k, v[8 * x + 1] * k)),
                                                  bits_of(__floats2bfloat162_rn(v[8 * x + 2] * k, v[8 * x + 3] * k)),
                                                  bits_of(__floats2bfloat162_rn(v[8 * x + 4] * k, v[8 * x + 5] * k)),
                                                  bits_of(__floats2bfloat162_rn(v[8 * x + 6] * k, v[8 * x + 7] * k)));
                }
            }
        } else if (warp < 8) {
            // ---- pages to operand tiles ----
            const int x = tid - 128;
            const int32_t *tab = a.table + (size_t)b * a.width;
            auto page_at = [&](int t) {   // of token t, -1 where there is none
                const int pg = t < seen ? __ldg(tab + t / P) : -1;
                return pg >= 0 && pg < a.c.n_pages ? pg : -1;
            };
            uint4 kw[KU], vw[KU];
            uint32_t mw = 0;
            // unit i of a thread: keys of token x % 64, dims 16 (x / 64 + 2 i) ..; values of dim u % D, tokens 16 (u / D) ..
            auto load = [&](int j) {
                const int t0 = (step0 + j) * kT;
                const int kp = page_at(t0 + x % kT), at = (t0 + x % kT) % P;
#pragma unroll
                for (int i = 0; i < KU; i++)
                    kw[i] = kp >= 0 ? __ldg(reinterpret_cast<const uint4 *>(a.c.k + ((size_t)kp * a.c.KVH + kvh) * (P * D) + (x / kT + 2 * i) * (P * 16) + at * 16))
                                    : make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int i = 0; i < KU; i++) {
                    const int u = x + 128 * i, dim = u % D, blk = u / D, t = t0 + 16 * blk, vp = page_at(t);
                    vw[i] = vp >= 0 ? __ldg(reinterpret_cast<const uint4 *>(a.c.v + ((size_t)vp * a.c.KVH + kvh) * (P * D) + (t % P) * D + dim * 16))
                                    : make_uint4(0, 0, 0, 0);
                }
                if (x < NP) {
                    const int pg = page_at(t0 + x * P);
                    const size_t ph = (size_t)max(pg, 0) * a.c.KVH + kvh;
                    mw = pg >= 0 ? (uint32_t)__ldg(a.c.ks + ph) | (uint32_t)__ldg(a.c.vs + ph) << 8 | 1u << 16 : 0u;
                }
            };
            load(0);
            for (int j = 0; j < steps; j++) {
                const int st = j % kStages, t0 = (step0 + j) * kT;
                if (j >= kStages && !bar_wait(&empty[st], (uint32_t)(j / kStages - 1) & 1, status, 103)) break;
                unsigned char *K = smem + L::kK + st * (kT * D * 2), *V = smem + L::kV + st * (kT * D * 2);
                const bool part = !whole(t0);
#pragma unroll
                for (int i = 0; i < KU; i++) {
                    uint4 c0, c1;
                    decode16(kw[i], true, c0, c1);
                    const int tok = x % kT, ch = 2 * (x / kT + 2 * i);   // 16-byte chunk of the row: dims 8 ch ..
                    unsigned char *to = K + (ch / 8) * (kT * 128);
                    *reinterpret_cast<uint4 *>(to + swizzled(tok, ch % 8)) = c0;
                    *reinterpret_cast<uint4 *>(to + swizzled(tok, ch % 8 + 1)) = c1;
                }
#pragma unroll
                for (int i = 0; i < KU; i++) {
                    const int u = x + 128 * i, dim = u % D, blk = u / D;
                    if (part) {
                        // tokens that no row sees to zero; a NaN among the others: not all rows see it
                        uint32_t w[4] = {vw[i].x, vw[i].y, vw[i].z, vw[i].w}, nan = 0;
#pragma unroll
                        for (int q = 0; q < 4; q++) {
#pragma unroll
                            for (int e = 0; e < 4; e++) {
                                const int t = t0 + 16 * blk + 2 * q + (e & 1) + 8 * (e >> 1);
                                if (t >= seen || t < lo) w[q] &= ~(0xFFu << (8 * e));
                            }
                            nan |= ((w[q] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
                        }
                        if (nan) odd = 1;
                        vw[i] = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                    uint4 c0, c1;
                    decode16(vw[i], false, c0, c1);
                    *reinterpret_cast<uint4 *>(V + swizzled(dim, 2 * blk)) = c0;
                    *reinterpret_cast<uint4 *>(V + swizzled(dim, 2 * blk + 1)) = c1;
                }
                if (x < NP) meta[st][x] = mw;
                fence_async();
                bar_arrive(&full[st]);
                if (j + 1 < steps) load(j + 1);
            }
        } else if (lane == 0) {
            // ---- the products ----
            const uint32_t Q = smem_u32(smem + L::kQ), Pt = smem_u32(smem + L::kP);
            bool ok = bar_wait(&q_full, 0, status, 104);
            auto scores = [&](int j) {   // into score buffer j & 1
                const int st = j % kStages;
                if (!bar_wait(&full[st], (uint32_t)(j / kStages) & 1, status, 105)) return false;
                fence_after();
                const uint32_t K = smem_u32(smem + L::kK + st * (kT * D * 2));
#pragma unroll
                for (int c = 0; c < D / 16; c++)
                    mma(tmem + (j & 1) * kT, tile_desc(Q + (c / 4) * (kM * 128) + (c % 4) * 32), tile_desc(K + (c / 4) * (kT * 128) + (c % 4) * 32),
                        inst_desc(kT), c != 0);
                commit(&s_full[j & 1]);
                return true;
            };
            if (ok) ok = scores(0);
            for (int j = 0; j < steps && ok; j++) {
                // the next scores go ahead of this step's values: their buffer was read before step j - 1's weights were
                if (j + 1 < steps) ok = scores(j + 1);
                if (ok) ok = bar_wait(&p_full, (uint32_t)j & 1, status, 106);
                if (!ok) break;
                fence_after();
                const int st = j % kStages;
                const uint32_t V = smem_u32(smem + L::kV + st * (kT * D * 2));
#pragma unroll
                for (int c = 0; c < kT / 16; c++)
                    mma(tmem + 2 * kT, tile_desc(Pt + c * 32), tile_desc(V + c * 32), inst_desc(D), j > 0 || c > 0);
                commit(&empty[st]);
                commit(&o_done);
            }
            if (!ok) {   // the products already issued finish before tensor memory is released
                commit(&drain);
                bar_wait(&drain, 0, status, 107, true);
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
    if (warp == 8) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 256;" ::"r"(tmem));
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
    const long long tiles = (long long)a.n_rows * f.G / kM + a.n_seqs;
    const long long most = (long long)a.n_seqs * (((long long)a.max_new * f.G + kM - 1) / kM);
    const dim3 grid((unsigned)std::min(tiles, most), a.c.KVH);
    return a.c.D == 64 ? prompt_page<64>(f, grid, st) : prompt_page<128>(f, grid, st);
}
