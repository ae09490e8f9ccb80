// moe_kv8_attend.cu -- attention over the 8-bit paged key/value cache.
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

}  // namespace

size_t kv8_workspace_bytes(int) { return 8192; }

cudaError_t launch_kv8_attend(const Kv8Attend &a, unsigned char *, cudaStream_t st) {
    const dim3 grid(a.QH, a.max_new, a.n_seqs);
    if (a.c.D == 64) return launch_pdl(moe_kv8_attend_kernel<64>, grid, dim3(128), 0, st, a);
    return launch_pdl(moe_kv8_attend_kernel<128>, grid, dim3(128), 0, st, a);
}
