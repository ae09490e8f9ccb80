// moe_kv4_attend.cu -- attention over the 4-bit paged key/value cache.
#include "moe_kv4.cuh"

#include <algorithm>

namespace {

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

}  // namespace

size_t kv4_workspace_bytes(int) { return kKv8ClearBytes; }

cudaError_t launch_kv4_attend(const Kv4Attend &a, unsigned char *, cudaStream_t st) {
    return launch_pdl(moe_kv4_attend_kernel, dim3((unsigned)((long long)a.n_seqs * a.max_new), a.QH), dim3(128), 0, st, a);
}
