// attn.cu -- causal attention over the 4-bit key/value cache.
#include <cuda_bf16.h>

#include "kv4.cuh"

namespace sherry {
namespace {

constexpr int kAttnThreads = 128;

struct AttnParams {
    Kv4View c;
    const uint16_t *q;
    uint16_t *out;
    long long q_stride, out_stride;
    int Hq;
    float scale;
    unsigned int *err;
};

// One CTA per (row, query head).  A warp takes 32 keys at a time, one per lane, then 32
// values, D / 32 elements per lane, with a running maximum and sum; the four warps'
// results are joined at the end.  Plain fp32 arithmetic on the decoded values.
template <int D>
__global__ void __launch_bounds__(kAttnThreads) attn_simple_kernel(const __grid_constant__ AttnParams p) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    constexpr int E = D / 32;
    __shared__ float qs[D];
    __shared__ float jm[4], jl[4], jo[4][D];
    const int t = blockIdx.x, hq = blockIdx.y;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int b = 0, pos = -1;
    if (!kv4_find(p.c, t, b, pos)) return;
    const int h = hq / (p.Hq / p.c.H);
    if (threadIdx.x < D) qs[threadIdx.x] = __uint_as_float((uint32_t)p.q[t * p.q_stride + hq * D + threadIdx.x] << 16);
    __syncthreads();
    float m = -INFINITY, l = 0.0f, o[E];
    for (int e = 0; e < E; e++) o[e] = 0.0f;
    for (int k0 = 32 * warp; k0 <= pos; k0 += 128) {
        const int key = k0 + lane;
        float x = -INFINITY;
        int page = -1;
        if (key <= pos) page = kv4_page(p.c, b, key, p.err);
        if (page >= 0) {
            const uint8_t *blk = kv4_block<D>(p.c, page, h, 0);
            const int slot = key % SHERRY_KV4_PAGE;
            const uint32_t sm = reinterpret_cast<const uint32_t *>(blk + Kv4<D>::kCodes)[slot];
            float dot = 0.0f;
            for (int d = 0; d < D; d += 2) {
                const uint32_t v = blk[slot * Kv4<D>::kRow + d / 2];
                dot += qs[d] * (kv4_low(sm) + kv4_step(sm) * (float)(v & 15)) +
                       qs[d + 1] * (kv4_low(sm) + kv4_step(sm) * (float)(v >> 4));
            }
            x = dot * p.scale;
        }
        float mx = x;
        for (int i = 16; i > 0; i >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, i));
        const float mn = fmaxf(m, mx);
        if (mn == -INFINITY) continue;  // no key of these 32 is there
        const float w = page >= 0 ? expf(x - mn) : 0.0f, f = expf(m - mn);
        float sum = w;
        for (int i = 16; i > 0; i >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, i);
        l = l * f + sum;
        m = mn;
        for (int e = 0; e < E; e++) o[e] *= f;
        for (int j = 0; j < 32; j++) {
            const float pj = __shfl_sync(0xFFFFFFFFu, w, j);
            const int pg = __shfl_sync(0xFFFFFFFFu, page, j);
            if (pg < 0) continue;
            const uint8_t *blk = kv4_block<D>(p.c, pg, h, 1);
            const int slot = (k0 + j) % SHERRY_KV4_PAGE;
            const uint32_t sm = reinterpret_cast<const uint32_t *>(blk + Kv4<D>::kCodes)[slot];
            for (int e = 0; e < E; e++) {
                const int d = lane * E + e;
                const uint32_t v = blk[slot * Kv4<D>::kRow + d / 2] >> (4 * (d & 1));
                o[e] += pj * (kv4_low(sm) + kv4_step(sm) * (float)(v & 15));
            }
        }
    }
    if (lane == 0) jm[warp] = m, jl[warp] = l;
    for (int e = 0; e < E; e++) jo[warp][lane * E + e] = o[e];
    __syncthreads();
    if (threadIdx.x < D) {
        const float mn = fmaxf(fmaxf(jm[0], jm[1]), fmaxf(jm[2], jm[3]));
        float sum = 0.0f, v = 0.0f;
        for (int w = 0; w < 4; w++) {
            const float f = jm[w] == -INFINITY ? 0.0f : expf(jm[w] - mn);
            sum += jl[w] * f;
            v += jo[w][threadIdx.x] * f;
        }
        const __nv_bfloat16 r = __float2bfloat16_rn(sum > 0.0f ? v / sum : (mn == -INFINITY ? 0.0f : v / sum));
        p.out[t * p.out_stride + hq * D + threadIdx.x] = __bfloat16_as_ushort(r);
    }
}

}  // namespace
}  // namespace sherry

extern "C" size_t sherry_attn_kv4_workspace_bytes(int64_t T, int Hq, int D) {
    if (T < 1 || Hq < 1 || (D != 64 && D != 128)) return 0;
    return 256;
}

extern "C" sherry_status sherry_attn_kv4(const sherry_kv4 *c, const uint16_t *q, int64_t q_stride, uint16_t *out,
                                         int64_t out_stride, int Hq, int64_t max_q, float scale, void *workspace,
                                         size_t workspace_bytes, sherry_stream_t stream) {
    using namespace sherry;
    const sherry_status st = kv4_check(c);
    if (st != SHERRY_OK) return st;
    if (!q || !out) return SHERRY_ERR_NULL;
    if (Hq < 1 || Hq % c->H || max_q < 0 || q_stride < (int64_t)Hq * c->D || out_stride < (int64_t)Hq * c->D)
        return SHERRY_ERR_SHAPE;
    if (Hq > 65535) return SHERRY_ERR_UNSUPPORTED;
    if (!aligned(q, 16) || !aligned(out, 16) || q_stride % 8 || out_stride % 8) return SHERRY_ERR_ALIGN;
    if (!workspace) return SHERRY_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return SHERRY_ERR_ALIGN;
    if (workspace_bytes < sherry_attn_kv4_workspace_bytes(c->T, Hq, c->D)) return SHERRY_ERR_WORKSPACE;
    AttnParams p;
    p.c = kv4_view(c);
    p.q = q;
    p.out = out;
    p.q_stride = q_stride;
    p.out_stride = out_stride;
    p.Hq = Hq;
    p.scale = scale;
    p.err = kv4_error_address();
    if (!p.err) return SHERRY_ERR_CUDA;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const dim3 grid((unsigned)c->T, (unsigned)Hq);
    if (c->D == 64) attn_simple_kernel<64><<<grid, kAttnThreads, 0, s>>>(p);
    else attn_simple_kernel<128><<<grid, kAttnThreads, 0, s>>>(p);
    return launch_status("sherry_attn_kv4");
}
