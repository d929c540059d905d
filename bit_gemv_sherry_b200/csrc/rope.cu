// rope.cu -- per-head RMS norm and rotary positions of queries and keys.
//
// For each head of a token: n = x / sqrt(mean(x^2) + eps) * w (where there is a
// weight), then every pair (a, b) of n turns by the token's angle,
// (a cos - b sin, b cos + a sin).  One read and one write per element: the bound
// is HBM, and for a few tokens the launch.
//
// One CTA per token: the R / 2 angles are made once (64-bit product and reduction
// to a fraction of a turn, then fp32 sincospi) and shared by all heads.  Four
// consecutive elements per lane; R / 2 is a multiple of 4, so a lane's partner
// elements lie in one other lane of the row.
#include <cuda_bf16.h>

#include "common.cuh"

namespace sherry {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeMaxD = 256;

struct RopeSide {
    const void *in;
    void *out;
    const float *weight;
    long long in_stride, out_stride;
    int heads;
};

struct RopeParams {
    RopeSide side[2];  // queries, keys
    const int *positions;
    const float *inv_freq;
    int D, R;
    int interleaved;
    float eps;
};

template <bool BF>
__device__ __forceinline__ float4 load4(const void *base, long long at) {
    if (BF) {
        const uint2 u = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(base) + at);
        return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xFFFF0000u),
                           __uint_as_float(u.y << 16), __uint_as_float(u.y & 0xFFFF0000u));
    }
    return *reinterpret_cast<const float4 *>(static_cast<const float *>(base) + at);
}

template <bool BF>
__device__ __forceinline__ void store4(void *base, long long at, float4 v) {
    if (BF) {
        const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
        uint2 u;
        u.x = *reinterpret_cast<const uint32_t *>(&a);
        u.y = *reinterpret_cast<const uint32_t *>(&b);
        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(base) + at) = u;
    } else {
        *reinterpret_cast<float4 *>(static_cast<float *>(base) + at) = v;
    }
}

__device__ __forceinline__ float4 shfl4(float4 v, int src) {
    return make_float4(__shfl_sync(0xFFFFFFFFu, v.x, src), __shfl_sync(0xFFFFFFFFu, v.y, src),
                       __shfl_sync(0xFFFFFFFFu, v.z, src), __shfl_sync(0xFFFFFFFFu, v.w, src));
}

// LP lanes per row (a power of two), NC chunks of 4 LP elements per row.
template <bool IN_BF, bool OUT_BF, int LP, int NC>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeParams p) {
    __shared__ float2 cs[kRopeMaxD / 2];  // (cos, sin) of the token's angles
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const long long t = blockIdx.x;
    const int half = p.R / 2;
    if (threadIdx.x < half) {
        // turns = pos * inv_freq / (2 pi), kept modulo one: sincospi takes half-turns
        const double turns = (double)__ldg(p.positions + t) * (double)__ldg(p.inv_freq + threadIdx.x) *
                             0.15915494309189533577;
        const float frac = (float)(turns - rint(turns));
        float s, c;
        sincospif(2.0f * frac, &s, &c);
        cs[threadIdx.x] = make_float2(c, s);
    }
    __syncthreads();
    constexpr int kRows = 32 / LP;  // rows of a warp
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int sub = lane & (LP - 1), base = lane - sub;
    const int heads = p.side[0].heads + p.side[1].heads;
    for (int r0 = warp * kRows; r0 < heads; r0 += (kRopeThreads / 32) * kRows) {
        int h = r0 + lane / LP;
        const bool row = h < heads;
        const RopeSide &s = p.side[row && h >= p.side[0].heads ? 1 : 0];
        if (h >= p.side[0].heads) h -= p.side[0].heads;
        float4 v[NC];
#pragma unroll
        for (int c = 0; c < NC; c++) {
            const int e = 4 * (c * LP + sub);
            v[c] = row && e < p.D ? load4<IN_BF>(s.in, t * s.in_stride + (long long)h * p.D + e)
                                  : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        }
        // a warp may hold rows of both sides: every lane takes part in the sum
        float sum = 0.0f;
#pragma unroll
        for (int c = 0; c < NC; c++)
            sum += v[c].x * v[c].x + v[c].y * v[c].y + v[c].z * v[c].z + v[c].w * v[c].w;
#pragma unroll
        for (int o = LP / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
        if (row && s.weight) {
            const float inv = 1.0f / sqrtf(sum / (float)p.D + p.eps);
#pragma unroll
            for (int c = 0; c < NC; c++) {
                const int e = 4 * (c * LP + sub);
                if (e >= p.D) continue;
                const float4 w = __ldg(reinterpret_cast<const float4 *>(s.weight + e));
                v[c] = make_float4(v[c].x * inv * w.x, v[c].y * inv * w.y, v[c].z * inv * w.z,
                                   v[c].w * inv * w.w);
            }
        }
        float4 out[NC];
        if (p.interleaved) {
#pragma unroll
            for (int c = 0; c < NC; c++) {
                const int e = 4 * (c * LP + sub);
                out[c] = v[c];
                if (e < p.R) {
                    const float2 a = cs[e / 2], b = cs[e / 2 + 1];
                    out[c] = make_float4(v[c].x * a.x - v[c].y * a.y, v[c].y * a.x + v[c].x * a.y,
                                         v[c].z * b.x - v[c].w * b.y, v[c].w * b.x + v[c].z * b.y);
                }
            }
        } else {
#pragma unroll
            for (int c = 0; c < NC; c++) {
                const int e = 4 * (c * LP + sub);
                const bool turn = e < p.R, low = e < half;
                // lane index, within the row, of the partner elements
                const int pl = turn ? (low ? e + half : e - half) / 4 : sub;
                float4 o = shfl4(v[0], base + (pl & (LP - 1)));
                if (NC == 2) {
                    const float4 o1 = shfl4(v[NC - 1], base + (pl & (LP - 1)));
                    if (pl >= LP) o = o1;
                }
                out[c] = v[c];
                if (turn) {
                    const float2 *q = cs + (low ? e : e - half);
                    const float sg = low ? -1.0f : 1.0f;
                    out[c] = make_float4(v[c].x * q[0].x + sg * (o.x * q[0].y),
                                         v[c].y * q[1].x + sg * (o.y * q[1].y),
                                         v[c].z * q[2].x + sg * (o.z * q[2].y),
                                         v[c].w * q[3].x + sg * (o.w * q[3].y));
                }
            }
        }
#pragma unroll
        for (int c = 0; c < NC; c++) {
            const int e = 4 * (c * LP + sub);
            if (row && e < p.D) store4<OUT_BF>(s.out, t * s.out_stride + (long long)h * p.D + e, out[c]);
        }
    }
}

template <bool IN_BF, bool OUT_BF>
void rope_launch(const RopeParams &p, int64_t T, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)T);
    cfg.blockDim = dim3(kRopeThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (p.D <= 16) cudaLaunchKernelEx(&cfg, rope_kernel<IN_BF, OUT_BF, 4, 1>, p);
    else if (p.D <= 32) cudaLaunchKernelEx(&cfg, rope_kernel<IN_BF, OUT_BF, 8, 1>, p);
    else if (p.D <= 64) cudaLaunchKernelEx(&cfg, rope_kernel<IN_BF, OUT_BF, 16, 1>, p);
    else if (p.D <= 128) cudaLaunchKernelEx(&cfg, rope_kernel<IN_BF, OUT_BF, 32, 1>, p);
    else cudaLaunchKernelEx(&cfg, rope_kernel<IN_BF, OUT_BF, 32, 2>, p);
}

// One side's pointers and strides; `unit` is the stride's and, in elements, 16 bytes' worth.
sherry_status check_side(const void *in, const void *out, const float *w, int64_t in_stride,
                         int64_t out_stride, int heads, const sherry_rope *r) {
    if (!in || !out) return SHERRY_ERR_NULL;
    if (in_stride < (int64_t)heads * r->D || out_stride < (int64_t)heads * r->D) return SHERRY_ERR_SHAPE;
    if (!aligned(in, 16) || !aligned(out, 16) || (w && !aligned(w, 16))) return SHERRY_ERR_ALIGN;
    if (in_stride % (r->in_type == SHERRY_F32 ? 4 : 8) || out_stride % (r->out_type == SHERRY_F32 ? 4 : 8))
        return SHERRY_ERR_ALIGN;
    return SHERRY_OK;
}

}  // namespace
}  // namespace sherry

extern "C" sherry_status sherry_qk_norm_rope(const sherry_rope *r, sherry_stream_t stream) {
    using namespace sherry;
    if (!r || !r->positions) return SHERRY_ERR_NULL;
    if (r->T < 1 || r->Hq < 0 || r->Hk < 0 || (r->Hq == 0 && r->Hk == 0)) return SHERRY_ERR_SHAPE;
    if (r->D < 8 || r->D > kRopeMaxD || r->D % 8 || r->R < 0 || r->R > r->D || r->R % 8) return SHERRY_ERR_SHAPE;
    if (r->R > 0 && !r->inv_freq) return SHERRY_ERR_NULL;
    if ((r->in_type != SHERRY_F32 && r->in_type != SHERRY_BF16) ||
        (r->out_type != SHERRY_F32 && r->out_type != SHERRY_BF16))
        return SHERRY_ERR_UNSUPPORTED;
    if (r->T > 0x7FFFFFFF || (int64_t)r->Hq + r->Hk > 65536) return SHERRY_ERR_UNSUPPORTED;
    if (!aligned(r->positions, 4) || !aligned(r->inv_freq, 4)) return SHERRY_ERR_ALIGN;
    RopeParams p = {};
    if (r->Hq > 0) {
        const sherry_status st = check_side(r->q, r->q_out, r->q_weight, r->q_stride, r->q_out_stride, r->Hq, r);
        if (st != SHERRY_OK) return st;
        p.side[0] = {r->q, r->q_out, r->q_weight, r->q_stride, r->q_out_stride, r->Hq};
    }
    if (r->Hk > 0) {
        const sherry_status st = check_side(r->k, r->k_out, r->k_weight, r->k_stride, r->k_out_stride, r->Hk, r);
        if (st != SHERRY_OK) return st;
        p.side[1] = {r->k, r->k_out, r->k_weight, r->k_stride, r->k_out_stride, r->Hk};
    }
    p.positions = r->positions;
    p.inv_freq = r->inv_freq;
    p.D = r->D;
    p.R = r->R;
    p.interleaved = r->interleaved;
    p.eps = r->eps;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (r->in_type == SHERRY_BF16) {
        if (r->out_type == SHERRY_BF16) rope_launch<true, true>(p, r->T, s);
        else rope_launch<true, false>(p, r->T, s);
    } else {
        if (r->out_type == SHERRY_BF16) rope_launch<false, true>(p, r->T, s);
        else rope_launch<false, false>(p, r->T, s);
    }
    return launch_status("sherry_qk_norm_rope");
}
