// rope.cu -- per-head RMS norm and rotary positions of queries and keys.
//
// For each head of a token: n = x / sqrt(mean(x^2) + eps) * w (where there is a
// weight), then every pair (a, b) of n turns by the token's angle,
// (a cos - b sin, b cos + a sin).  One read and one write per element: the bound
// is HBM, and for a few tokens the launch.
//
// One CTA per token: the R / 2 angles are made once (64-bit product and reduction to a fraction of a
// turn, then fp32 sincospi) and shared by all heads, while the first rows are on their way.  Eight
// consecutive elements per lane where R / 2 is a multiple of 8, else four: a lane's partner elements then
// lie in one other lane of the row.  8,191 tokens of 40 heads of 128 in bf16, normed: 36 us, 4.7 TB/s
// (four elements a lane, nothing loaded ahead: 59 us; a warp per token, angles in registers: 38 us, and
// with four rows under way 37 us and 13 instead of 7 for 2,048 tokens in fp32).  One token: 1.7 us.
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

// E (4 or 8) consecutive elements, as they are in memory and as fp32.
template <bool BF, int E>
struct Raw {
    uint4 u[BF ? 1 : E / 4];
};

template <bool BF, int E>
__device__ __forceinline__ void load_raw(Raw<BF, E> &r, const void *base, long long at) {
    if (BF) {
        const uint16_t *p = static_cast<const uint16_t *>(base) + at;
        if (E == 8) {
            r.u[0] = *reinterpret_cast<const uint4 *>(p);
        } else {
            const uint2 v = *reinterpret_cast<const uint2 *>(p);
            r.u[0].x = v.x, r.u[0].y = v.y;
        }
    } else {
        const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const float *>(base) + at);
#pragma unroll
        for (int i = 0; i < E / 4; i++) r.u[i] = p[i];
    }
}

template <bool BF, int E>
__device__ __forceinline__ void to_floats(const Raw<BF, E> &r, float (&x)[E]) {
    if (BF) {
        const uint32_t w[4] = {r.u[0].x, r.u[0].y, r.u[0].z, r.u[0].w};
#pragma unroll
        for (int i = 0; i < E / 2; i++) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    } else {
#pragma unroll
        for (int i = 0; i < E / 4; i++) {
            x[4 * i] = __uint_as_float(r.u[i].x), x[4 * i + 1] = __uint_as_float(r.u[i].y);
            x[4 * i + 2] = __uint_as_float(r.u[i].z), x[4 * i + 3] = __uint_as_float(r.u[i].w);
        }
    }
}

template <bool BF, int E>
__device__ __forceinline__ void store_floats(void *base, long long at, const float (&x)[E]) {
    if (BF) {
        uint32_t w[E / 2];
#pragma unroll
        for (int i = 0; i < E / 2; i++) {
            const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&v);
        }
        uint16_t *p = static_cast<uint16_t *>(base) + at;
        if (E == 8) *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[E / 2 - 2], w[E / 2 - 1]);
        else *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
    } else {
        float4 *p = reinterpret_cast<float4 *>(static_cast<float *>(base) + at);
#pragma unroll
        for (int i = 0; i < E / 4; i++) p[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
    }
}

// LP lanes per row (a power of two), NC chunks of E LP elements per row.
template <bool IN_BF, bool OUT_BF, int E, int LP, int NC>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeParams p) {
    __shared__ __align__(16) float2 cs[kRopeMaxD / 2];  // (cos, sin) of the token's angles
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    constexpr int kRows = 32 / LP;        // rows of a warp
    const long long t = blockIdx.x;
    const int half = p.R / 2;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int sub = lane & (LP - 1), base = lane - sub;
    const int heads = p.side[0].heads + p.side[1].heads;
    const bool any_weight = p.side[0].weight || p.side[1].weight;
    const float inv_d = 1.0f / (float)p.D;
    // where a lane's first element of a row is, per side (head h at + h D)
    const long long in0 = t * p.side[0].in_stride + E * sub, in1 = t * p.side[1].in_stride - p.side[0].heads * p.D + E * sub;
    const long long out0 = t * p.side[0].out_stride + E * sub, out1 = t * p.side[1].out_stride - p.side[0].heads * p.D + E * sub;
    auto load = [&](int r0, Raw<IN_BF, E> (&v)[NC]) {
        const int r = r0 + lane / LP;
        if (r >= heads) return;
        const bool k = r >= p.side[0].heads;
        const void *in = k ? p.side[1].in : p.side[0].in;
        const long long at = (k ? in1 : in0) + r * p.D;
#pragma unroll
        for (int c = 0; c < NC; c++)
            if (E * (c * LP + sub) < p.D) load_raw<IN_BF, E>(v[c], in, at + E * LP * c);
    };
    Raw<IN_BF, E> raw[NC];
    load(warp * kRows, raw);
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
    for (int r0 = warp * kRows; r0 < heads; r0 += (kRopeThreads / 32) * kRows) {
        const int r = r0 + lane / LP;
        const bool row = r < heads, k = r >= p.side[0].heads;
        float v[NC][E];
#pragma unroll
        for (int c = 0; c < NC; c++) to_floats<IN_BF, E>(raw[c], v[c]);
        load(r0 + (kRopeThreads / 32) * kRows, raw);  // the next rows
        const float *weight = row ? (k ? p.side[1].weight : p.side[0].weight) : nullptr;
        if (any_weight) {  // a warp may hold rows of both sides: every lane takes part in the sum
            float sum = 0.0f;
#pragma unroll
            for (int c = 0; c < NC; c++) {
                if (E * (c * LP + sub) >= p.D) continue;
#pragma unroll
                for (int i = 0; i < E; i++) sum += v[c][i] * v[c][i];
            }
#pragma unroll
            for (int o = LP / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
            if (weight) {
                const float inv = rsqrtf(sum * inv_d + p.eps);
#pragma unroll
                for (int c = 0; c < NC; c++) {
                    const int e = E * (c * LP + sub);
                    if (e >= p.D) continue;
#pragma unroll
                    for (int i = 0; i < E; i += 4) {
                        const float4 w = __ldg(reinterpret_cast<const float4 *>(weight + e + i));
                        v[c][i] *= inv * w.x;
                        v[c][i + 1] *= inv * w.y;
                        v[c][i + 2] *= inv * w.z;
                        v[c][i + 3] *= inv * w.w;
                    }
                }
            }
        }
        float out[NC][E];
        if (p.interleaved) {
#pragma unroll
            for (int c = 0; c < NC; c++) {
                const int e = E * (c * LP + sub);
#pragma unroll
                for (int i = 0; i < E; i++) out[c][i] = v[c][i];
                if (e < p.R) {
#pragma unroll
                    for (int i = 0; i < E; i += 4) {
                        const float4 a = *reinterpret_cast<const float4 *>(cs + (e + i) / 2);  // two (cos, sin)
                        out[c][i] = v[c][i] * a.x - v[c][i + 1] * a.y;
                        out[c][i + 1] = v[c][i + 1] * a.x + v[c][i] * a.y;
                        out[c][i + 2] = v[c][i + 2] * a.z - v[c][i + 3] * a.w;
                        out[c][i + 3] = v[c][i + 3] * a.z + v[c][i + 2] * a.w;
                    }
                }
            }
        } else {
#pragma unroll
            for (int c = 0; c < NC; c++) {
                const int e = E * (c * LP + sub);
                const bool turn = e < p.R, low = e < half;
                // lane index, within the row, of the partner elements
                const int pl = turn ? (low ? e + half : e - half) / E : sub;
                const float2 *q = cs + (turn ? (low ? e : e - half) : 0);
                const float sg = low ? -1.0f : 1.0f;
#pragma unroll
                for (int i = 0; i < E; i++) {
                    float o = __shfl_sync(0xFFFFFFFFu, v[0][i], base + (pl & (LP - 1)));
                    if (NC == 2) {
                        const float o1 = __shfl_sync(0xFFFFFFFFu, v[NC - 1][i], base + (pl & (LP - 1)));
                        if (pl >= LP) o = o1;
                    }
                    out[c][i] = turn ? v[c][i] * q[i].x + sg * (o * q[i].y) : v[c][i];
                }
            }
        }
        if (row) {
            void *to = k ? p.side[1].out : p.side[0].out;
            const long long at = (k ? out1 : out0) + r * p.D;
#pragma unroll
            for (int c = 0; c < NC; c++)
                if (E * (c * LP + sub) < p.D) store_floats<OUT_BF, E>(to, at + E * LP * c, out[c]);
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
    if (p.R % 16 == 0) {
        if (p.D <= 32) cudaLaunchKernelEx(&cfg, rope_kernel<IN_BF, OUT_BF, 8, 4, 1>, p);
        else if (p.D <= 64) cudaLaunchKernelEx(&cfg, rope_kernel<IN_BF, OUT_BF, 8, 8, 1>, p);
        else if (p.D <= 128) cudaLaunchKernelEx(&cfg, rope_kernel<IN_BF, OUT_BF, 8, 16, 1>, p);
        else cudaLaunchKernelEx(&cfg, rope_kernel<IN_BF, OUT_BF, 8, 32, 1>, p);
    } else {
        if (p.D <= 32) cudaLaunchKernelEx(&cfg, rope_kernel<IN_BF, OUT_BF, 4, 8, 1>, p);
        else if (p.D <= 128) cudaLaunchKernelEx(&cfg, rope_kernel<IN_BF, OUT_BF, 4, 32, 1>, p);
        else cudaLaunchKernelEx(&cfg, rope_kernel<IN_BF, OUT_BF, 4, 32, 2>, p);
    }
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
