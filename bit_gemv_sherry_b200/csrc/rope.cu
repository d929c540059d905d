// rope.cu -- per-head RMS norm and rotary positions of queries and keys.
//
// For each head of a token: n = x / sqrt(mean(x^2) + eps) * w (where there is a
// weight), then every pair (a, b) of n turns by the token's angle,
// (a cos - b sin, b cos + a sin).  One read and one write per element: the bound
// is HBM, and for a few tokens the launch.
//
// A CTA takes one token or four: their R / 2 angles each are made once (64-bit product and reduction to a
// fraction of a turn, then fp32 sincospi) and shared by all heads, while the first rows are on their way.
// A lane holds both elements of its pairs, 16 bytes of bf16 from either half (8 where R / 2 is no multiple
// of 8).  8,191 tokens of 40 heads of 128 in bf16, normed, half of each head turned: 31 us, 5.4 TB/s, which
// is HBM's within a fifth; 2,048 tokens of 40 heads of 64, fp32: 5.1 us; one token: 1.7 us.  Earlier forms of
// the first: partner elements by shuffles, one token a CTA, 36 us; a warp per token 38 us; three CTAs per SM
// 34 us (fewer loads under way), five 43 us (spills).
#include <cuda_bf16.h>

#include "common.cuh"

namespace sherry {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeCtas = 4;    // per SM
constexpr int kRopeTokens = 4;  // of a CTA
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
    int T, D, R;
    int interleaved;
    int step_rows;  // rows of a token, up to a warp's whole steps
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

// LP lanes per row (a power of two), two chunks of E elements each: E pairs, so that a lane turns them by itself.
template <bool IN_BF, bool OUT_BF, int E, int LP, int TOKENS>
__global__ void __launch_bounds__(kRopeThreads, kRopeCtas) rope_kernel(const __grid_constant__ RopeParams p) {
    __shared__ __align__(16) float cos_of[TOKENS][kRopeMaxD / 2], sin_of[TOKENS][kRopeMaxD / 2];  // of the tokens' angles
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    constexpr int kRows = 32 / LP;        // rows of a warp
    const int t0 = blockIdx.x * TOKENS, tokens = min(TOKENS, p.T - t0);
    const int half = p.R / 2;
    const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    const int sub = lane & (LP - 1);
    const int hq = p.side[0].heads, heads = hq + p.side[1].heads;
    // the lane's chunks and its angles' groups of four; where halves are paired, what is not turned is in the
    // lanes behind the pairs.  Neighbouring lanes have neighbouring chunks (a lane with two of them in a row
    // writes half sectors: 50 us instead of 31 for 8,191 tokens of 40 heads of 128, bf16).
    int e0 = E * sub, e1 = e0 + E * LP, a0 = e0 / 2, a1 = e1 / 2;
    if (!p.interleaved) {
        const int tail = sub - half / E, tails = (p.D - p.R + 2 * E - 1) / (2 * E);
        a0 = e0, a1 = e0 + 4;
        if (tail < 0) e1 = e0 + half;
        else e0 = tail < tails ? p.R + E * tail : p.D, e1 = e0 + E * tails;
    }
    const bool on0 = e0 < p.D, on1 = e1 < p.D, turn0 = e0 < p.R, turn1 = e1 < p.R;
    auto load = [&](int t, int r, Raw<IN_BF, E> (&v)[2]) {
        if (t >= tokens || r >= heads) return;
        const bool k = r >= hq;
        const long long at = (t0 + t) * p.side[k].in_stride + (k ? r - hq : r) * p.D + e0;
        if (on0) load_raw<IN_BF, E>(v[0], p.side[k].in, at);
        if (on1) load_raw<IN_BF, E>(v[1], p.side[k].in, at + (e1 - e0));
    };
    // the warp's steps: kRows rows of one token each, every `warps`-th of the CTA's
    int token = 0, first = (threadIdx.x >> 5) * kRows;
    auto next = [&](int &t, int &f) {
        f += warps * kRows;
        while (f >= p.step_rows && t < tokens) f -= p.step_rows, t++;
    };
    if (first >= p.step_rows) first -= warps * kRows, next(token, first);
    Raw<IN_BF, E> raw[2] = {};
    load(token, first + lane / LP, raw);
    for (int j = threadIdx.x; j < tokens * half; j += blockDim.x) {
        // turns = pos * inv_freq / (2 pi), kept modulo one: sincospi takes half-turns
        const int t = TOKENS == 1 ? 0 : j / half, i = j - t * half;
        const double turns = (double)__ldg(p.positions + t0 + t) * (double)__ldg(p.inv_freq + i) * 0.15915494309189533577;
        const float frac = (float)(turns - rint(turns));
        sincospif(2.0f * frac, &sin_of[t][i], &cos_of[t][i]);
    }
    __syncthreads();
    const bool any_weight = p.side[0].weight || p.side[1].weight;
    const float inv_d = 1.0f / (float)p.D;
    while (token < tokens) {
        const int t = token, r = first + lane / LP;
        const bool row = r < heads, k = r >= hq;
        float x[2][E];
        to_floats<IN_BF, E>(raw[0], x[0]);
        to_floats<IN_BF, E>(raw[1], x[1]);
        f2 v[2][E / 2];
#pragma unroll
        for (int c = 0; c < 2; c++)
#pragma unroll
            for (int i = 0; i < E / 2; i++) v[c][i] = pair2(x[c][2 * i], x[c][2 * i + 1]);
        next(token, first);
        load(token, first + lane / LP, raw);  // the next rows
        if (any_weight) {  // a warp may hold rows of both sides: every lane takes part in the sum
            f2 sums = pair2(0.0f, 0.0f);
            if (on0) {
#pragma unroll
                for (int i = 0; i < E / 2; i++) sums = fma2(v[0][i], v[0][i], sums);
            }
            if (on1) {
#pragma unroll
                for (int i = 0; i < E / 2; i++) sums = fma2(v[1][i], v[1][i], sums);
            }
            float sum, odd;
            split2(sums, sum, odd);
            sum += odd;
#pragma unroll
            for (int o = LP / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
            const float *weight = p.side[k].weight;
            if (weight) {
                const float inv = rsqrtf(sum * inv_d + p.eps);
#pragma unroll
                for (int c = 0; c < 2; c++) {
                    if (!(c ? on1 : on0)) continue;
#pragma unroll
                    for (int i = 0; i < E; i += 4) {
                        const float4 w = __ldg(reinterpret_cast<const float4 *>(weight + (c ? e1 : e0) + i));
                        v[c][i / 2] = mul2(v[c][i / 2], mul2(pair2(inv, inv), pair2(w.x, w.y)));
                        v[c][i / 2 + 1] = mul2(v[c][i / 2 + 1], mul2(pair2(inv, inv), pair2(w.z, w.w)));
                    }
                }
            }
        }
        f2 co[E / 2], si[E / 2];
#pragma unroll
        for (int i = 0; i < E; i += 4) {
            const int a = min(i ? a1 : a0, kRopeMaxD / 2 - 4);
            const float4 c = *reinterpret_cast<const float4 *>(cos_of[t] + a), s = *reinterpret_cast<const float4 *>(sin_of[t] + a);
            co[i / 2] = pair2(c.x, c.y), co[i / 2 + 1] = pair2(c.z, c.w);
            si[i / 2] = pair2(s.x, s.y), si[i / 2 + 1] = pair2(s.z, s.w);
        }
        if (p.interleaved) {
#pragma unroll
            for (int c = 0; c < 2; c++) {
                if (!(c ? turn1 : turn0)) continue;
#pragma unroll
                for (int i = 0; i < E / 2; i++) {
                    float a, b, cs[2], sn[2];
                    split2(v[c][i], a, b);
                    const int n = c * 4 + i;  // angle
                    split2(co[n / 2], cs[0], cs[1]);
                    split2(si[n / 2], sn[0], sn[1]);
                    v[c][i] = pair2(a * cs[n & 1] - b * sn[n & 1], b * cs[n & 1] + a * sn[n & 1]);
                }
            }
        } else if (turn0) {
#pragma unroll
            for (int i = 0; i < E / 2; i++) {
                const f2 a = v[0][i], b = v[1][i];
                v[0][i] = fma2(a, co[i], mul2(b, mul2(si[i], pair2(-1.0f, -1.0f))));
                v[1][i] = fma2(b, co[i], mul2(a, si[i]));
            }
        }
        if (row) {
            void *to = p.side[k].out;
            const long long at = (t0 + t) * p.side[k].out_stride + (k ? r - hq : r) * p.D + e0;
#pragma unroll
            for (int c = 0; c < 2; c++) {
                if (!(c ? on1 : on0)) continue;
                float y[E];
#pragma unroll
                for (int i = 0; i < E / 2; i++) split2(v[c][i], y[2 * i], y[2 * i + 1]);
                store_floats<OUT_BF, E>(to, at + (c ? e1 - e0 : 0), y);
            }
        }
    }
}

template <bool IN_BF, bool OUT_BF, int E, int LP, int TOKENS>
void rope_start(RopeParams &p, cudaStream_t stream) {
    constexpr int kRows = 32 / LP, kMaxWarps = kRopeThreads / 32;
    // a warp's steps, shared out evenly
    const int steps = (p.side[0].heads + p.side[1].heads + kRows - 1) / kRows;
    const int turns = (TOKENS * steps + kMaxWarps - 1) / kMaxWarps;
    p.step_rows = steps * kRows;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((p.T + TOKENS - 1) / TOKENS));
    cfg.blockDim = dim3(32 * ((TOKENS * steps + turns - 1) / turns));
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaLaunchKernelEx(&cfg, rope_kernel<IN_BF, OUT_BF, E, LP, TOKENS>, p);
}

template <bool IN_BF, bool OUT_BF, int E, int LP>
void rope_tokens(RopeParams &p, cudaStream_t stream) {
    // Four tokens a CTA where that fills its waves to four fifths (8,191 tokens of 40 heads of 128: 31.3 us
    // against 34.3 with one), one token elsewhere (2,600 tokens of 40 heads of 64: 6.2 us against 7.2).
    const long long ctas = ((long long)p.T + kRopeTokens - 1) / kRopeTokens, slots = (long long)sm_count() * kRopeCtas;
    if (5 * ctas >= 4 * slots * ((ctas + slots - 1) / slots)) rope_start<IN_BF, OUT_BF, E, LP, kRopeTokens>(p, stream);
    else rope_start<IN_BF, OUT_BF, E, LP, 1>(p, stream);
}

template <bool IN_BF, bool OUT_BF>
void rope_launch(RopeParams &p, cudaStream_t stream) {
    if (p.interleaved || p.R % 16 == 0) {
        if (p.D <= 32) rope_tokens<IN_BF, OUT_BF, 8, 2>(p, stream);
        else if (p.D <= 64) rope_tokens<IN_BF, OUT_BF, 8, 4>(p, stream);
        else if (p.D <= 128) rope_tokens<IN_BF, OUT_BF, 8, 8>(p, stream);
        else rope_tokens<IN_BF, OUT_BF, 8, 16>(p, stream);
    } else {
        if (p.D <= 32) rope_tokens<IN_BF, OUT_BF, 4, 4>(p, stream);
        else if (p.D <= 128) rope_tokens<IN_BF, OUT_BF, 4, 16>(p, stream);
        else rope_tokens<IN_BF, OUT_BF, 4, 32>(p, stream);
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
    p.T = (int)r->T;
    p.D = r->D;
    p.R = r->R;
    p.interleaved = r->interleaved;
    p.eps = r->eps;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (r->in_type == SHERRY_BF16) {
        if (r->out_type == SHERRY_BF16) rope_launch<true, true>(p, s);
        else rope_launch<true, false>(p, s);
    } else {
        if (r->out_type == SHERRY_BF16) rope_launch<false, true>(p, s);
        else rope_launch<false, false>(p, s);
    }
    return launch_status("sherry_qk_norm_rope");
}
