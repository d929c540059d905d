// attn.cuh -- shared by the attention kernels (internal).
//
// For a row q (a new token and a query head) and the tokens t it sees,
//     out = sum_t p_t v_t / sum_t p_t,   p_t = 2^(x_t - m),   x_t = scale log2(e) (q . k_t).
// With k_t = m_t + s_t c_t and c_t in 0 .. 15,  q . k_t = s_t (q . c_t) + m_t sum(q): the first
// product runs on the codes, which fp16 holds exactly, and the step and low end come in after it.
// Likewise sum_t p_t v_t = sum_t (p_t s_t) (c_t - 8) + sum_t p_t (m_t + 8 s_t).
#pragma once

#include <cuda_bf16.h>

#include "kv4.cuh"

namespace sherry {

constexpr float kLog2e = 1.4426950408889634f;

struct AttnParams {
    Kv4View c;
    const uint16_t *q;
    uint16_t *out;
    float *ws;          // few rows: [2 grid][rows][D] sums, then [2 grid][rows] pairs (m, l)
    long long q_stride, out_stride;
    long long wait_limit;
    int g;              // query heads per key/value head
    int grid;           // few rows: runs
    int few_rows;       // sequences with more rows (new tokens times g) are the tile kernel's
    float scale2;       // scale * log2(e)
    unsigned int *err;
};

// Sequences of more than p.few_rows rows: 256 rows a CTA, two tiles of 128 on the tensor cores.
sherry_status attn_tile_launch(const AttnParams &p, int D, cudaStream_t stream);

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// 2^e for any e (0 or the largest power where that is out of range).
__device__ __forceinline__ float pow2(int e) {
    return e < -126 ? (e < -149 ? 0.0f : __int_as_float(1 << (e + 149))) : __int_as_float((min(e, 127) + 127) << 23);
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

}  // namespace sherry
