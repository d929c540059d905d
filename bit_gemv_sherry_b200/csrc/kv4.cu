// kv4.cu -- the 4-bit key/value cache: coding new tokens into it, reading them back.
#include <cuda_bf16.h>

#include "kv4.cuh"

namespace sherry {

// First bad page number or length met by a kernel of this cache (see sherry_device_error).
__device__ unsigned int g_kv4_device_error = 0;

namespace {

constexpr int kKvThreads = 256;
constexpr long long kManySteps = 148 * 128;  // warp steps of a wave or two

struct KvIo {
    void *k, *v;
    long long k_stride, v_stride;
};

// min and max of three that keep a NaN
__device__ __forceinline__ float min_nan(float a, float b, float c) {
    float d;
    asm("min.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
__device__ __forceinline__ float max_nan(float a, float b, float c) {
    float d;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// Eight consecutive elements as they are in memory, and as fp32.
template <bool BF>
__device__ __forceinline__ void load8(const void *base, long long at, uint4 (&u)[BF ? 1 : 2]) {
    if (BF) {
        u[0] = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(base) + at);
    } else {
        const uint4 *f = reinterpret_cast<const uint4 *>(static_cast<const float *>(base) + at);
        u[0] = f[0];
        u[BF ? 0 : 1] = f[1];
    }
}
template <bool BF>
__device__ __forceinline__ void floats8(const uint4 (&u)[BF ? 1 : 2], float (&x)[8]) {
    if (BF) {
        const uint32_t w[4] = {u[0].x, u[0].y, u[0].z, u[0].w};
#pragma unroll
        for (int i = 0; i < 4; i++) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 2; i++) {
            const uint4 v = u[BF ? 0 : i];
            x[4 * i] = __uint_as_float(v.x), x[4 * i + 1] = __uint_as_float(v.y);
            x[4 * i + 2] = __uint_as_float(v.z), x[4 * i + 3] = __uint_as_float(v.w);
        }
    }
}

// min and max of two bf16 pairs, keeping a NaN
__device__ __forceinline__ uint32_t min2_nan(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t max2_nan(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// Smallest and largest element of a row of L lanes.  bf16: both in one register, (min, -max), so that one
// shuffle a level serves both.
template <bool BF, int L, int C>
__device__ __forceinline__ void row_range(const uint4 (&u)[C][BF ? 1 : 2], const float (&x)[C][8], float &lo, float &hi) {
    if (BF) {
        uint32_t a = u[0][0].x, b = u[0][0].x;
#pragma unroll
        for (int c = 0; c < C; c++) {
            const uint32_t w[4] = {u[c][0].x, u[c][0].y, u[c][0].z, u[c][0].w};
#pragma unroll
            for (int i = c ? 0 : 1; i < 4; i++) a = min2_nan(a, w[i]), b = max2_nan(b, w[i]);
        }
        b ^= 0x80008000u;
        // (a.lo, b.lo) and (a.hi, b.hi)
        uint32_t m = min2_nan(__byte_perm(a, b, 0x5410), __byte_perm(a, b, 0x7632));
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) m = min2_nan(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        lo = __uint_as_float(m << 16);
        hi = -__uint_as_float(m & 0xFFFF0000u);
    } else {
        lo = x[0][0], hi = x[0][0];
#pragma unroll
        for (int c = 0; c < C; c++)
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
                lo = min_nan(lo, x[c][j], x[c][j + 1]);
                hi = max_nan(hi, x[c][j], x[c][j + 1]);
            }
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) {
            const float other = __shfl_xor_sync(0xFFFFFFFFu, lo, o), top = __shfl_xor_sync(0xFFFFFFFFu, hi, o);
            lo = min_nan(lo, other, other);
            hi = max_nan(hi, top, top);
        }
    }
}

// A row of D elements is D / (8 C) lanes of C chunks of eight elements, a code word each.  A warp takes up to
// STEPS times 32 lanes' worth of one token's rows (the key heads, then the value heads): the token's page is
// looked up once, and all of the warp's loads are under way before the first is used.  One read and one
// write per element bound it, if the conversions keep to the fast pipes: a code becomes a float, and a
// float a code, by adding 2^23 or 1.5 2^23 (the conversion instructions run at a quarter of the rate:
// 32,768 tokens of 8 heads of 128, bf16, took 139 us to write and read with them, 82 without, and 62 with four
// chunks a lane, which share the row's step and addresses; the bytes take 53).
template <int D, int C, int STEPS>
__host__ __device__ constexpr int rows_per_warp() { return STEPS * 32 / (D / (8 * C)); }

template <int D, bool BF, bool WRITE, int C, int STEPS>
__global__ void __launch_bounds__(kKvThreads)
    kv4_rows_kernel(const __grid_constant__ Kv4View c, const __grid_constant__ KvIo io, unsigned int *err) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    constexpr int L = D / (8 * C), kRows = rows_per_warp<D, C, STEPS>();
    const int lane = threadIdx.x & 31, sub = lane & (L - 1);
    const unsigned parts = (unsigned)(2 * c.H + kRows - 1) / kRows;
    const unsigned w = blockIdx.x * (kKvThreads / 32) + (threadIdx.x >> 5);
    const int t = (int)(w / parts), row0 = (int)(w % parts) * kRows + lane / L;
    if (t >= c.T) return;
    // row r: head r of the keys, or head r - H of the values; chunk k of the lane is elements 8 (sub + k L) ...
    const long long k_at = t * io.k_stride + 8 * sub, v_at = t * io.v_stride - (long long)c.H * D + 8 * sub;
    auto at = [&](int r) { return (r < c.H ? k_at : v_at) + (long long)r * D; };
    uint4 u[STEPS][C][BF ? 1 : 2];
    if (WRITE) {
#pragma unroll
        for (int i = 0; i < STEPS; i++) {
            const int r = row0 + i * (32 / L);
            if (r >= 2 * c.H) continue;
#pragma unroll
            for (int k = 0; k < C; k++) load8<BF>(r < c.H ? io.k : io.v, at(r) + 8 * L * k, u[i][k]);
        }
    }
    int b = 0, pos = -1, page = -1;
    if (kv4_find(c, t, b, pos) && pos >= 0) page = kv4_page(c, b, pos, err);
    if (page < 0) return;
    const int slot = pos % SHERRY_KV4_PAGE;
    uint8_t *first = kv4_block<D>(c, page, 0, 0);
    // (below 2^31 for 65,535 heads)
    auto block = [&](int r) { return first + (unsigned)(r < c.H ? 2 * r : 2 * (r - c.H) + 1) * (unsigned)Kv4<D>::kBlock; };
    if (WRITE) {
#pragma unroll
        for (int i = 0; i < STEPS; i++) {
            const int r = row0 + i * (32 / L);
            const bool in = r < 2 * c.H;
            float x[C][8], lo, hi;
#pragma unroll
            for (int k = 0; k < C; k++) floats8<BF>(u[i][k], x[k]);
            row_range<BF, L, C>(u[i], x, lo, hi);  // (lanes past the last row take part with whatever they hold)
            const uint32_t s16 = __bfloat16_as_ushort(__float2bfloat16_rn(__fmul_rn(__fsub_rn(hi, lo), 1.0f / 15.0f)));
            const uint32_t m16 = __bfloat16_as_ushort(__float2bfloat16_rn(lo));
            uint32_t pair = s16 | (m16 << 16);
            const float s = kv4_step(pair), m = kv4_low(pair);
            const bool bad = !(fabsf(s) < INFINITY && fabsf(m) < INFINITY);
            const bool flat = s < 7.52316384526264e-37f;  // 2^-120: 1 / s would overflow soon after
            uint32_t word[C] = {};
            if (!bad && !flat) {
                const float inv = __frcp_rn(s);
                // Every operation is monotone, so the row's ends tell whether any code needs clamping.
                const bool inside = __fmul_rn(__fsub_rn(lo, m), inv) >= -0.5f && __fmul_rn(__fsub_rn(hi, m), inv) < 15.5f;
#pragma unroll
                for (int k = 0; k < C; k++) {
                    if (inside) {
#pragma unroll
                        for (int j = 0; j < 8; j += 2) {
                            float a, b;  // 0x4B400000 + rint (the product is not paired: it must be rounded before the sum)
                            split2(add2(pair2(x[k][j], x[k][j + 1]), pair2(-m, -m)), a, b);
                            split2(add2(pair2(__fmul_rn(a, inv), __fmul_rn(b, inv)), pair2(12582912.0f, 12582912.0f)), a, b);
                            word[k] += (__float_as_uint(a) << (4 * j)) + (__float_as_uint(b) << (4 * j + 4));
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 8; j++) {
                            // clamped first: the bounds are whole numbers, so the rounding commutes with them
                            const float q = fminf(fmaxf(__fmul_rn(__fsub_rn(x[k][j], m), inv), 0.0f), 15.0f);
                            word[k] += __float_as_uint(__fadd_rn(q, 12582912.0f)) << (4 * j);
                        }
                    }
                    word[k] -= 0x3F400000u;  // what is left of the eight constants: 0x4B400000 (1 + 16 + 256) modulo 2^32
                }
            }
            if (bad) pair = 0x7FFF7FFFu;        // NaN, NaN
            else if (flat) pair &= 0xFFFF0000u;
            if (in) {
                uint8_t *blk = block(r);
#pragma unroll
                for (int k = 0; k < C; k++) reinterpret_cast<uint32_t *>(blk + slot * Kv4<D>::kRow)[sub + k * L] = word[k];
                if (sub == 0) reinterpret_cast<uint32_t *>(blk + Kv4<D>::kCodes)[slot] = pair;
            }
        }
    } else {
        uint32_t word[STEPS][C], pair[STEPS];
#pragma unroll
        for (int i = 0; i < STEPS; i++) {
            const int r = row0 + i * (32 / L);
            if (r >= 2 * c.H) continue;
            const uint8_t *blk = block(r);
#pragma unroll
            for (int k = 0; k < C; k++) word[i][k] = reinterpret_cast<const uint32_t *>(blk + slot * Kv4<D>::kRow)[sub + k * L];
            pair[i] = reinterpret_cast<const uint32_t *>(blk + Kv4<D>::kCodes)[slot];
        }
#pragma unroll
        for (int i = 0; i < STEPS; i++) {
            const int r = row0 + i * (32 / L);
            if (r >= 2 * c.H) continue;
            const float s = kv4_step(pair[i]), m = kv4_low(pair[i]);
            // code j stays where it is in its half word: 2^23 + c 16^j, so the step is s 16^-j
            const float sj[4] = {s, s * 0.0625f, s * 0.00390625f, s * 0.000244140625f};
            void *base = r < c.H ? io.k : io.v;
#pragma unroll
            for (int k = 0; k < C; k++) {
                float x[8];
#pragma unroll
                for (int j = 0; j < 8; j += 2) {
                    const uint32_t half = j < 4 ? word[i][k] : word[i][k] >> 16;
                    const f2 code = add2(pair2u((half & (15u << (4 * (j & 3)))) | 0x4B000000u, (half & (15u << (4 * (j & 3) + 4))) | 0x4B000000u),
                                         pair2(-8388608.0f, -8388608.0f));  // exact
                    split2(fma2(pair2(sj[j & 3], sj[(j & 3) + 1]), code, pair2(m, m)), x[j], x[j + 1]);
                }
                if (BF) {
                    uint32_t w[4];
#pragma unroll
                    for (int j = 0; j < 4; j++) {
                        const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * j], x[2 * j + 1]);
                        w[j] = *reinterpret_cast<const uint32_t *>(&v);
                    }
                    *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(base) + at(r) + 8 * L * k) = make_uint4(w[0], w[1], w[2], w[3]);
                } else {
                    float4 *f = reinterpret_cast<float4 *>(static_cast<float *>(base) + at(r) + 8 * L * k);
                    f[0] = make_float4(x[0], x[1], x[2], x[3]);
                    f[1] = make_float4(x[4], x[5], x[6], x[7]);
                }
            }
        }
    }
}

template <int D, bool BF, bool WRITE, int C, int STEPS>
void rows_launch_steps(const Kv4View &c, const KvIo &io, unsigned int *err, cudaStream_t stream) {
    const long long threads = 32LL * c.T * ((2 * c.H + rows_per_warp<D, C, STEPS>() - 1) / rows_per_warp<D, C, STEPS>());
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((threads + kKvThreads - 1) / kKvThreads));
    cfg.blockDim = dim3(kKvThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaLaunchKernelEx(&cfg, kv4_rows_kernel<D, BF, WRITE, C, STEPS>, c, io, err);
}

template <int D, bool BF, bool WRITE>
void rows_launch(const Kv4View &c, const KvIo &io, unsigned int *err, cudaStream_t stream) {
    // Few rows: a chunk per lane and a step per warp, for the latency (16 tokens of 8 heads of 64, written and
    // read: 3.5 us against 5.7).  Many: two steps for the loads under way, of rows on four lanes in bf16 and
    // eight in fp32 (a load or store of the warp then has at least 64 bytes in a row): 2,500 tokens of 8 heads
    // of 128, bf16, 10.1 us against 12.1; 32,768, 62 us against 130 (rows on 16 lanes and four steps 82, on
    // two lanes 92); fp32, 126 us against 139 (on four lanes 149).
    if ((long long)c.T * 2 * c.H * (D / 8) / 32 < kManySteps) rows_launch_steps<D, BF, WRITE, 1, 1>(c, io, err, stream);
    else rows_launch_steps<D, BF, WRITE, BF ? D / 32 : D / 64, 2>(c, io, err, stream);
}

template <bool WRITE>
sherry_status rows_call(const sherry_kv4 *c, void *k, void *v, int type, int64_t k_stride, int64_t v_stride,
                        sherry_stream_t stream, const char *what) {
    const sherry_status st = kv4_check(c);
    if (st != SHERRY_OK) return st;
    if (!k || !v) return SHERRY_ERR_NULL;
    if (type != SHERRY_F32 && type != SHERRY_BF16) return SHERRY_ERR_UNSUPPORTED;
    if (k_stride < (int64_t)c->H * c->D || v_stride < (int64_t)c->H * c->D) return SHERRY_ERR_SHAPE;
    const int unit = type == SHERRY_F32 ? 4 : 8;
    if (!aligned(k, 16) || !aligned(v, 16) || k_stride % unit || v_stride % unit) return SHERRY_ERR_ALIGN;
    if (c->T * 2 * c->H >= 0x7FFFFFFF) return SHERRY_ERR_UNSUPPORTED;
    const Kv4View view = kv4_view(c);
    const KvIo io = {k, v, k_stride, v_stride};
    unsigned int *err = kv4_error_address();
    if (!err) return SHERRY_ERR_CUDA;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (c->D == 64) {
        if (type == SHERRY_BF16) rows_launch<64, true, WRITE>(view, io, err, s);
        else rows_launch<64, false, WRITE>(view, io, err, s);
    } else {
        if (type == SHERRY_BF16) rows_launch<128, true, WRITE>(view, io, err, s);
        else rows_launch<128, false, WRITE>(view, io, err, s);
    }
    return launch_status(what);
}

}  // namespace

// Device address of the error word, looked up once per device and context.
unsigned int *kv4_error_address() {
    static std::atomic<unsigned long long> ctx[64];
    static std::atomic<unsigned int *> at[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) dev = 0;
    const int i = dev & 63;
    const unsigned long long id = context_id();
    unsigned int *p = at[i].load(std::memory_order_acquire);
    if (p && id != 0 && ctx[i].load(std::memory_order_acquire) == id) return p;
    void *q = nullptr;
    const cudaError_t e = cudaGetSymbolAddress(&q, g_kv4_device_error);
    if (e != cudaSuccess) {
        set_last_error("sherry_kv4 (error word)", e);
        return nullptr;
    }
    at[i].store(static_cast<unsigned int *>(q), std::memory_order_release);
    ctx[i].store(id, std::memory_order_release);
    return static_cast<unsigned int *>(q);
}

sherry_status kv4_device_error() {
    unsigned int v = 0;
    cudaError_t err = cudaMemcpyFromSymbol(&v, g_kv4_device_error, sizeof(v));
    if (err != cudaSuccess) {
        set_last_error("sherry_device_error (read)", err);
        return SHERRY_ERR_CUDA;
    }
    if (v != 0) {
        const unsigned int zero = 0;
        err = cudaMemcpyToSymbol(g_kv4_device_error, &zero, sizeof(zero));
        if (err != cudaSuccess) {
            set_last_error("sherry_device_error (clear)", err);
            return SHERRY_ERR_CUDA;
        }
    }
    return static_cast<sherry_status>(v);
}

sherry_status kv4_check(const sherry_kv4 *c) {
    if (!c || !c->cache || !c->page_table || !c->ctx_lens) return SHERRY_ERR_NULL;
    if (c->pages < 1 || c->H < 1 || c->width < 1 || c->table_stride < c->width || c->B < 1 || c->T < 1)
        return SHERRY_ERR_SHAPE;
    if (!c->cu_q && c->T != c->B) return SHERRY_ERR_SHAPE;
    if (c->D != 64 && c->D != 128) return SHERRY_ERR_UNSUPPORTED;
    // positions and row numbers are 32-bit in the kernels; byte offsets are 64-bit
    if (c->pages > 0x7FFFFFFF || c->H > 65535 || c->width > 0x7FFFFFFF / SHERRY_KV4_PAGE || c->B > 65535 ||
        c->T > 0x7FFFFFFF)
        return SHERRY_ERR_UNSUPPORTED;
    if (!aligned(c->cache, 16) || !aligned(c->page_table, 4) || !aligned(c->ctx_lens, 4) || !aligned(c->cu_q, 4))
        return SHERRY_ERR_ALIGN;
    return SHERRY_OK;
}

Kv4View kv4_view(const sherry_kv4 *c) {
    Kv4View v;
    v.cache = static_cast<uint8_t *>(c->cache);
    v.table = c->page_table;
    v.lens = c->ctx_lens;
    v.cu = c->cu_q;
    v.pages = c->pages;
    v.table_stride = c->table_stride;
    v.H = c->H;
    v.width = (int)c->width;
    v.B = (int)c->B;
    v.T = (int)c->T;
    return v;
}

}  // namespace sherry

extern "C" size_t sherry_kv4_bytes(int64_t pages, int H, int D) {
    if (pages < 1 || pages > 0x7FFFFFFF || H < 1 || H > 65535 || (D != 64 && D != 128)) return 0;
    return (size_t)pages * (size_t)H * 2 * (size_t)(SHERRY_KV4_PAGE * (D / 2 + 4));
}

extern "C" sherry_status sherry_kv4_write(const sherry_kv4 *c, const void *k, const void *v, int type,
                                          int64_t k_stride, int64_t v_stride, sherry_stream_t stream) {
    return sherry::rows_call<true>(c, const_cast<void *>(k), const_cast<void *>(v), type, k_stride, v_stride,
                                   stream, "sherry_kv4_write");
}

extern "C" sherry_status sherry_kv4_read(const sherry_kv4 *c, void *k, void *v, int type, int64_t k_stride,
                                         int64_t v_stride, sherry_stream_t stream) {
    return sherry::rows_call<false>(c, k, v, type, k_stride, v_stride, stream, "sherry_kv4_read");
}
