// kv4.cu -- the 4-bit key/value cache: coding new tokens into it, reading them back.
#include <cuda_bf16.h>

#include "kv4.cuh"

namespace sherry {

// First bad page number or length met by a kernel of this cache (see sherry_device_error).
__device__ unsigned int g_kv4_device_error = 0;

namespace {

constexpr int kKvThreads = 256;

struct KvIo {
    void *k, *v;
    long long k_stride, v_stride;
};

// min and max that keep a NaN
__device__ __forceinline__ float min_nan(float a, float b) {
    float d;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}
__device__ __forceinline__ float max_nan(float a, float b) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}

// Eight consecutive elements as fp32.
template <bool BF>
__device__ __forceinline__ void load8(const void *base, long long at, float (&x)[8]) {
    if (BF) {
        const uint4 u = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(base) + at);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; i++) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    } else {
        const float4 *f = reinterpret_cast<const float4 *>(static_cast<const float *>(base) + at);
        const float4 a = f[0], b = f[1];
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
        x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    }
}

// A row of D elements is D / 8 lanes of eight elements, one code word each.  A
// thread's row index runs over (row, head, K or V): neighbouring lanes read
// neighbouring memory of the tensors.
template <int D, bool BF, bool WRITE>
__global__ void __launch_bounds__(kKvThreads)
    kv4_rows_kernel(const __grid_constant__ Kv4View c, const __grid_constant__ KvIo io, unsigned int *err) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    constexpr int L = D / 8;
    const int sub = threadIdx.x & (L - 1);
    const long long i = ((long long)blockIdx.x * kKvThreads + threadIdx.x) / L;
    const int per = 2 * c.H;
    const long long t = i / per;
    const int rest = (int)(i - t * per);
    const int kv = rest >= c.H ? 1 : 0, h = rest - kv * c.H;
    int b = 0, pos = -1, page = -1;
    if (t < c.T && kv4_find(c, (int)t, b, pos) && pos >= 0) page = kv4_page(c, b, pos, err);
    // a row's lanes share t, h and kv, so they leave together; the shuffles below
    // name only the row's lanes
    if (page < 0) return;
    const int slot = pos % SHERRY_KV4_PAGE;
    uint8_t *blk = kv4_block<D>(c, page, h, kv);
    uint32_t *code = reinterpret_cast<uint32_t *>(blk + slot * Kv4<D>::kRow) + sub;
    uint32_t *sm = reinterpret_cast<uint32_t *>(blk + Kv4<D>::kCodes) + slot;
    void *base = kv ? io.v : io.k;
    const long long at = t * (kv ? io.v_stride : io.k_stride) + (long long)h * D + 8 * sub;
    if (WRITE) {
        float x[8];
        load8<BF>(base, at, x);
        float lo = x[0], hi = x[0];
#pragma unroll
        for (int j = 1; j < 8; j++) {
            lo = min_nan(lo, x[j]);
            hi = max_nan(hi, x[j]);
        }
        const uint32_t mask = (L == 32 ? 0xFFFFFFFFu : ((1u << L) - 1u)) << ((threadIdx.x & 31) & ~(L - 1));
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) {
            lo = min_nan(lo, __shfl_xor_sync(mask, lo, o));
            hi = max_nan(hi, __shfl_xor_sync(mask, hi, o));
        }
        const uint32_t s16 = __bfloat16_as_ushort(__float2bfloat16_rn(__fmul_rn(__fsub_rn(hi, lo), 1.0f / 15.0f)));
        const uint32_t m16 = __bfloat16_as_ushort(__float2bfloat16_rn(lo));
        uint32_t pair = s16 | (m16 << 16);
        const float s = kv4_step(pair), m = kv4_low(pair);
        uint32_t word = 0;
        if (!(isfinite(s) && isfinite(m))) {
            pair = 0x7FFF7FFFu;  // NaN, NaN
        } else if (s < 7.52316384526264e-37f) {  // 2^-120: 1 / s would overflow soon after
            pair &= 0xFFFF0000u;
        } else {
            const float inv = __frcp_rn(s);
#pragma unroll
            for (int j = 0; j < 8; j++) {
                const float q = rintf(__fmul_rn(__fsub_rn(x[j], m), inv));
                word |= (uint32_t)fminf(fmaxf(q, 0.0f), 15.0f) << (4 * j);
            }
        }
        *code = word;
        if (sub == 0) *sm = pair;
    } else {
        const uint32_t word = *code, pair = *sm;
        const float s = kv4_step(pair), m = kv4_low(pair);
        float x[8];
#pragma unroll
        for (int j = 0; j < 8; j++) x[j] = __fmaf_rn(s, (float)((word >> (4 * j)) & 15u), m);
        if (BF) {
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; j++) {
                const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * j], x[2 * j + 1]);
                w[j] = *reinterpret_cast<const uint32_t *>(&v);
            }
            *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(base) + at) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
            float4 *f = reinterpret_cast<float4 *>(static_cast<float *>(base) + at);
            f[0] = make_float4(x[0], x[1], x[2], x[3]);
            f[1] = make_float4(x[4], x[5], x[6], x[7]);
        }
    }
}

template <int D, bool BF, bool WRITE>
void rows_launch(const Kv4View &c, const KvIo &io, unsigned int *err, cudaStream_t stream) {
    const long long threads = (long long)c.T * 2 * c.H * (D / 8);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((threads + kKvThreads - 1) / kKvThreads));
    cfg.blockDim = dim3(kKvThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaLaunchKernelEx(&cfg, kv4_rows_kernel<D, BF, WRITE>, c, io, err);
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
    if (c->T * 2 * c->H * (c->D / 8) / kKvThreads >= 0x7FFFFFFF) return SHERRY_ERR_UNSUPPORTED;
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
