// attn_tile.cu -- causal attention over the 4-bit cache for sequences with many new tokens
// (prompts, chunks of prompts): both products on the tcgen05 tensor cores.
//
// A CTA takes 256 rows of one key/value head, as two tiles of 128, so that each decoded key and
// value serves both (and all query heads of the group: a row is a new token and a query head).
// Per 128 tokens:
//     S = Q C_k^T        codes c - 8 as bf16, K-major, in shared memory; S in tensor memory
//     x = s_k S + (m_k + 8 s_k) sum(q)      (times scale log2 e), masked at the diagonal only
//     P = bf16(2^(x - m) s_v) back into S's tensor memory, the A operand of
//     O += P C_v         codes transposed to [D][tokens], so that both operands are K-major
// and in fp32 registers  l += sum p,  corr += sum p (m_v + 8 s_v);  out = (O + corr) / l.
// Roles: warps 0-3 and 4-7 the softmax of a tile each (a thread owns a row: no shuffles), warps
// 8-9 decode keys, 10-11 values, warp 12 issues the products.  The tiles alternate: while one's
// softmax runs, the tensor cores work for the other.
// The bound is shared by the exponentials (16 a clock and SM: 2048 clocks per 256 x 128 scores),
// the products (1024 clocks for heads of 64, 2048 for 128) and the issue of about six
// instructions per score in 64-bit pairs.
#include <algorithm>

#include "attn.cuh"

namespace sherry {
namespace {

constexpr int kRowsTile = 128;
constexpr int kRowsCta = 2 * kRowsTile;
constexpr int kKeys = 128;                 // tokens per step: two pages
constexpr int kTileThreads = 13 * 32;
constexpr int kScaleSlots = 4;
constexpr int kAllSeen = 0x7FFFFFFF - 2 * kKeys;
constexpr int kTmemCols = 512;             // S0, S1 (128 columns each), O0, O1 (D each)
constexpr long long kDrainLimit = 1000000000LL;

template <int D>
struct Tile {
    static constexpr int kQ = kRowsTile * D * 2;      // one tile's queries
    static constexpr int kOp = kKeys * D * 2;         // decoded keys or values of a step
    static constexpr int kScales = kScaleSlots * 4 * kKeys * 4;
    static constexpr int kBars = 256;
    // one CTA per SM in any case (its tensor memory), so heads of 64 ask for as much as keeps
    // a second one away
    static constexpr size_t kUse = 2 * kQ + 4 * kOp + kScales + kBars + 1024;
    static constexpr size_t kSmem = kUse < 120 * 1024 ? 120 * 1024 : kUse;
};

// D = fp32, A and B = bf16, both K-major, 128 x N
template <int N>
constexpr uint32_t kIdescBf16 = (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) |
                                ((uint32_t)(kRowsTile >> 4) << 24);

struct TileBars {
    uint64_t q_full, k_full[2], k_empty[2], v_full[2], v_empty[2], sc_full[kScaleSlots];
    uint64_t s_full[2], p_full[2], o_full[2], drain;
    uint32_t tmem;
    int abort;
    int there[kScaleSlots];  // bit 0, 1: the step's first, second page is in the cache
};

// ---- pairs of fp32 ----
using f2 = unsigned long long;
__device__ __forceinline__ f2 pair2(float a, float b) {
    f2 d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
    return d;
}
__device__ __forceinline__ f2 pair2u(uint32_t a, uint32_t b) {
    f2 d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ void split2(f2 v, float &a, float &b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
    f2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
    f2 d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
    f2 d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// Two codes as bf16 c - 8.
__device__ __forceinline__ uint32_t code_pair8(uint32_t x) {
    uint32_t d;
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(code_pair(x)), "r"(0x43084308u));
    return d;
}

// A row tile's place in the batch.
struct Place {
    int b, first, rows, len, tile;  // sequence, its first row, rows (tokens), length; tile of 256 rows
};

__device__ __forceinline__ int seq_tiles(const AttnParams &p, int b) {
    if (b >= p.c.B) return 0;
    int first, n;
    kv4_rows(p.c, b, first, n);
    const long long rows = (long long)n * p.g;
    return rows > p.few_rows ? (int)((rows + kRowsCta - 1) / kRowsCta) : 0;
}

// The i-th row tile of the batch, the longest of each sequence first (every lane of a full warp).
__device__ __forceinline__ bool find_tile(const AttnParams &p, int i, Place &w) {
    const int lane = threadIdx.x & 31;
    int base = 0;
    for (int b0 = 0; b0 < p.c.B; b0 += 32) {
        const int mine = seq_tiles(p, b0 + lane);
        int sum = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xFFFFFFFFu, sum, o);
            if (lane >= o) sum += v;
        }
        const unsigned hit = __ballot_sync(0xFFFFFFFFu, base + sum > i);
        if (hit) {
            const int l = __ffs(hit) - 1;
            w.b = b0 + l;
            w.tile = base + __shfl_sync(0xFFFFFFFFu, sum, l) - 1 - i;
            kv4_rows(p.c, w.b, w.first, w.rows);
            w.len = max(__ldg(p.c.lens + w.b), 0);
            return true;
        }
        base += __shfl_sync(0xFFFFFFFFu, sum, 31);
    }
    return false;
}

// One thread's row over one step of 128 tokens.
struct RowState {
    float m, l;      // reference of the exponentials, sum
    float corr;      // sum p (m_v + 8 s_v)
};

// Largest score of the row in this step (-inf if none is seen).
__device__ __forceinline__ float step_max(uint32_t s_tmem, const float *sc, float qsum, int seen, int there) {
    float mx = -INFINITY;
#pragma unroll 1
    for (int c0 = 0; c0 < kKeys; c0 += 32) {
        uint32_t r[32];
        tmem_ld32(s_tmem + c0, r);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 32; i++) {
            const float x = sc[c0 + i] * __uint_as_float(r[i]) + sc[kKeys + c0 + i] * qsum;
            const bool ok = c0 + i < seen && (there >> ((c0 + i) / SHERRY_KV4_PAGE) & 1);
            mx = fmaxf(mx, ok ? x : -INFINITY);
        }
    }
    return mx;
}

// Probabilities of the step against the reference m, packed for the second product; sum and corr of
// the step alone.  MASK: the row sees the step's first `seen` tokens, of pages that are there.
template <bool MASK>
__device__ __forceinline__ void step_probs(uint32_t s_tmem, const float *sc, float qsum, float ref, int seen, int there,
                                           uint32_t (&pk)[64], float &sum, float &corr) {
    const f2 q2 = pair2(qsum, qsum), nm = pair2(-ref, -ref);
    f2 sum2 = pair2(0.0f, 0.0f), corr2 = sum2;
#pragma unroll
    for (int c0 = 0; c0 < kKeys; c0 += 32) {
        uint32_t r[32];
        tmem_ld32(s_tmem + c0, r);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
            const ulonglong2 sk = *reinterpret_cast<const ulonglong2 *>(sc + c0 + i);
            const ulonglong2 mk = *reinterpret_cast<const ulonglong2 *>(sc + kKeys + c0 + i);
            const ulonglong2 sv = *reinterpret_cast<const ulonglong2 *>(sc + 2 * kKeys + c0 + i);
            const ulonglong2 cv = *reinterpret_cast<const ulonglong2 *>(sc + 3 * kKeys + c0 + i);
#pragma unroll
            for (int k = 0; k < 2; k++) {
                const int t = c0 + i + 2 * k;
                const f2 y = fma2(k ? sk.y : sk.x, pair2u(r[i + 2 * k], r[i + 2 * k + 1]), fma2(k ? mk.y : mk.x, q2, nm));
                float ya, yb;
                split2(y, ya, yb);
                bool oka = true, okb = true;
                if (MASK) {
                    const bool pg = there >> (t / SHERRY_KV4_PAGE) & 1;
                    oka = pg && t < seen;
                    okb = pg && t + 1 < seen;
                }
                const float pa = oka ? exp2_fast(ya) : 0.0f, pb = okb ? exp2_fast(yb) : 0.0f;
                const f2 p2 = pair2(pa, pb);
                sum2 = add2(sum2, p2);
                f2 sv2 = k ? sv.y : sv.x, cv2 = k ? cv.y : cv.x;
                if (MASK) {  // a token that is not seen may hold anything, NaN too
                    float a, b;
                    split2(sv2, a, b);
                    sv2 = pair2(oka ? a : 0.0f, okb ? b : 0.0f);
                    split2(cv2, a, b);
                    cv2 = pair2(oka ? a : 0.0f, okb ? b : 0.0f);
                }
                corr2 = fma2(p2, cv2, corr2);
                float a, b;
                split2(mul2(p2, sv2), a, b);
                pk[t / 2] = pack_bf16(a, b);
            }
        }
    }
    float a, b;
    split2(sum2, a, b);
    sum = a + b;
    split2(corr2, a, b);
    corr = a + b;
}

template <int D>
__global__ void __launch_bounds__(kTileThreads, 1) attn_tile_kernel(const __grid_constant__ AttnParams p) {
    using T = Tile<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    uint8_t *sq = smem, *sk = sq + 2 * T::kQ, *sv = sk + 2 * T::kOp;
    float *scales = reinterpret_cast<float *>(sv + 2 * T::kOp);  // [slot][s_k, m_k, s_v, m_v][128]
    TileBars *bar = reinterpret_cast<TileBars *>(reinterpret_cast<uint8_t *>(scales) + T::kScales);
    static_assert(sizeof(TileBars) <= T::kBars, "barriers");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int h = blockIdx.x % p.c.H;
    Place w;
    if (!find_tile(p, blockIdx.x / p.c.H, w)) return;
    const int nrow = w.rows * p.g, row0 = w.tile * kRowsCta, pos0 = w.len - w.rows;
    const int hi_row = min(row0 + kRowsCta, nrow) - 1;
    // steps: up to the last token that the last row sees, and no further than the table
    const int keys = min(pos0 + hi_row / p.g + 1, p.c.width * SHERRY_KV4_PAGE);
    const int steps = keys > 0 ? (keys + kKeys - 1) / kKeys : 0;
    const long long limit = p.wait_limit;

    if (threadIdx.x == 0) {
        mbar_init(&bar->q_full, kRowsCta);
        for (int i = 0; i < 2; i++) {
            mbar_init(&bar->k_full[i], 64);
            mbar_init(&bar->v_full[i], 64);
            mbar_init(&bar->k_empty[i], 1);
            mbar_init(&bar->v_empty[i], 1);
            mbar_init(&bar->s_full[i], 1);
            mbar_init(&bar->p_full[i], kRowsTile);
            mbar_init(&bar->o_full[i], 1);
        }
        for (int i = 0; i < kScaleSlots; i++) mbar_init(&bar->sc_full[i], 128);
        mbar_init(&bar->drain, 1);
        bar->abort = 0;
        if (w.len > p.c.width * SHERRY_KV4_PAGE) atomicCAS(p.err, 0u, (unsigned int)SHERRY_ERR_INDEX);
        fence_mbar_init();
    }
    if (warp == 12) {
        tmem_alloc(&bar->tmem, kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bar->tmem;
    volatile int *abort = &bar->abort;

    if (warp < 8) {
        // ---------------- softmax: a thread owns a row ----------------
        const int i = warp >> 2, r = threadIdx.x & 127;      // tile, row of the tile
        const int rw = row0 + i * kRowsTile + r;
        const bool live = rw < nrow;
        const int last = live ? pos0 + rw / p.g : kAllSeen;  // a row past the end sees all and is dropped
        const int lo_row = row0 + i * kRowsTile;
        const int last_min = lo_row < nrow ? pos0 + lo_row / p.g : kAllSeen;
        // queries to shared memory (elements of each eight in the order 0 4 1 5 2 6 3 7, as the codes
        // come out of their words), K-major with 128-byte rows swizzled
        float qsum = 0.0f;
        {
            const uint16_t *src = p.q + (long long)(w.first + rw / p.g) * p.q_stride + (long long)(h * p.g + rw % p.g) * D;
            uint8_t *dst = sq + i * T::kQ + r * 128;
#pragma unroll
            for (int c = 0; c < D / 8; c++) {
                uint4 u = make_uint4(0, 0, 0, 0);
                if (live) u = *reinterpret_cast<const uint4 *>(src + 8 * c);
                const uint32_t e[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                for (int k = 0; k < 4; k++)
                    qsum += __uint_as_float(e[k] << 16) + __uint_as_float(e[k] & 0xFFFF0000u);
                const uint4 v = make_uint4(prmt(u.x, u.z, 0x5410), prmt(u.x, u.z, 0x7632), prmt(u.y, u.w, 0x5410),
                                           prmt(u.y, u.w, 0x7632));
                *reinterpret_cast<uint4 *>(dst + (c / 8) * (kRowsTile * 128) + (((c & 7) ^ (r & 7)) << 4)) = v;
            }
        }
        fence_proxy_async_smem();
        mbar_arrive(&bar->q_full);
        const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t s_tmem = tmem + lane_base + i * kKeys;
        const uint32_t o_tmem = tmem + lane_base + 2 * kKeys + i * D;
        float m = -INFINITY, l = 0.0f, corr = 0.0f;
        bool dead = false;
        for (int j = 0; j < steps; j++) {
            const int slot = j % kScaleSlots;
            if (!__all_sync(0xFFFFFFFFu, mbar_wait(&bar->sc_full[slot], (j / kScaleSlots) & 1, abort, p.err, limit) &&
                                             mbar_wait(&bar->s_full[i], j & 1, abort, p.err, limit))) {
                dead = true;
                break;
            }
            tc_fence_after();
            const float *sc = scales + slot * 4 * kKeys;
            const int there = bar->there[slot], t0 = j * kKeys;
            const int seen = min(max(last - t0 + 1, 0), kKeys);
            const bool whole = there == 3 && t0 + kKeys - 1 <= last_min;
            uint32_t pk[64];
            float sum, cs;
            bool fresh = j == 0;
            for (;;) {
                if (fresh) {
                    // set the reference to the row's maximum so far and bring the sums to it
                    const float mx = fmaxf(m, step_max(s_tmem, sc, qsum, seen, there));
                    const float f = m == -INFINITY ? 0.0f : exp2_fast(m - mx);
                    m = mx;
                    l *= f;
                    corr *= f;
                    if (j > 0) {  // the products up to step j - 1 are complete: S of step j was issued after them
#pragma unroll 1
                        for (int c0 = 0; c0 < D; c0 += 32) {
                            uint32_t o[32];
                            tmem_ld32(o_tmem + c0, o);
                            tmem_ld_wait();
#pragma unroll
                            for (int k = 0; k < 32; k++) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                            tmem_st32(o_tmem + c0, o);
                        }
                        tmem_st_wait();
                    }
                }
                const float ref = m == -INFINITY ? 0.0f : m;
                if (whole) step_probs<false>(s_tmem, sc, qsum, ref, seen, there, pk, sum, cs);
                else step_probs<true>(s_tmem, sc, qsum, ref, seen, there, pk, sum, cs);
                // The reference may lag behind the maximum: only a step whose probabilities add up to more
                // than 2^16 moves it, and is then taken again; so does the first step in which a row sees
                // anything (the pages before may be missing).
                if (fresh || !__any_sync(0xFFFFFFFFu, sum > 65536.0f || (m == -INFINITY && seen > 0))) break;
                fresh = true;
            }
            l += sum;
            corr += cs;
            {
                uint32_t half[32];
#pragma unroll
                for (int k = 0; k < 32; k++) half[k] = pk[k];
                tmem_st32(s_tmem, half);
#pragma unroll
                for (int k = 0; k < 32; k++) half[k] = pk[32 + k];
                tmem_st32(s_tmem + 32, half);
            }
            tmem_st_wait();
            tc_fence_before();
            mbar_arrive(&bar->p_full[i]);
        }
        if (!dead && steps > 0)
            dead = !__all_sync(0xFFFFFFFFu, mbar_wait(&bar->o_full[i], 0, abort, p.err, limit));
        if (!dead) {
            tc_fence_after();
            const float inv = l == 0.0f ? 0.0f : 1.0f / l;
            uint16_t *dst = p.out + (long long)(w.first + rw / p.g) * p.out_stride + (long long)(h * p.g + rw % p.g) * D;
#pragma unroll 1
            for (int c0 = 0; c0 < D; c0 += 32) {
                uint32_t o[32];
                if (steps > 0) {
                    tmem_ld32(o_tmem + c0, o);
                    tmem_ld_wait();
                } else {
#pragma unroll
                    for (int k = 0; k < 32; k++) o[k] = 0;
                }
                if (live) {
#pragma unroll
                    for (int k = 0; k < 32; k += 8) {
                        uint32_t u[4];
#pragma unroll
                        for (int e = 0; e < 4; e++)
                            u[e] = pack_bf16((__uint_as_float(o[k + 2 * e]) + corr) * inv,
                                             (__uint_as_float(o[k + 2 * e + 1]) + corr) * inv);
                        *reinterpret_cast<uint4 *>(dst + c0 + k) = make_uint4(u[0], u[1], u[2], u[3]);
                    }
                }
            }
        }
    } else if (warp < 10) {
        // ---------------- keys: two tokens per thread ----------------
        const int th = threadIdx.x - 256;  // 0 .. 63: token th of the step's first and second page
        for (int j = 0; j < steps; j++) {
            const int slot = j % kScaleSlots, s = j & 1;
            uint4 u[2][D / 32];
            uint32_t sm[2];
            int there = 0;
#pragma unroll
            for (int k = 0; k < 2; k++) {
                const int t0 = j * kKeys + k * SHERRY_KV4_PAGE;
                int page = -1;
                if (t0 < keys) {
                    page = t0 / SHERRY_KV4_PAGE < p.c.width ? __ldg(p.c.table + (long long)w.b * p.c.table_stride + t0 / SHERRY_KV4_PAGE) : -1;
                    if (page < 0 || page >= p.c.pages) {
                        page = -1;
                        if (th == 0) atomicCAS(p.err, 0u, (unsigned int)SHERRY_ERR_INDEX);
                    }
                }
                sm[k] = 0;
#pragma unroll
                for (int e = 0; e < D / 32; e++) u[k][e] = make_uint4(0, 0, 0, 0);
                if (page >= 0) {
                    there |= 1 << k;
                    const uint8_t *blk = kv4_block<D>(p.c, page, h, 0);
                    const uint4 *src = reinterpret_cast<const uint4 *>(blk + th * Kv4<D>::kRow);
#pragma unroll
                    for (int e = 0; e < D / 32; e++) u[k][e] = __ldg(src + e);
                    sm[k] = __ldg(reinterpret_cast<const uint32_t *>(blk + Kv4<D>::kCodes) + th);
                }
            }
            // The slot is free: k_empty of step j - 3 was waited for, and its products were issued after
            // the softmax of step j - 4 was done.
            float *sc = scales + slot * 4 * kKeys;
#pragma unroll
            for (int k = 0; k < 2; k++) {
                const float st = kv4_step(sm[k]);
                sc[64 * k + th] = st * p.scale2;
                sc[kKeys + 64 * k + th] = (kv4_low(sm[k]) + 8.0f * st) * p.scale2;
            }
            if (th == 0) bar->there[slot] = there;
            mbar_arrive(&bar->sc_full[slot]);
            if (!__all_sync(0xFFFFFFFFu, mbar_wait(&bar->k_empty[s], ((j >> 1) & 1) ^ 1, abort, p.err, limit))) break;
#pragma unroll
            for (int k = 0; k < 2; k++) {
                const int t = 64 * k + th;
                uint8_t *dst = sk + s * T::kOp + t * 128;
#pragma unroll
                for (int e = 0; e < D / 32; e++) {
                    const uint32_t x[4] = {u[k][e].x, u[k][e].y, u[k][e].z, u[k][e].w};
#pragma unroll
                    for (int i = 0; i < 4; i++) {
                        const int c = 4 * e + i;  // 8-element chunk of the row
                        *reinterpret_cast<uint4 *>(dst + (c / 8) * (kKeys * 128) + (((c & 7) ^ (t & 7)) << 4)) =
                            make_uint4(code_pair8(x[i]), code_pair8(x[i] >> 4), code_pair8(x[i] >> 8), code_pair8(x[i] >> 12));
                    }
                }
            }
            fence_proxy_async_smem();
            mbar_arrive(&bar->k_full[s]);
        }
    } else if (warp < 12) {
        // ---------------- values: eight tokens of D / 32 words per thread, transposed ----------------
        const int th = threadIdx.x - 320;           // 0 .. 63
        const int grp = (th & 7) + 8 * (th >> 5);   // tokens 8 grp .. 8 grp + 7 of the step
        const int qd = (th >> 3) & 3;               // words qd D / 32 ...
        constexpr int NW = D / 32;
        for (int j = 0; j < steps; j++) {
            const int slot = j % kScaleSlots, s = j & 1;
            uint32_t x[8][NW];
            uint32_t sm[2] = {0, 0};
#pragma unroll
            for (int t = 0; t < 8; t++)
#pragma unroll
                for (int e = 0; e < NW; e++) x[t][e] = 0;
#pragma unroll
            for (int k = 0; k < 2; k++) {
                const int t0 = j * kKeys + k * SHERRY_KV4_PAGE;
                if (t0 >= keys) continue;
                const int page = t0 / SHERRY_KV4_PAGE < p.c.width ? __ldg(p.c.table + (long long)w.b * p.c.table_stride + t0 / SHERRY_KV4_PAGE) : -1;
                if (page < 0 || page >= p.c.pages) continue;
                const uint8_t *blk = kv4_block<D>(p.c, page, h, 1);
                sm[k] = __ldg(reinterpret_cast<const uint32_t *>(blk + Kv4<D>::kCodes) + th);
                if (grp / 8 == k) {
                    const uint8_t *src = blk + (grp & 7) * 8 * Kv4<D>::kRow + qd * NW * 4;
#pragma unroll
                    for (int t = 0; t < 8; t++) {
                        if (NW == 4) {
                            const uint4 v = __ldg(reinterpret_cast<const uint4 *>(src + t * Kv4<D>::kRow));
                            x[t][0] = v.x, x[t][1] = v.y, x[t][NW - 2] = v.z, x[t][NW - 1] = v.w;
                        } else {
                            const uint2 v = __ldg(reinterpret_cast<const uint2 *>(src + t * Kv4<D>::kRow));
                            x[t][0] = v.x, x[t][1] = v.y;
                        }
                    }
                }
            }
            // free as the keys' part is: v_empty of step j - 3 was waited for
            float *sc = scales + slot * 4 * kKeys + 2 * kKeys;
#pragma unroll
            for (int k = 0; k < 2; k++) {
                const float st = kv4_step(sm[k]);
                sc[64 * k + th] = st;
                sc[kKeys + 64 * k + th] = kv4_low(sm[k]) + 8.0f * st;
            }
            mbar_arrive(&bar->sc_full[slot]);
            if (!__all_sync(0xFFFFFFFFu, mbar_wait(&bar->v_empty[s], ((j >> 1) & 1) ^ 1, abort, p.err, limit))) break;
            uint8_t *dst = sv + s * T::kOp + (grp / 8) * (D * 128);
#pragma unroll
            for (int e = 0; e < NW; e++) {
                const int d0 = 8 * (qd * NW + e);
                uint32_t lo[4], hi[4];
#pragma unroll
                for (int t = 0; t < 4; t++) {
                    lo[t] = prmt(x[2 * t][e], x[2 * t + 1][e], 0x5410);
                    hi[t] = prmt(x[2 * t][e], x[2 * t + 1][e], 0x7632);
                }
#pragma unroll
                for (int i = 0; i < 8; i++) {
                    const uint32_t *y = i < 4 ? lo : hi;
                    const int d = d0 + i;
                    *reinterpret_cast<uint4 *>(dst + d * 128 + (((grp & 7) ^ (d & 7)) << 4)) =
                        make_uint4(code_pair8(y[0] >> (4 * (i & 3))), code_pair8(y[1] >> (4 * (i & 3))),
                                   code_pair8(y[2] >> (4 * (i & 3))), code_pair8(y[3] >> (4 * (i & 3))));
                }
            }
            fence_proxy_async_smem();
            mbar_arrive(&bar->v_full[s]);
        }
    } else if (lane == 0 && steps > 0) {
        // ---------------- products ----------------
        bool ok = mbar_wait(&bar->q_full, 0, abort, p.err, limit);
        bool issued = false;
        const uint32_t q_addr = smem_u32(sq), k_addr = smem_u32(sk), v_addr = smem_u32(sv);
        auto scores = [&](int i, int s) {  // S_i = Q_i K^T
            tc_fence_after();
#pragma unroll
            for (int k = 0; k < D / 16; k++) {
                const uint32_t off = (k / 4) * (128 * 128) + (k & 3) * 32;
                umma_f16(tmem + i * kKeys, smem_desc_sw128(q_addr + i * T::kQ + off),
                         smem_desc_sw128(k_addr + s * T::kOp + off), kIdescBf16<kKeys>, k != 0);
            }
            issued = true;
            umma_commit(&bar->s_full[i]);
        };
        if (ok) ok = mbar_wait(&bar->k_full[0], 0, abort, p.err, limit);
        if (ok) {
            scores(0, 0);
            scores(1, 0);
            umma_commit(&bar->k_empty[0]);
        }
        for (int j = 0; ok && j < steps; j++) {
            const int s = j & 1, ph = (j >> 1) & 1;
            ok = mbar_wait(&bar->v_full[s], ph, abort, p.err, limit);
            for (int i = 0; ok && i < 2; i++) {
                ok = mbar_wait(&bar->p_full[i], j & 1, abort, p.err, limit);
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int k = 0; k < kKeys / 16; k++)
                    umma_f16_tmem_a(tmem + 2 * kKeys + i * D, tmem + i * kKeys + 8 * k,
                                    smem_desc_sw128(v_addr + s * T::kOp + (k / 4) * (D * 128) + (k & 3) * 32), kIdescBf16<D>,
                                    j != 0 || k != 0);
                if (j + 1 < steps) {
                    if (i == 0) {
                        ok = mbar_wait(&bar->k_full[s ^ 1], ((j + 1) >> 1) & 1, abort, p.err, limit);
                        if (!ok) break;
                    }
                    scores(i, s ^ 1);
                } else {
                    umma_commit(&bar->o_full[i]);
                }
            }
            if (ok) {
                umma_commit(&bar->v_empty[s]);
                if (j + 1 < steps) umma_commit(&bar->k_empty[s ^ 1]);
            }
        }
        // every issued product is done before tensor and shared memory are released
        if (issued) {
            umma_commit(&bar->drain);
            volatile int no_abort = 0;
            mbar_wait(&bar->drain, 0, &no_abort, p.err, kDrainLimit);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 12) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

template <int D>
sherry_status tile_launch(const AttnParams &p, cudaStream_t stream) {
    static OccupancyCache cache;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) dev = 0;
    const int i = dev & 63;
    const unsigned long long id = context_id();
    if (cache.bps[i].load(std::memory_order_acquire) == 0 || id == 0 || cache.ctx[i].load(std::memory_order_acquire) != id) {
        const cudaError_t e = cudaFuncSetAttribute(attn_tile_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Tile<D>::kSmem);
        if (e != cudaSuccess) {
            set_last_error("sherry_attn_kv4 (attributes)", e);
            return SHERRY_ERR_CUDA;
        }
        cache.bps[i].store(1, std::memory_order_release);
        cache.ctx[i].store(id, std::memory_order_release);
    }
    // at most this many row tiles: whole ones, and one more for each sequence that has more than
    // few_rows rows
    const long long rows = (long long)p.c.T * p.g;
    const long long seqs = p.few_rows > 0 ? std::min<long long>(p.c.B, rows / p.few_rows + 1) : p.c.B;
    const long long ctas = (rows / kRowsCta + seqs) * p.c.H;
    if (ctas > 0x7FFFFFFF || rows > 0x7FFFFFFF) return SHERRY_ERR_UNSUPPORTED;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(kTileThreads);
    cfg.dynamicSmemBytes = Tile<D>::kSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaLaunchKernelEx(&cfg, attn_tile_kernel<D>, p);
    return launch_status("sherry_attn_kv4 (tiles)");
}

}  // namespace

sherry_status attn_tile_launch(const AttnParams &p, int D, cudaStream_t stream) {
    return D == 64 ? tile_launch<64>(p, stream) : tile_launch<128>(p, stream);
}

}  // namespace sherry
