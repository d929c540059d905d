// attn.cu -- causal attention over the 4-bit key/value cache: the calls, and the kernels for
// sequences with few new tokens (decode steps, drafts).
#include <algorithm>

#include "attn.cuh"

namespace sherry {
namespace {

// ---------------------------------------------------------------------------
// Few rows: mma.sync on fragments decoded in registers
// ---------------------------------------------------------------------------
// The bytes of the cache are the bound: 2 (D / 2 + 4) per token and head.  A unit of work is one
// page for one key/value head and up to 8 NT rows (query heads that share it, times new tokens).
// All units of the batch, in the order (sequence, head, row tile, page), are cut into equal runs,
// one per CTA, so that long and short sequences load every SM alike; a run's pieces that are not
// whole go to the workspace and a second kernel joins them in the order of the CTAs (no atomics:
// results do not depend on timing).  One warp copies pages into a ring (a page's keys and values
// are one contiguous block: one bulk copy); four warps take 16 of a page's tokens each.  The
// product is S^T = K q^T with 16 tokens by 8 rows: the 8-wide side carries the few rows, so
// 4 query heads per key/value head fill half of the instruction instead of a quarter.  The 128 of
// the codes' bf16 is taken out of the first product by starting it at -128 sum(q), and out of the
// second by -136 times the sum of the rounded p s.
constexpr int kFewWarps = 4;
constexpr int kFewThreads = 32 * (kFewWarps + 1);
constexpr int kFewCtasMax = 1024;  // bounds the workspace
constexpr int kFewRows = 32;       // rows of a sequence up to which this kernel takes it

template <int D, int NT>
struct Few {
    static constexpr int kRows = 8 * NT;
    static constexpr int kStage = 2 * Kv4<D>::kBlock;
    static constexpr int kStages = D == 64 ? 8 : 5;
    static constexpr int kRing = kStages * kStage;
    static constexpr int kJoin = kRows * D * 4;   // [rows][D] sums of the four warps
    static constexpr size_t kSmem = kRing + kJoin + 256 * NT + 256;
};

// Work of a batch: sequence b has `tiles` row tiles of `pages` pages for each head.
struct SeqWork {
    int first, rows, pages, tiles, len;
};

template <int ROWS>
__device__ __forceinline__ SeqWork seq_work(const AttnParams &p, int b) {
    const Kv4View &c = p.c;
    const int g = p.g;
    SeqWork s;
    int n;
    kv4_rows(c, b, s.first, n);
    s.rows = n;
    s.len = max(__ldg(c.lens + b), 0);
    const long long rows = (long long)n * g;
    s.tiles = rows > p.few_rows ? 0 : (int)((rows + ROWS - 1) / ROWS);
    // an empty sequence has one page without keys: its rows are written as zeros
    s.pages = max((min(s.len, c.width * SHERRY_KV4_PAGE) + SHERRY_KV4_PAGE - 1) / SHERRY_KV4_PAGE, 1);
    return s;
}

template <int ROWS>
__device__ __forceinline__ long long seq_units(const AttnParams &p, int b) {
    if (b >= p.c.B) return 0;
    const SeqWork s = seq_work<ROWS>(p, b);
    return (long long)p.c.H * s.tiles * s.pages;
}

// Sum of the batch's units (every lane of a full warp).
template <int ROWS>
__device__ long long all_units(const AttnParams &p) {
    long long sum = 0;
    for (int b = threadIdx.x & 31; b < p.c.B; b += 32) sum += seq_units<ROWS>(p, b);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    return sum;
}

// The sequence that holds unit w (w below all_units) and the units before it.
template <int ROWS>
__device__ void find_unit(const AttnParams &p, long long w, int &b, long long &before) {
    const int lane = threadIdx.x & 31;
    long long base = 0;
    for (int b0 = 0; b0 < p.c.B; b0 += 32) {
        const long long mine = seq_units<ROWS>(p, b0 + lane);
        long long sum = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long v = __shfl_up_sync(0xFFFFFFFFu, sum, o);
            if (lane >= o) sum += v;
        }
        const unsigned hit = __ballot_sync(0xFFFFFFFFu, base + sum > w);
        if (hit) {
            const int l = __ffs(hit) - 1;
            b = b0 + l;
            before = base + __shfl_sync(0xFFFFFFFFu, sum - mine, l);
            return;
        }
        base += __shfl_sync(0xFFFFFFFFu, sum, 31);
    }
    b = p.c.B;
    before = base;
}

// CTA i of n takes units [i W / n, (i + 1) W / n); unit w lies with CTA ((w + 1) n - 1) / W.
__device__ __forceinline__ long long run_start(long long W, int i, int n) { return W * i / n; }
__device__ __forceinline__ int run_of(long long W, long long w, int n) { return (int)(((w + 1) * n - 1) / W); }

// A CTA's walk over its run, one piece (part of a (sequence, head, row tile)) at a time.
template <int ROWS>
struct Walk {
    long long w, end, before;  // position, end of the run, units before sequence b
    int b;
    SeqWork s;
    int h, tile, page0, page1;

    __device__ __forceinline__ void start(const AttnParams &p, long long from, long long to) {
        w = from;
        end = to;
        find_unit<ROWS>(p, w, b, before);
        if (b < p.c.B) s = seq_work<ROWS>(p, b);
    }
    // The next piece: pages [page0, page1) of (b, h, tile); false at the end.
    __device__ __forceinline__ bool next(const AttnParams &p) {
        if (w >= end) return false;
        while (w - before >= (long long)p.c.H * s.tiles * s.pages) {
            before += (long long)p.c.H * s.tiles * s.pages;
            if (++b >= p.c.B) return false;
            s = seq_work<ROWS>(p, b);
        }
        const long long u = w - before;
        const int unit = (int)(u / s.pages);
        page0 = (int)(u - (long long)unit * s.pages);
        page1 = (int)min((long long)s.pages, page0 + (end - w));
        h = unit / s.tiles;
        tile = unit - h * s.tiles;
        w += page1 - page0;
        return true;
    }
};

__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9},"
        " {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(v));
    return d;
}

// Barrier of the consumer warps alone.
__device__ __forceinline__ void few_sync() { asm volatile("bar.sync 1, %0;" ::"n"(32 * kFewWarps) : "memory"); }

template <int D, int NT>
__global__ void __launch_bounds__(kFewThreads) attn_few_kernel(const __grid_constant__ AttnParams p) {
    using F = Few<D, NT>;
    constexpr int kRows = F::kRows, kS = F::kStages, MT = D / 16, WK = D / 32;
    extern __shared__ __align__(128) uint8_t smem[];
    float *join = reinterpret_cast<float *>(smem + F::kRing);
    float *stat = join + kRows * D;                       // [4 warps][rows] maxima, then [rows] sums
    uint64_t *full = reinterpret_cast<uint64_t *>(stat + 8 * kRows), *empty = full + kS;
    int *there = reinterpret_cast<int *>(empty + kS);     // per stage: the page exists
    int *abort = there + kS;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kS; s++) {
            mbar_init(full + s, 1);
            mbar_init(empty + s, kFewWarps);
        }
        *abort = 0;
        fence_mbar_init();
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    __syncthreads();
    asm volatile("griddepcontrol.wait;" ::: "memory");  // lengths and cache come from the kernels before
    const long long W = all_units<kRows>(p);
    const int n = (int)min((long long)p.grid, W);
    if ((int)blockIdx.x >= n) return;
    const long long from = run_start(W, blockIdx.x, n), to = run_start(W, blockIdx.x + 1, n);
    Walk<kRows> walk;
    walk.start(p, from, to);

    if (warp == kFewWarps) {
        // ---------------- copies ----------------
        if (lane == 0) {
            uint32_t it = 0;
            while (walk.next(p)) {
                if (walk.s.len > p.c.width * SHERRY_KV4_PAGE) atomicCAS(p.err, 0u, (unsigned int)SHERRY_ERR_INDEX);
                for (int pg = walk.page0; pg < walk.page1; pg++, it++) {
                    const int s = it % kS;
                    // where a wait gives up, the rest of the walk waits no more and copies nothing
                    const bool ok = mbar_wait(empty + s, ((it / kS) & 1) ^ 1, abort, p.err, p.wait_limit) && !*(volatile int *)abort;
                    int page = -1;
                    if (ok && walk.s.len > 0) page = kv4_page(p.c, walk.b, pg * SHERRY_KV4_PAGE, p.err);
                    there[s] = page >= 0;
                    if (page >= 0) {
                        mbar_arrive_expect_tx(full + s, F::kStage);
                        bulk_load(smem_u32(smem + s * F::kStage), kv4_block<D>(p.c, page, walk.h, 0), F::kStage, full + s);
                    } else {
                        mbar_arrive(full + s);
                    }
                }
            }
            // every copy lands before the CTA's shared memory is released
            volatile int no_abort = 0;
            for (uint32_t j = it < (uint32_t)kS ? 0 : it - kS; j < it; j++)
                mbar_wait(full + j % kS, (j / kS) & 1, &no_abort, p.err, 1000000000LL);
        }
        return;
    }

    // ---------------- products ----------------
    const int r = lane >> 2, c = lane & 3;
    // Row m of a 16-token tile is token tok(m); chosen so that neither the keys' loads (a token per
    // four lanes) nor the values' (four tokens per lane) meet in a bank.
    const int tok_r = r ^ (r >> 2 & 1);                       // rows r and r + 8 (+ 8)
    const int tok_v0 = (2 * c) ^ (c >> 1 & 1), tok_v1 = (2 * c + 1) ^ (c >> 1 & 1);
    uint32_t it = 0;
    while (walk.next(p)) {
        const int nrow = walk.s.rows * p.g, row0 = walk.tile * kRows;
        const int pos0 = walk.s.len - walk.s.rows;            // position of the first new token
        // q: lane (r, c) holds elements [c D / 4, (c + 1) D / 4) of row r of each row group
        uint32_t qf[NT][MT][2];
        float qsum[NT][2];                                    // of rows 2 c, 2 c + 1
        int last[NT][2];                                      // last token those rows see
        int last_min = 0x7FFFFFFF, last_max = -1;
#pragma unroll
        for (int t = 0; t < NT; t++) {
            const int row = row0 + 8 * t + r;
            float sum = 0.0f;
            const uint16_t *src = nullptr;
            if (row < nrow)
                src = p.q + (long long)(walk.s.first + row / p.g) * p.q_stride +
                      (long long)(walk.h * p.g + row % p.g) * D + c * (D / 4);
#pragma unroll
            for (int w = 0; w < WK; w++) {
                uint4 u = make_uint4(0, 0, 0, 0);
                if (src) u = *reinterpret_cast<const uint4 *>(src + 8 * w);
                const uint32_t e[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                for (int i = 0; i < 4; i++)
                    sum += __uint_as_float(e[i] << 16) + __uint_as_float(e[i] & 0xFFFF0000u);
                // a code word's pairs are elements (i, i + 4)
                qf[t][2 * w][0] = prmt(u.x, u.z, 0x5410);
                qf[t][2 * w][1] = prmt(u.x, u.z, 0x7632);
                qf[t][2 * w + 1][0] = prmt(u.y, u.w, 0x5410);
                qf[t][2 * w + 1][1] = prmt(u.y, u.w, 0x7632);
            }
            sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 1);
            sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 2);
#pragma unroll
            for (int j = 0; j < 2; j++) {
                qsum[t][j] = __shfl_sync(0xFFFFFFFFu, sum, (2 * c + j) * 4);
                const int rw = row0 + 8 * t + 2 * c + j;
                last[t][j] = rw < nrow ? pos0 + rw / p.g : -1;
            }
        }
        {
            const int lo_row = row0, hi_row = min(row0 + kRows, nrow) - 1;
            last_min = hi_row == row0 + kRows - 1 ? pos0 + lo_row / p.g : -1;  // rows past the end see nothing
            last_max = pos0 + hi_row / p.g;
        }
        float o[NT][MT][4];
        float m[NT][2], l[NT][2], corr[NT][2];
#pragma unroll
        for (int t = 0; t < NT; t++) {
#pragma unroll
            for (int i = 0; i < MT; i++)
#pragma unroll
                for (int j = 0; j < 4; j++) o[t][i][j] = 0.0f;
#pragma unroll
            for (int j = 0; j < 2; j++) m[t][j] = -INFINITY, l[t][j] = 0.0f, corr[t][j] = 0.0f;
        }
        for (int pg = walk.page0; pg < walk.page1; pg++, it++) {
            const int s = it % kS;
            const bool ok = __all_sync(0xFFFFFFFFu, mbar_wait(full + s, (it / kS) & 1, abort, p.err, p.wait_limit));
            const int t0 = pg * SHERRY_KV4_PAGE + 16 * warp;  // first token of this warp's tile
            if (ok && there[s] && t0 <= last_max) {
                const uint8_t *kb = smem + s * F::kStage, *vb = kb + Kv4<D>::kBlock;
                const int ta = 16 * warp + tok_r;             // rows r, r + 8 of the tile
                uint32_t kw[2][WK];
#pragma unroll
                for (int i = 0; i < 2; i++) {
                    const uint8_t *src = kb + (ta + 8 * i) * Kv4<D>::kRow + c * (D / 8);
                    if (D == 64) {
                        const uint2 u = *reinterpret_cast<const uint2 *>(src);
                        kw[i][0] = u.x, kw[i][1] = u.y;
                    } else {
                        const uint4 u = *reinterpret_cast<const uint4 *>(src);
                        kw[i][0] = u.x, kw[i][1] = u.y;
                        kw[i][WK - 2] = u.z, kw[i][WK - 1] = u.w;
                    }
                }
                const uint32_t *ksm = reinterpret_cast<const uint32_t *>(kb + Kv4<D>::kCodes) + ta;
                const uint32_t *vsm = reinterpret_cast<const uint32_t *>(vb + Kv4<D>::kCodes) + ta;
                const uint32_t kp[2] = {ksm[0], ksm[8]}, vp[2] = {vsm[0], vsm[8]};
                float x[NT][4];
#pragma unroll
                for (int t = 0; t < NT; t++) {
                    x[t][0] = x[t][2] = -128.0f * qsum[t][0];
                    x[t][1] = x[t][3] = -128.0f * qsum[t][1];
                }
#pragma unroll
                for (int w = 0; w < WK; w++) {
                    uint32_t a[4];
#pragma unroll
                    for (int k = 0; k < 2; k++) {
                        a[0] = code_pair(kw[0][w] >> (8 * k));
                        a[1] = code_pair(kw[1][w] >> (8 * k));
                        a[2] = code_pair(kw[0][w] >> (8 * k + 4));
                        a[3] = code_pair(kw[1][w] >> (8 * k + 4));
#pragma unroll
                        for (int t = 0; t < NT; t++) mma_bf16(x[t], a, qf[t][2 * w + k][0], qf[t][2 * w + k][1]);
                    }
                }
                const bool whole = t0 + 15 <= last_min;
                bool grow = false;
#pragma unroll
                for (int t = 0; t < NT; t++)
#pragma unroll
                    for (int i = 0; i < 2; i++) {
                        const float sk = kv4_step(kp[i]) * p.scale2, mk = kv4_low(kp[i]) * p.scale2;
#pragma unroll
                        for (int j = 0; j < 2; j++) {
                            float v = sk * x[t][2 * i + j] + mk * qsum[t][j];
                            if (!whole && t0 + tok_r + 8 * i > last[t][j]) v = -INFINITY;
                            x[t][2 * i + j] = v;
                            grow |= v > m[t][j] + 8.0f;
                        }
                    }
                // The reference of the exponentials follows the maximum only when a score exceeds it by
                // 2^8: probabilities stay below 2^8, and most tiles skip the shuffles and the rescaling.
                if (__any_sync(0xFFFFFFFFu, grow)) {
#pragma unroll
                    for (int t = 0; t < NT; t++)
#pragma unroll
                        for (int j = 0; j < 2; j++) {
                            float mx = fmaxf(m[t][j], fmaxf(x[t][j], x[t][2 + j]));
                            mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 4));
                            mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 8));
                            mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 16));
                            const float f = m[t][j] == -INFINITY ? 0.0f : exp2_fast(m[t][j] - mx);
                            m[t][j] = mx;
                            l[t][j] *= f;
                            corr[t][j] *= f;
#pragma unroll
                            for (int i = 0; i < MT; i++) {
                                o[t][i][j] *= f;
                                o[t][i][2 + j] *= f;
                            }
                        }
                }
                uint32_t pb[NT][2];
#pragma unroll
                for (int t = 0; t < NT; t++)
#pragma unroll
                    for (int i = 0; i < 2; i++) {
                        const float sv = kv4_step(vp[i]), cv = kv4_low(vp[i]) + 8.0f * sv;
                        float ps[2];
#pragma unroll
                        for (int j = 0; j < 2; j++) {
                            const float ref = m[t][j] == -INFINITY ? 0.0f : m[t][j];
                            const float pr = exp2_fast(x[t][2 * i + j] - ref);
                            const bool seen = whole || t0 + tok_r + 8 * i <= last[t][j];
                            l[t][j] += pr;
                            // a token that the row does not see may hold anything, NaN too
                            ps[j] = seen ? pr * sv : 0.0f;
                            corr[t][j] += seen ? pr * cv : 0.0f;
                        }
                        const uint32_t u = pack_bf16(ps[0], ps[1]);
                        corr[t][0] -= 136.0f * __uint_as_float(u << 16);
                        corr[t][1] -= 136.0f * __uint_as_float(u & 0xFFFF0000u);
                        pb[t][i] = transpose8x8(u);
                    }
                // values: lane (r, c) holds word(s) r of four tokens; a pair of tokens per register
#pragma unroll
                for (int w = 0; w < D / 64; w++) {
                    const uint8_t *src = vb + 16 * warp * Kv4<D>::kRow + (r * (D / 64) + w) * 4;
                    const uint32_t w0 = *reinterpret_cast<const uint32_t *>(src + tok_v0 * Kv4<D>::kRow);
                    const uint32_t w1 = *reinterpret_cast<const uint32_t *>(src + tok_v1 * Kv4<D>::kRow);
                    const uint32_t w2 = *reinterpret_cast<const uint32_t *>(src + (tok_v0 + 8) * Kv4<D>::kRow);
                    const uint32_t w3 = *reinterpret_cast<const uint32_t *>(src + (tok_v1 + 8) * Kv4<D>::kRow);
                    const uint32_t al = prmt(w0, w1, 0x5410), ah = prmt(w0, w1, 0x7632);
                    const uint32_t bl = prmt(w2, w3, 0x5410), bh = prmt(w2, w3, 0x7632);
#pragma unroll
                    for (int i = 0; i < 4; i++) {
                        const uint32_t a[4] = {code_pair(al >> (4 * i)), code_pair(ah >> (4 * i)),
                                               code_pair(bl >> (4 * i)), code_pair(bh >> (4 * i))};
#pragma unroll
                        for (int t = 0; t < NT; t++) mma_bf16(o[t][4 * w + i], a, pb[t][0], pb[t][1]);
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(empty + s);
        }

        // ---------------- the four warps' sums together ----------------
#pragma unroll
        for (int t = 0; t < NT; t++)
#pragma unroll
            for (int j = 0; j < 2; j++) {
#pragma unroll
                for (int k = 4; k < 32; k <<= 1) {
                    l[t][j] += __shfl_xor_sync(0xFFFFFFFFu, l[t][j], k);
                    corr[t][j] += __shfl_xor_sync(0xFFFFFFFFu, corr[t][j], k);
                }
                if (r == 0) stat[warp * kRows + 8 * t + 2 * c + j] = m[t][j];
            }
        few_sync();
        float mx[NT][2];
#pragma unroll
        for (int t = 0; t < NT; t++)
#pragma unroll
            for (int j = 0; j < 2; j++) {
                const int row = 8 * t + 2 * c + j;
                float v = stat[row];
#pragma unroll
                for (int w = 1; w < kFewWarps; w++) v = fmaxf(v, stat[w * kRows + row]);
                mx[t][j] = v;
                const float f = m[t][j] == -INFINITY ? 0.0f : exp2_fast(m[t][j] - v);
                // a NaN score leaves m at -inf but reaches l: keep it
                l[t][j] = m[t][j] == -INFINITY && l[t][j] == 0.0f ? 0.0f : l[t][j] * (m[t][j] == -INFINITY ? 1.0f : f);
                corr[t][j] *= f;
#pragma unroll
                for (int i = 0; i < MT; i++) {
                    o[t][i][j] = (o[t][i][j] * f) + corr[t][j];
                    o[t][i][2 + j] = (o[t][i][2 + j] * f) + corr[t][j];
                }
            }
        float *sums = stat + 4 * kRows;
        for (int w = 0; w < kFewWarps; w++) {
            if (w == warp) {
#pragma unroll
                for (int t = 0; t < NT; t++)
#pragma unroll
                    for (int j = 0; j < 2; j++) {
                        const int row = 8 * t + 2 * c + j;
                        float *dst = join + row * D + r * (D / 8);
#pragma unroll
                        for (int i = 0; i < MT; i += 4)
#pragma unroll
                            for (int k = 0; k < 2; k++) {
                                // elements 8 word + 4 k + 0 .. 3
                                float4 v = make_float4(o[t][i][2 * k + j], o[t][i + 1][2 * k + j],
                                                       o[t][i + 2][2 * k + j], o[t][i + 3][2 * k + j]);
                                float4 *d4 = reinterpret_cast<float4 *>(dst + 2 * i + 4 * k);
                                if (w > 0) {
                                    const float4 u = *d4;
                                    v = make_float4(u.x + v.x, u.y + v.y, u.z + v.z, u.w + v.w);
                                }
                                *d4 = v;
                            }
                        if (r == 0) sums[row] = w == 0 ? l[t][j] : sums[row] + l[t][j];
                    }
            }
            few_sync();
        }
        // whole: the result; else this run's part to the workspace
        const bool all = walk.page0 == 0 && walk.page1 == walk.s.pages;
        const int tid = threadIdx.x;
        if (all) {
            for (int i = tid; i < kRows * (D / 8); i += 32 * kFewWarps) {
                const int row = i / (D / 8), d = (i % (D / 8)) * 8, rw = row0 + row;
                if (rw >= nrow) continue;
                const float sum = sums[row];
                const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
                const float4 a = *reinterpret_cast<const float4 *>(join + row * D + d);
                const float4 b = *reinterpret_cast<const float4 *>(join + row * D + d + 4);
                uint16_t *dst = p.out + (long long)(walk.s.first + rw / p.g) * p.out_stride +
                                (long long)(walk.h * p.g + rw % p.g) * D + d;
                *reinterpret_cast<uint4 *>(dst) =
                    make_uint4(pack_bf16(a.x * inv, a.y * inv), pack_bf16(a.z * inv, a.w * inv),
                               pack_bf16(b.x * inv, b.y * inv), pack_bf16(b.z * inv, b.w * inv));
            }
        } else {
            // the piece that began before this run takes slot 0, one that begins inside it slot 1
            const long long begin = walk.w - walk.page1;      // the unit's first page
            const long long slot = 2LL * blockIdx.x + (begin > from ? 1 : 0);
            float4 *dst = reinterpret_cast<float4 *>(p.ws + slot * kRows * D);
            for (int i = tid; i < kRows * D / 4; i += 32 * kFewWarps) dst[i] = reinterpret_cast<const float4 *>(join)[i];
            if (r == 0 && warp == 0) {
                float2 *ml = reinterpret_cast<float2 *>(p.ws + 2LL * p.grid * kRows * D) + slot * kRows;
#pragma unroll
                for (int t = 0; t < NT; t++)
#pragma unroll
                    for (int j = 0; j < 2; j++) {
                        const int row = 8 * t + 2 * c + j;
                        ml[row] = make_float2(mx[t][j], sums[row]);
                    }
            }
        }
        few_sync();  // join and stat are free for the next piece
    }
}

// Joins the parts of the row tiles that the runs cut: CTA i takes the one that begins in run i and
// goes on in the next, one warp per row, its parts in the order of the CTAs.
template <int D, int NT>
__global__ void __launch_bounds__(256 * NT, 2) attn_join_kernel(const __grid_constant__ AttnParams p) {
    constexpr int kRows = 8 * NT, E = D / 32;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x & 31, row = threadIdx.x >> 5;
    const long long W = all_units<kRows>(p);
    const int n = (int)min((long long)p.grid, W), i0 = blockIdx.x;
    if (i0 >= n - 1) return;
    const long long from = run_start(W, i0, n), to = run_start(W, i0 + 1, n);
    int b;
    long long before;
    find_unit<kRows>(p, to - 1, b, before);
    if (b >= p.c.B) return;
    const SeqWork s = seq_work<kRows>(p, b);
    const int unit = (int)((to - 1 - before) / s.pages);
    const long long w0 = before + (long long)unit * s.pages, w1 = w0 + s.pages;
    if (w1 <= to || w0 < from) return;  // not cut here, or begun by an earlier CTA
    const int h = unit / s.tiles, rw = (unit - h * s.tiles) * kRows + row;
    if (rw >= s.rows * p.g) return;
    const int i1 = run_of(W, w1 - 1, n);
    const float2 *ml = reinterpret_cast<const float2 *>(p.ws + 2LL * p.grid * kRows * D);
    const int first_slot = w0 > from ? 1 : 0;
    float m = -INFINITY;
    for (int i = i0 + lane; i <= i1; i += 32) m = fmaxf(m, ml[(2LL * i + (i == i0 ? first_slot : 0)) * kRows + row].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    float l = 0.0f, acc[E];
#pragma unroll
    for (int e = 0; e < E; e++) acc[e] = 0.0f;
    for (int ib = i0; ib <= i1; ib += 32) {
        const int i = ib + lane;
        float f = 0.0f;
        if (i <= i1) {
            const float2 v = ml[(2LL * i + (i == i0 ? first_slot : 0)) * kRows + row];
            // a part without keys has sum 0; a NaN among its scores shows in the sum
            f = v.x == -INFINITY ? (v.y == 0.0f ? 0.0f : v.y) : exp2_fast(v.x - m);
            l += v.y * f;
        }
        const int k1 = min(32, i1 - ib + 1);
#pragma unroll 8
        for (int k = 0; k < k1; k++) {
            const float fk = __shfl_sync(0xFFFFFFFFu, f, k);
            const long long slot = 2LL * (ib + k) + (ib + k == i0 ? first_slot : 0);
            const float *src = p.ws + (slot * kRows + row) * D + lane * E;
            if (E == 2) {
                const float2 v = *reinterpret_cast<const float2 *>(src);
                acc[0] += fk * v.x, acc[1] += fk * v.y;
            } else {
                const float4 v = *reinterpret_cast<const float4 *>(src);
                acc[0] += fk * v.x, acc[1] += fk * v.y, acc[E - 2] += fk * v.z, acc[E - 1] += fk * v.w;
            }
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, o);
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    uint16_t *dst = p.out + (long long)(s.first + rw / p.g) * p.out_stride + (long long)(h * p.g + rw % p.g) * D + lane * E;
#pragma unroll
    for (int e = 0; e < E; e += 2) *reinterpret_cast<uint32_t *>(dst + e) = pack_bf16(acc[e] * inv, acc[e + 1] * inv);
}

// Blocks per SM of the kernel, with its shared-memory attribute set, once per device and context.
template <typename K>
int few_blocks_per_sm(K kernel, size_t smem, OccupancyCache &cache) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) dev = 0;
    const int i = dev & 63;
    const unsigned long long id = context_id();
    const int have = cache.bps[i].load(std::memory_order_acquire);
    if (have > 0 && id != 0 && cache.ctx[i].load(std::memory_order_acquire) == id) return have;
    int n = 0;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess ||
        cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, kFewThreads, smem) != cudaSuccess || n < 1)
        n = 1;
    cache.bps[i].store(n, std::memory_order_release);
    cache.ctx[i].store(id, std::memory_order_release);
    return n;
}

template <typename K>
void launch_after(K kernel, dim3 grid, int threads, size_t smem, cudaStream_t stream, const AttnParams &p) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaLaunchKernelEx(&cfg, kernel, p);
}

template <int D, int NT>
sherry_status few_launch(AttnParams p, cudaStream_t stream) {
    using F = Few<D, NT>;
    static OccupancyCache cache;
    const int bps = few_blocks_per_sm(attn_few_kernel<D, NT>, F::kSmem, cache);
    p.grid = std::min(sm_count() * bps, kFewCtasMax);
    launch_after(attn_few_kernel<D, NT>, dim3((unsigned)p.grid), kFewThreads, F::kSmem, stream, p);
    const sherry_status st = launch_status("sherry_attn_kv4");
    // a table of one page cuts nothing
    if (st != SHERRY_OK || p.c.width == 1) return st;
    launch_after(attn_join_kernel<D, NT>, dim3((unsigned)p.grid), 256 * NT, 0, stream, p);
    return launch_status("sherry_attn_kv4 (join)");
}

}  // namespace
}  // namespace sherry

// The parts of the row tiles that the runs of the few-row kernel cut: at most two per CTA, each
// with 16 rows of D sums, a maximum and a total.
extern "C" size_t sherry_attn_kv4_workspace_bytes(int64_t T, int Hq, int D) {
    if (T < 1 || Hq < 1 || (D != 64 && D != 128)) return 0;
    return (size_t)2 * sherry::kFewCtasMax * 16 * (size_t)(D + 2) * 4;
}

extern "C" sherry_status sherry_attn_kv4(const sherry_kv4 *c, const uint16_t *q, int64_t q_stride, uint16_t *out,
                                         int64_t out_stride, int Hq, int64_t max_q, float scale, void *workspace,
                                         size_t workspace_bytes, sherry_stream_t stream) {
    using namespace sherry;
    sherry_status st = kv4_check(c);
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
    p.ws = static_cast<float *>(workspace);
    p.q_stride = q_stride;
    p.out_stride = out_stride;
    p.g = Hq / c->H;
    p.grid = 0;
    p.scale2 = scale * kLog2e;
    p.err = kv4_error_address();
    if (!p.err) return SHERRY_ERR_CUDA;
    const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const int64_t most = (c->cu_q ? (max_q > 0 ? std::min(max_q, c->T) : c->T) : 1) * p.g;  // rows of a sequence
    p.wait_limit = wait_limit();
    p.few_rows = 0x7FFFFFFF;
    if (most > kFewRows) {
        // a batch may hold both kinds; a lone sequence is one or the other
        p.few_rows = c->B == 1 ? -1 : kFewRows;
        st = attn_tile_launch(p, c->D, s);
        if (st != SHERRY_OK || c->B == 1) return st;
    }
    const bool one = most <= 8;
    if (c->D == 64) return one ? few_launch<64, 1>(p, s) : few_launch<64, 2>(p, s);
    return one ? few_launch<128, 1>(p, s) : few_launch<128, 2>(p, s);
}
