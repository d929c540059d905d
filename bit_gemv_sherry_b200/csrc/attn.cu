// attn.cu -- causal attention over the 4-bit key/value cache: the calls, and the kernels for
// sequences with few new tokens (decode steps, drafts).
#include <algorithm>
#include <type_traits>

#include "attn.cuh"
#include "page_ring.h"

namespace sherry {
namespace {

// ---------------------------------------------------------------------------
// Few rows: mma.sync on fragments decoded in registers
// ---------------------------------------------------------------------------
// The bytes of the cache are the bound: 2 (D / 2 + 4) per token and head.  The work is the pages of the
// batch in the order (sequence, head, row tile, page), a row tile being up to 8 NT rows (query heads that
// share a key/value head, times new tokens).  It is cut into equal runs, one per warp, so that long and
// short sequences load the machine alike (and as few runs as that takes: fewer parts to join); row tiles
// that a run does not hold whole go to the workspace and a second kernel joins their parts in the order of
// the runs (no atomics: results do not depend on timing).  Few row tiles of few pages go to a cluster each
// instead, which joins its warps' parts in shared memory.  A warp works alone: it copies its pages into its
// own ring (a page's keys and values are one contiguous block: one bulk copy), and no other warp waits for it.
// The product is S^T = K q^T, 16 tokens by 8 rows: the 8-wide side carries the few rows, so 4 query heads
// per key/value head fill half of the instruction instead of a quarter.
// Decoding is what bounds it next (integer instructions, half of an SM's rate): a code's four bits at the
// bottom of a half word are the fp16 c 2^-24, one up c 2^-20, so a word of eight codes takes a shift and
// four ANDs; the keys' powers of two go into q (fp16, exact after a power of two per row).
// 32 sequences of 32,768 tokens, 8 heads of 128, 4 query heads each (floor 177 us): 209 us in a graph, 5.5
// TB/s, 935 instructions a page; 232 us in calls back to back.  Earlier forms: a page shared by four warps and
// filled by a fifth, 357 us; a warp per page with codes as bf16 128 + c (a shift and an OR more per pair),
// 320 us; selects for unseen tokens on every page and 64-bit divisions in the walk, 234 us; the softmax on
// single floats, 1,090 instructions, 220 us; the first page's references set before its first pass, 217 us.
// Short contexts are latency: two pages 6.1 us as a cluster, 8.9 as runs and a join.
constexpr int kFewWarps = 4;
constexpr int kFewThreads = 32 * kFewWarps;
constexpr int kFewRunsMax = 2560;  // bounds the workspace
constexpr int kFewRows = 32;       // rows of a sequence up to which this kernel takes it
// Starting and ending a row tile costs a warp about as much as this many pages; counted as work where
// there is enough of it.
constexpr int kUnitCost = 1;
constexpr int kJoinPages = 3;

template <int D, int NT>
struct Few {
    static constexpr int kRows = 8 * NT;
    static constexpr int kStage = 2 * Kv4<D>::kBlock;
    static constexpr int kStages = D == 64 ? 3 : 2;
    static constexpr int kTiles = 2;  // 16-token tiles whose scores are held at a time
    static constexpr int kCtas = NT == 1 ? (D == 64 ? 4 : 3) : 2;
    static constexpr size_t kSmem = kFewWarps * (kStages * (kStage + 16) + 128) + 16;
};

// A sequence's part of the work: `tiles` row tiles of `pages` pages for each head.
struct SeqWork {
    int first, rows, pages, tiles, len;
};

template <int ROWS>
__device__ __forceinline__ SeqWork seq_work(const AttnParams &p, int b) {
    SeqWork s;
    int n;
    kv4_rows(p.c, b, s.first, n);
    s.rows = n;
    s.len = max(__ldg(p.c.lens + b), 0);
    const long long rows = (long long)n * p.g;
    s.tiles = rows > p.few_rows ? 0 : (int)((rows + ROWS - 1) / ROWS);
    // an empty sequence has one page without keys: its rows are written as zeros
    s.pages = max((min(s.len, p.c.width * SHERRY_KV4_PAGE) + SHERRY_KV4_PAGE - 1) / SHERRY_KV4_PAGE, 1);
    return s;
}

// The batch's work as this launch divides it.
struct Work {
    long long total;  // work of all row tiles: pages, and `cost` for each row tile
    long long each;   // a run's share: run i takes places [i each, (i + 1) each)
    int cost;
};

// a / b for a >= 0, b > 0, mostly small.
__device__ __forceinline__ long long quotient(long long a, long long b) {
    return ((a | b) >> 32) == 0 ? (long long)((uint32_t)a / (uint32_t)b) : a / b;
}

template <int ROWS>
__device__ Work all_work(const AttnParams &p) {
    long long pages = 0, units = 0;
    for (int b = threadIdx.x & 31; b < p.c.B; b += 32) {
        const SeqWork s = seq_work<ROWS>(p, b);
        units += (long long)p.c.H * s.tiles;
        pages += (long long)p.c.H * s.tiles * s.pages;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        pages += __shfl_xor_sync(0xFFFFFFFFu, pages, o);
        units += __shfl_xor_sync(0xFFFFFFFFu, units, o);
    }
    Work w;
    w.cost = pages >= 4LL * p.grid ? kUnitCost : 0;
    w.total = pages + units * w.cost;
    w.each = quotient(w.total + p.grid - 1, p.grid);
    return w;
}

// The sequence that holds place x of the work (x below the total), and the work before it; or, with
// UNITS, the sequence that holds row tile x, and the row tiles before it.
template <int ROWS, bool UNITS>
__device__ void find_seq(const AttnParams &p, const Work &w, long long x, int &b, long long &before) {
    const int lane = threadIdx.x & 31;
    long long base = 0;
    for (int b0 = 0; b0 < p.c.B; b0 += 32) {
        long long mine = 0;
        if (b0 + lane < p.c.B) {
            const SeqWork s = seq_work<ROWS>(p, b0 + lane);
            mine = (long long)p.c.H * s.tiles * (UNITS ? 1 : s.pages + w.cost);
        }
        long long sum = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long v = __shfl_up_sync(0xFFFFFFFFu, sum, o);
            if (lane >= o) sum += v;
        }
        const unsigned hit = __ballot_sync(0xFFFFFFFFu, base + sum > x);
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

// A walk over a run, one piece (pages of one (sequence, head, row tile)) at a time.
template <int ROWS>
struct Walk {
    long long x, end, before;  // place, end of the run, work before sequence b
    int b, cost;
    SeqWork s;
    int h, tile, page0, page1;

    __device__ __forceinline__ void start(const AttnParams &p, const Work &w, long long from, long long to) {
        x = from;
        end = to;
        cost = w.cost;
        find_seq<ROWS, false>(p, w, x, b, before);
        if (b < p.c.B) s = seq_work<ROWS>(p, b);
    }
    // The next piece: pages [page0, page1) of (b, h, tile); false at the end.
    __device__ __forceinline__ bool next(const AttnParams &p) {
        for (;;) {
            if (x >= end) return false;
            while (x - before >= (long long)p.c.H * s.tiles * (s.pages + cost)) {
                before += (long long)p.c.H * s.tiles * (s.pages + cost);
                if (++b >= p.c.B) return false;
                s = seq_work<ROWS>(p, b);
            }
            const int unit = (int)quotient(x - before, s.pages + cost);
            const long long at = before + (long long)unit * (s.pages + cost);  // the row tile's first place
            page0 = max((int)(x - at) - cost, 0);
            page1 = (int)min((long long)s.pages, end - at - cost);
            h = unit / s.tiles;
            tile = unit - h * s.tiles;
            x = at + cost + max(page1, 0);
            if (page1 > page0) return true;
            if (page1 <= 0) x = end;  // the run ends before the row tile's first page
        }
    }
};

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9},"
        " {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(v));
    return d;
}

// The softmax's state, for each row: with x a score in powers of two,
//     p = 2^(x - ref),   l = sum p,   corr = sum p (m + 8 s),   o = sum fp16(p s 2^-ve) c.
// ref is a whole number, kDown above the largest score when it was set; it moves when p passes 2^-8, so that
// the weights of 65,536 equal tokens sum to no more than 2^8 and l and corr stay in fp32's range for any value.
// (Weights below 2^-110 of the row's largest are flushed: the price of kDown, of which 2^-126 leaves 2^-110.)
// ve follows the largest p s that the row met, not the largest s: tokens that the row does not see, or that have
// no weight in it, cost the others nothing (one power for all rows and tokens, and one reference for l and o,
// gave inf for a constant value row of 2^22 and zeros beside an unseen value of 1e30).  The largest p s 2^-ve is
// 2^kUp when ve is set: fp16 has room for it to grow by 2^8 before ve moves, and 2^-21 of it still has its 11
// bits.  Moves are by whole powers of two, so no sum is rounded by them.
constexpr int kUp = 7, kDown = 16;
constexpr float kPTop = 0.00390625f;  // four of a lane's p sum up to more: ref has to move
constexpr float kPsTop = 32768.0f;    // four of a lane's p s 2^-ve sum up to more: ve has to move
constexpr float kNoRef = -1e38f;      // before the first score: any score passes it, and unseen tokens (-inf) do not

// CL > 0: a cluster of CL CTAs takes one row tile, its warps every 4 CL-th page each, and their parts meet
// through distributed shared memory: no second kernel.  For few row tiles of few pages (see few_launch).
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Address of this CTA's shared-memory address in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t peer_address(uint32_t addr, int rank) {
    uint32_t d;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(d) : "r"(addr), "r"(rank));
    return d;
}
__device__ __forceinline__ float peer_load(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

template <int D, int NT, int CL>
__global__ void __launch_bounds__(kFewThreads, (Few<D, NT>::kCtas)) attn_few_kernel(const __grid_constant__ AttnParams p) {
    using F = Few<D, NT>;
    constexpr int kCl = CL ? CL : 1;
    constexpr int kStep = CL ? CL * kFewWarps : 1;  // pages from one of a warp to its next
    constexpr int kRows = F::kRows, kS = F::kStages, MT = D / 16, WK = D / 32, kTiles = F::kTiles;
    extern __shared__ __align__(128) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint8_t *ring = smem + warp * kS * F::kStage;
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + kFewWarps * kS * F::kStage) + warp * kS;
    int *there = reinterpret_cast<int *>(smem + kFewWarps * kS * (F::kStage + 8)) + warp * kS;  // the stage's page exists
    int *abort = reinterpret_cast<int *>(smem + kFewWarps * kS * (F::kStage + 12));
    // lane 0's walk ahead, for the copies (in shared memory: one lane's few accesses a page)
    static_assert(sizeof(Walk<kRows>) <= 120, "walk");
    Walk<kRows> &ahead = *reinterpret_cast<Walk<kRows> *>(smem + kFewWarps * (kS * (F::kStage + 16)) + 16 + 128 * warp);
    int &ahead_page = *reinterpret_cast<int *>(reinterpret_cast<uint8_t *>(&ahead) + 120);
    if (lane == 0) {
        for (int s = 0; s < kS; s++) mbar_init(full + s, 1);
        fence_mbar_init();
    }
    if (threadIdx.x == 0) *abort = 0;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    __syncthreads();
    asm volatile("griddepcontrol.wait;" ::: "memory");  // lengths and cache come from the kernels before
    int run = 0;
    Walk<kRows> walk;
    if (CL) {
        long long units;
        find_seq<kRows, true>(p, Work{}, blockIdx.x / kCl, walk.b, units);
        if (walk.b >= p.c.B) return;  // the whole cluster
        walk.s = seq_work<kRows>(p, walk.b);
        const int unit = (int)(blockIdx.x / kCl - units);
        walk.h = unit / walk.s.tiles;
        walk.tile = unit - walk.h * walk.s.tiles;
        walk.page0 = (int)(blockIdx.x % kCl) * kFewWarps + warp;
        walk.page1 = walk.s.pages;
        if (threadIdx.x == 0 && walk.s.len > p.c.width * SHERRY_KV4_PAGE) atomicCAS(p.err, 0u, (unsigned int)SHERRY_ERR_INDEX);
    } else {
        const Work work = all_work<kRows>(p);
        run = blockIdx.x + gridDim.x * warp;  // neighbouring runs on different SMs
        const long long from = run * work.each, to = min(from + work.each, work.total);
        if (from >= to) return;
        walk.start(p, work, from, to);
    }

    PageRing<kS> pages;
    if (lane == 0) {
        ahead = walk;
        ahead_page = walk.page0;
        if (!CL) ahead.page1 = ahead_page = 0;
    }
    auto copy_next = [&]() {
        while (ahead_page >= ahead.page1) {
            if (CL || !ahead.next(p)) return;
            ahead_page = ahead.page0;
            if (ahead.s.len > p.c.width * SHERRY_KV4_PAGE) atomicCAS(p.err, 0u, (unsigned int)SHERRY_ERR_INDEX);
        }
        const int s = pages.to;
        const int page = ahead.s.len > 0 ? kv4_page(p.c, ahead.b, ahead_page * SHERRY_KV4_PAGE, p.err) : -1;
        there[s] = page >= 0;
        if (page >= 0) {
            mbar_arrive_expect_tx(full + s, F::kStage);
            bulk_load(smem_u32(ring + s * F::kStage), kv4_block<D>(p.c, page, ahead.h, 0), F::kStage, full + s);
        } else {
            mbar_arrive(full + s);
        }
        ahead_page += kStep;
        pages.copy();
    };
    if (lane == 0)
        for (int s = 0; s < kS; s++) copy_next();
    __syncwarp();

    const int r = lane >> 2, c = lane & 3;
    // Row m of a 16-token tile is token tok(m); chosen so that neither the keys' loads (a token per
    // four lanes) nor the values' (four tokens per lane) meet in a bank.
    const int tok_r = r ^ (r >> 2 & 1);                       // rows r and r + 8 (+ 8)
    const int tok_v0 = (2 * c) ^ (c >> 1 & 1), tok_v1 = (2 * c + 1) ^ (c >> 1 & 1);
    const uint32_t flip = p.scale2 < 0.0f ? 0x80008000u : 0u;  // a negative scale turns q's signs
    // After a wait that ran out: copies in flight land before their memory is used again or released.
    auto drain = [&]() {
        volatile int no_abort = 0;
        if (lane == 0)
            pages.drain([&](int s, uint32_t phase) { mbar_wait(full + s, phase, &no_abort, p.err, 1000000000LL); });
        __syncwarp();
    };
    if (p.wait_limit == 1) {  // a drill: no wait is given a look, with the first copies on their way
        pages.dead = true;
        if (lane == 0) atomicCAS(p.err, 0u, (unsigned int)SHERRY_ERR_TIMEOUT);
    }
    for (bool more = CL || walk.next(p); more; more = !CL && walk.next(p)) {
        const int nrow = walk.s.rows * p.g, row0 = walk.tile * kRows;
        const int pos0 = walk.s.len - walk.s.rows;            // position of the first new token
        // q: lane (r, c) holds elements [c D / 4, (c + 1) D / 4) of row r of each row group
        // as fp16 of q 2^-e, the odd nibbles' elements 2^-4 of it again
        uint32_t qf[NT][MT][2];
        float qsum[NT][2];                                    // of rows 2 c, 2 c + 1: sum(q),
        f2 sc[NT];                                            // scale of a score
        int last[NT][2];                                      // last token those rows see
#pragma unroll
        for (int t = 0; t < NT; t++) {
            const int row = row0 + 8 * t + r;
            float sum = 0.0f, most = 0.0f;
            const uint16_t *src = nullptr;
            if (row < nrow)
                src = p.q + (long long)(walk.s.first + row / p.g) * p.q_stride +
                      (long long)(walk.h * p.g + row % p.g) * D + c * (D / 4);
            uint4 u[WK];
#pragma unroll
            for (int w = 0; w < WK; w++) {
                u[w] = make_uint4(0, 0, 0, 0);
                if (src) u[w] = *reinterpret_cast<const uint4 *>(src + 8 * w);
                u[w].x ^= flip, u[w].y ^= flip, u[w].z ^= flip, u[w].w ^= flip;
                const uint32_t e[4] = {u[w].x, u[w].y, u[w].z, u[w].w};
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const float lo = __uint_as_float(e[i] << 16), hi = __uint_as_float(e[i] & 0xFFFF0000u);
                    sum += lo + hi;
                    most = fmaxf(most, fmaxf(fabsf(lo), fabsf(hi)));
                }
            }
            sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 1);
            sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 2);
            most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, 1));
            most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, 2));
            const int e = max((int)(__float_as_uint(most) >> 23) - 127 - 13, -120);  // the largest below 2^14
            const float d0 = pow2(-e), d1 = d0 * 0.0625f;
#pragma unroll
            for (int w = 0; w < WK; w++) {
                // a code word's pairs are elements (i, i + 4)
                const uint32_t lo[2] = {u[w].x, u[w].y}, hi[2] = {u[w].z, u[w].w};
#pragma unroll
                for (int k = 0; k < 2; k++) {
                    qf[t][2 * w + k][0] = pack_f16(__uint_as_float(lo[k] << 16) * d0, __uint_as_float(hi[k] << 16) * d0);
                    qf[t][2 * w + k][1] =
                        pack_f16(__uint_as_float(lo[k] & 0xFFFF0000u) * d1, __uint_as_float(hi[k] & 0xFFFF0000u) * d1);
                }
            }
            sum *= d0 * 5.9604644775390625e-08f;              // 2^-24: in units of the product
            float scale[2];
#pragma unroll
            for (int j = 0; j < 2; j++) {
                qsum[t][j] = __shfl_sync(0xFFFFFFFFu, sum, (2 * c + j) * 4);
                // (not 0: a score of -inf has to stay one)
                scale[j] = fmaxf(fabsf(p.scale2) * pow2(24 + __shfl_sync(0xFFFFFFFFu, e, (2 * c + j) * 4)), 1e-37f);
                const int rw = row0 + 8 * t + 2 * c + j;
                last[t][j] = rw < nrow ? pos0 + rw / p.g : -1;
            }
            sc[t] = pair2(scale[0], scale[1]);
        }
        const int hi_row = min(row0 + kRows, nrow) - 1;
        // rows past the end see nothing; their sums are dropped, so they need no mask
        const int last_min = pos0 + row0 / p.g, last_max = pos0 + hi_row / p.g;
        float o[NT][MT][4];
        f2 nref[NT], down[NT], l[NT], corr[NT];               // of rows 2 c, 2 c + 1: -ref, 2^-ve, ...
#pragma unroll
        for (int t = 0; t < NT; t++) {
#pragma unroll
            for (int i = 0; i < MT; i++)
#pragma unroll
                for (int j = 0; j < 4; j++) o[t][i][j] = 0.0f;
            nref[t] = pair2(-kNoRef, -kNoRef);
            down[t] = pair2(pow2(126), pow2(126));
            l[t] = corr[t] = pair2(0.0f, 0.0f);
        }
        for (int pg = walk.page0; pg < walk.page1; pg += kStep) {
            const int s = pages.at;
            if (!pages.dead) pages.take(__all_sync(0xFFFFFFFFu, mbar_wait(full + s, pages.lap, abort, p.err, p.wait_limit)));
            const int t0 = pg * SHERRY_KV4_PAGE;              // first token of the page
            if (!pages.dead && there[s] && t0 <= last_max) {
                const uint8_t *kb = ring + s * F::kStage, *vb = kb + Kv4<D>::kBlock;
                const bool whole = t0 + SHERRY_KV4_PAGE - 1 <= last_min;
                const uint32_t a1[4] = {0x3C003C00u, 0x3C003C00u, 0x3C003C00u, 0x3C003C00u};
                float ones[NT][4];                            // sums of the page's p s
#pragma unroll
                for (int t = 0; t < NT; t++) ones[t][0] = ones[t][1] = ones[t][2] = ones[t][3] = 0.0f;
#pragma unroll 1
                for (int q0 = 0; q0 < 4; q0 += kTiles) {
                    float x[kTiles][NT][4];                       // scores of tiles of 16 tokens
#pragma unroll
                    for (int qi = 0; qi < kTiles; qi++) {
                        const int q = q0 + qi;
                        const int ta = 16 * q + tok_r;            // rows r, r + 8 of the tile
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
                        const uint32_t kp[2] = {ksm[0], ksm[8]};
#pragma unroll
                        for (int t = 0; t < NT; t++) x[qi][t][0] = x[qi][t][1] = x[qi][t][2] = x[qi][t][3] = 0.0f;
#pragma unroll
                        for (int w = 0; w < WK; w++)
#pragma unroll
                            for (int k = 0; k < 2; k++) {
                                const uint32_t u0 = kw[0][w] >> (8 * k), u1 = kw[1][w] >> (8 * k);
                                const uint32_t a[4] = {u0 & 0x000F000Fu, u1 & 0x000F000Fu, u0 & 0x00F000F0u, u1 & 0x00F000F0u};
#pragma unroll
                                for (int t = 0; t < NT; t++) mma_f16(x[qi][t], a, qf[t][2 * w + k][0], qf[t][2 * w + k][1]);
                            }
#pragma unroll
                        for (int t = 0; t < NT; t++)
#pragma unroll
                            for (int i = 0; i < 2; i++)
#pragma unroll
                                for (int j = 0; j < 2; j++)
                                    x[qi][t][2 * i + j] = kv4_step(kp[i]) * x[qi][t][2 * i + j] + kv4_low(kp[i]) * qsum[t][j];
                    }
                    float sv[kTiles][2], mv[kTiles][2];           // steps and centres of the values
#pragma unroll
                    for (int qi = 0; qi < kTiles; qi++)
#pragma unroll
                        for (int i = 0; i < 2; i++) {
                            const uint32_t vp = reinterpret_cast<const uint32_t *>(vb + Kv4<D>::kCodes)[16 * (q0 + qi) + tok_r + 8 * i];
                            sv[qi][i] = kv4_step(vp);
                            mv[qi][i] = kv4_low(vp) + 8.0f * sv[qi][i];
                        }
                    if (!whole) {
                        // A token that a row does not see may hold anything: its probability is 2^-inf, and a step or
                        // centre that is not a number goes to the score of the rows that do see it.
#pragma unroll
                        for (int qi = 0; qi < kTiles; qi++)
#pragma unroll
                            for (int i = 0; i < 2; i++) {
                                const int tok = t0 + 16 * (q0 + qi) + tok_r + 8 * i;
                                const bool bad = !(fabsf(sv[qi][i]) < INFINITY && fabsf(mv[qi][i]) < INFINITY);
                                if (bad || tok > last_max) sv[qi][i] = mv[qi][i] = 0.0f;
#pragma unroll
                                for (int t = 0; t < NT; t++)
#pragma unroll
                                    for (int j = 0; j < 2; j++) {
                                        if (bad) x[qi][t][2 * i + j] = __int_as_float(0x7FFFFFFF);
                                        if (tok > last[t][j]) x[qi][t][2 * i + j] = -INFINITY;
                                    }
                            }
                    }
                    uint32_t pb[kTiles][NT][2];
                    f2 sum[NT], csum[NT];
                    // References and powers move only when a lane's sums outgrow them: most pages skip the shuffles and
                    // the rescaling.
                    for (bool moved = false;; moved = true) {
                        f2 most[NT];
#pragma unroll
                        for (int t = 0; t < NT; t++) sum[t] = csum[t] = most[t] = pair2(0.0f, 0.0f);
#pragma unroll
                        for (int qi = 0; qi < kTiles; qi++)
#pragma unroll
                            for (int i = 0; i < 2; i++) {
                                const f2 s2 = pair2(sv[qi][i], sv[qi][i]), m2 = pair2(mv[qi][i], mv[qi][i]);
#pragma unroll
                                for (int t = 0; t < NT; t++) {
                                    float a, b;
                                    split2(fma2(pair2(x[qi][t][2 * i], x[qi][t][2 * i + 1]), sc[t], nref[t]), a, b);
                                    const f2 pr = pair2(exp2_fast(a), exp2_fast(b));
                                    const f2 ps = mul2(mul2(pr, s2), down[t]);
                                    sum[t] = add2(sum[t], pr);
                                    csum[t] = fma2(pr, m2, csum[t]);
                                    most[t] = add2(most[t], ps);
                                    split2(ps, a, b);
                                    pb[qi][t][i] = pack_f16(a, b);
                                }
                            }
                        bool grow = false;
#pragma unroll
                        for (int t = 0; t < NT; t++) {
                            float a, b;
                            split2(sum[t], a, b);
                            grow |= fmaxf(a, b) > kPTop;
                            split2(most[t], a, b);
                            grow |= fmaxf(a, b) > kPsTop;
                        }
                        // once is enough (a row of nothing but NaN has no reference after it either)
                        if (moved || !__any_sync(0xFFFFFFFFu, grow)) break;
#pragma unroll
                        for (int t = 0; t < NT; t++) {
                            float scale[2], old[2], d[2], f[2], fo[2];
                            split2(sc[t], scale[0], scale[1]);
                            split2(nref[t], old[0], old[1]);
                            split2(down[t], d[0], d[1]);
#pragma unroll
                            for (int j = 0; j < 2; j++) {
                                // largest score, and largest score of p s (up to a factor of two)
                                float mx = -INFINITY, ms = -INFINITY;
#pragma unroll
                                for (int k = 0; k < 2 * kTiles; k++) {
                                    const float y = x[k >> 1][t][2 * (k & 1) + j] * scale[j];
                                    mx = fmaxf(mx, y);
                                    ms = fmaxf(ms, y + (float)((int)(__float_as_uint(sv[k >> 1][k & 1]) >> 23 & 255) - 126));
                                }
#pragma unroll
                                for (int k = 4; k < 32; k <<= 1) {
                                    mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, k));
                                    ms = fmaxf(ms, __shfl_xor_sync(0xFFFFFFFFu, ms, k));
                                }
                                const float ref = fmaxf(-old[j], ceilf(mx) + (float)kDown), by = -old[j] - ref;   // by <= 0
                                // what is summed already needs no more than its power, by lower
                                const float ve = (float)(127 - (int)(__float_as_uint(d[j]) >> 23));
                                const float to = fmaxf(fmaxf(ve + by, ceilf(ms - ref) - (float)kUp), -126.0f);
                                old[j] = -ref;
                                d[j] = __int_as_float((127 - (int)to) << 23);
                                f[j] = exp2_fast(by);
                                fo[j] = exp2_fast(ve + by - to);
                                ones[t][j] *= fo[j];
#pragma unroll
                                for (int i = 0; i < MT; i++) {
                                    o[t][i][j] *= fo[j];
                                    o[t][i][2 + j] *= fo[j];
                                }
                            }
                            nref[t] = pair2(old[0], old[1]);
                            down[t] = pair2(d[0], d[1]);
                            l[t] = mul2(l[t], pair2(f[0], f[1]));
                            corr[t] = mul2(corr[t], pair2(f[0], f[1]));
                        }
                    }
#pragma unroll
                    for (int t = 0; t < NT; t++) {
                        l[t] = add2(l[t], sum[t]);
                        corr[t] = add2(corr[t], csum[t]);
                    }
#pragma unroll
                    for (int qi = 0; qi < kTiles; qi++) {
                        const int q = q0 + qi;
#pragma unroll
                        for (int t = 0; t < NT; t++)
#pragma unroll
                            for (int i = 0; i < 2; i++) pb[qi][t][i] = transpose8x8(pb[qi][t][i]);
                        // values: lane (r, c) holds word(s) r of four tokens; a pair of tokens per register
#pragma unroll
                        for (int w = 0; w < D / 64; w++) {
                            const uint8_t *src = vb + 16 * q * Kv4<D>::kRow + (r * (D / 64) + w) * 4;
                            const uint32_t w0 = *reinterpret_cast<const uint32_t *>(src + tok_v0 * Kv4<D>::kRow);
                            const uint32_t w1 = *reinterpret_cast<const uint32_t *>(src + tok_v1 * Kv4<D>::kRow);
                            const uint32_t w2 = *reinterpret_cast<const uint32_t *>(src + (tok_v0 + 8) * Kv4<D>::kRow);
                            const uint32_t w3 = *reinterpret_cast<const uint32_t *>(src + (tok_v1 + 8) * Kv4<D>::kRow);
                            const uint32_t al = prmt(w0, w1, 0x5410), ah = prmt(w0, w1, 0x7632);
                            const uint32_t bl = prmt(w2, w3, 0x5410), bh = prmt(w2, w3, 0x7632);
#pragma unroll
                            for (int i = 0; i < 4; i++) {
                                const uint32_t mask = i & 1 ? 0x00F000F0u : 0x000F000Fu;
                                const int sh = 8 * (i >> 1);
                                const uint32_t a[4] = {(al >> sh) & mask, (ah >> sh) & mask, (bl >> sh) & mask, (bh >> sh) & mask};
#pragma unroll
                                for (int t = 0; t < NT; t++) mma_f16(o[t][4 * w + i], a, pb[qi][t][0], pb[qi][t][1]);
                            }
                        }
#pragma unroll
                        for (int t = 0; t < NT; t++) mma_f16(ones[t], a1, pb[qi][t][0], pb[qi][t][1]);
                    }
                }
                // The tensor cores' sums round towards zero, and a long sum of codes 0 .. 15 drifts (32,768 tokens
                // came out at twice the error of a bf16 result): the page's 8 sum(p s) comes off again, so that the
                // sums stay small.  (Codes less 8 as operands cost an instruction per pair: 251 us against 212.)
#pragma unroll
                for (int t = 0; t < NT; t++)
#pragma unroll
                    for (int j = 0; j < 2; j++) {
                        const float e0 = ones[t][j] * -4.76837158203125e-07f, e1 = ones[t][j] * -7.62939453125e-06f;  // -8 2^-24, -8 2^-20
#pragma unroll
                        for (int i = 0; i < MT; i++) {
                            o[t][i][j] += i & 1 ? e1 : e0;
                            o[t][i][2 + j] += i & 1 ? e1 : e0;
                        }
                    }
            }
            __syncwarp();
            if (lane == 0 && !pages.dead) copy_next();
        }

        // ---------------- the piece's result: references, totals, sums p v ----------------
        float ref[NT][2], tot[NT][2];
#pragma unroll
        for (int t = 0; t < NT; t++) {
            float add[2], d[2];
            split2(nref[t], ref[t][0], ref[t][1]);
            split2(l[t], tot[t][0], tot[t][1]);
            split2(corr[t], add[0], add[1]);
            split2(down[t], d[0], d[1]);
#pragma unroll
            for (int j = 0; j < 2; j++) {
                ref[t][j] = -ref[t][j];
#pragma unroll
                for (int k = 4; k < 32; k <<= 1) {
                    tot[t][j] += __shfl_xor_sync(0xFFFFFFFFu, tot[t][j], k);
                    add[j] += __shfl_xor_sync(0xFFFFFFFFu, add[j], k);
                }
                const float up = __uint_as_float((254u << 23) - __float_as_uint(d[j]));  // 2^ve
#pragma unroll
                for (int i = 0; i < MT; i++) {
                    const float f = i & 1 ? 1048576.0f : 16777216.0f;  // the codes' 2^-20 and 2^-24
                    o[t][i][j] = o[t][i][j] * f * up + add[j];
                    o[t][i][2 + j] = o[t][i][2 + j] * f * up + add[j];
                }
            }
        }
        if (CL) {
            if (pages.dead) drain();
            // each warp's part into its own ring: [row][D] sums, then the rows' references and totals
            float *part = reinterpret_cast<float *>(ring);
#pragma unroll
            for (int t = 0; t < NT; t++)
#pragma unroll
                for (int j = 0; j < 2; j++) {
                    const int row = 8 * t + 2 * c + j;
#pragma unroll
                    for (int i = 0; i < MT; i += 4)
#pragma unroll
                        for (int k = 0; k < 2; k++)
                            *reinterpret_cast<float4 *>(part + row * D + r * (D / 8) + 2 * i + 4 * k) =
                                make_float4(o[t][i][2 * k + j], o[t][i + 1][2 * k + j], o[t][i + 2][2 * k + j],
                                            o[t][i + 3][2 * k + j]);
                    if (r == 0)
                        reinterpret_cast<float2 *>(part + kRows * D)[row] =
                            make_float2(ref[t][j], tot[t][j]);
                }
            cluster_sync();
            // the cluster's CTAs share the rows; lane i holds the weight of part i, the parts in order
            constexpr int kParts = kCl * kFewWarps, kMine = kRows / kCl;
            static_assert(kParts <= 32 && kMine * kCl == kRows, "a lane per part");
            const uint32_t mine = smem_u32(smem);
            const int part_i = lane % kParts;
            const uint32_t from = peer_address(mine + (part_i % kFewWarps) * kS * F::kStage, part_i / kFewWarps);
            for (int n = warp; n < kMine * (D / 32); n += kFewWarps) {
                const int row = (int)(blockIdx.x % kCl) * kMine + n / (D / 32), d = n % (D / 32) * 32 + lane, rw = row0 + row;
                const float pm = peer_load(from + (kRows * D + 2 * row) * 4), pl = peer_load(from + (kRows * D + 2 * row + 1) * 4);
                float mx = pm;
#pragma unroll
                for (int k = 16; k > 0; k >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, k));
                const float f = exp2_fast(pm - mx);  // (a part without keys has kNoRef and sums of 0)
                float sum = lane < kParts ? pl * f : 0.0f, acc = 0.0f;
#pragma unroll
                for (int k = 16; k > 0; k >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, k);
#pragma unroll 16
                for (int k = 0; k < kParts; k++)
                    acc += __shfl_sync(0xFFFFFFFFu, f, k) * peer_load(__shfl_sync(0xFFFFFFFFu, from, k) + (row * D + d) * 4);
                if (rw < nrow)
                    p.out[(long long)(walk.s.first + rw / p.g) * p.out_stride + (long long)(walk.h * p.g + rw % p.g) * D + d] =
                        __bfloat16_as_ushort(__float2bfloat16_rn(sum == 0.0f ? 0.0f : acc * (1.0f / sum)));
            }
            cluster_sync();  // no CTA leaves while its memory is read
            return;
        }
        const bool all = walk.page0 == 0 && walk.page1 == walk.s.pages;
        // parts of a row tile: slot 1 of the run that holds its first page, slot 0 of the others
        const long long slot = 2LL * run + (walk.page0 == 0 ? 1 : 0);
#pragma unroll
        for (int t = 0; t < NT; t++)
#pragma unroll
            for (int j = 0; j < 2; j++) {
                const int row = 8 * t + 2 * c + j, rw = row0 + row;
                if (rw >= nrow) continue;
                if (all) {
                    const float inv = tot[t][j] == 0.0f ? 0.0f : 1.0f / tot[t][j];
                    uint16_t *dst = p.out + (long long)(walk.s.first + rw / p.g) * p.out_stride +
                                    (long long)(walk.h * p.g + rw % p.g) * D + r * (D / 8);
#pragma unroll
                    for (int i = 0; i < MT; i += 4) {
                        float v[8];  // elements 2 i ... 2 i + 7 of the lane's D / 8
#pragma unroll
                        for (int k = 0; k < 8; k++) v[k] = o[t][i + (k & 3)][2 * (k >> 2) + j] * inv;
                        *reinterpret_cast<uint4 *>(dst + 2 * i) =
                            make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
                    }
                } else {
                    float *dst = p.ws + (slot * kRows + row) * D + r * (D / 8);
#pragma unroll
                    for (int i = 0; i < MT; i += 4)
#pragma unroll
                        for (int k = 0; k < 2; k++)
                            *reinterpret_cast<float4 *>(dst + 2 * i + 4 * k) =
                                make_float4(o[t][i][2 * k + j], o[t][i + 1][2 * k + j], o[t][i + 2][2 * k + j],
                                            o[t][i + 3][2 * k + j]);
                    if (r == 0)
                        reinterpret_cast<float2 *>(p.ws + 2LL * p.grid * kRows * D)[slot * kRows + row] =
                            make_float2(ref[t][j], tot[t][j]);
                }
            }
    }
    if (pages.dead) drain();
}

// Joins the parts of the row tiles that the runs cut: a CTA per 8 rows of one, JW warps per row, which take
// 32 parts in turn and whose sums are added in order.
template <int D, int NT, int JW>
__global__ void __launch_bounds__(256 * JW, JW == 1 ? 2 : 1) attn_join_kernel(const __grid_constant__ AttnParams p) {
    constexpr int kRows = 8 * NT, E = D / 32;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int mine = warp % JW, row = warp / JW + 8 * blockIdx.y;
    const Work work = all_work<kRows>(p);
    int b;
    long long units, before;
    find_seq<kRows, true>(p, work, blockIdx.x, b, units);
    if (b >= p.c.B) return;
    const SeqWork s = seq_work<kRows>(p, b);
    const int unit = (int)(blockIdx.x - units);
    before = 0;
    for (int i = lane; i < b; i += 32) {
        const SeqWork t = seq_work<kRows>(p, i);
        before += (long long)p.c.H * t.tiles * (t.pages + work.cost);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) before += __shfl_xor_sync(0xFFFFFFFFu, before, o);
    const int h = unit / s.tiles, rw = (unit - h * s.tiles) * kRows + row;
    const long long x0 = before + (long long)unit * (s.pages + work.cost) + work.cost;  // the first page's place
    const int i0 = (int)quotient(x0, work.each), i1 = (int)quotient(x0 + s.pages - 1, work.each);
    if (i0 == i1) return;  // one run held all of it and wrote the result
    const bool live = rw < s.rows * p.g;
    if (JW == 1 && !live) return;
    const float2 *ml = reinterpret_cast<const float2 *>(p.ws + 2LL * p.grid * kRows * D);
    float m = -INFINITY;
    for (int i = i0 + lane; live && i <= i1; i += 32) m = fmaxf(m, ml[(2LL * i + (i == i0)) * kRows + row].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    float l = 0.0f, acc[E];
#pragma unroll
    for (int e = 0; e < E; e++) acc[e] = 0.0f;
    for (int ib = i0 + 32 * mine; live && ib <= i1; ib += 32 * JW) {
        const int i = ib + lane;
        float f = 0.0f;
        if (i <= i1) {
            const float2 v = ml[(2LL * i + (i == i0)) * kRows + row];
            f = exp2_fast(v.x - m);  // (a part without keys has kNoRef and sums of 0)
            l += v.y * f;
        }
        const int k1 = min(32, i1 - ib + 1);
#pragma unroll 16
        for (int k = 0; k < k1; k++) {
            const float fk = __shfl_sync(0xFFFFFFFFu, f, k);
            const long long slot = 2LL * (ib + k) + (ib + k == i0);
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
    if (JW > 1) {
        __shared__ float part[8][JW][D + 1];
        float *to = part[warp / JW][mine];
#pragma unroll
        for (int e = 0; e < E; e++) to[lane * E + e] = acc[e];
        if (lane == 0) to[D] = l;
        __syncthreads();
        if (!live || mine != 0) return;
#pragma unroll
        for (int w = 1; w < JW; w++) {
            const float *from = part[warp / JW][w];
            l += from[D];
#pragma unroll
            for (int e = 0; e < E; e++) acc[e] += from[lane * E + e];
        }
    }
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
void launch_after(K kernel, dim3 grid, int threads, size_t smem, cudaStream_t stream, const AttnParams &p, int cluster = 1) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    cudaLaunchKernelEx(&cfg, kernel, p);
}

template <int D, int NT>
sherry_status few_launch(AttnParams p, cudaStream_t stream) {
    using F = Few<D, NT>;
    static OccupancyCache cache;
    const int bps = few_blocks_per_sm(attn_few_kernel<D, NT, 0>, F::kSmem, cache);
    // at most this many row tiles, and with the rows shared out evenly so many
    const long long seqs = std::min(p.c.B, p.c.T), rows = (long long)p.c.T * p.g;  // sequences with rows, at most
    long long tiles = rows / F::kRows + seqs;
    if (p.few_rows < 0x7FFFFFFF) tiles = std::min(tiles, seqs * ((p.few_rows + F::kRows - 1) / F::kRows));
    if (!p.c.cu) tiles = seqs * ((p.g + F::kRows - 1) / F::kRows);
    const long long even = std::min(tiles, (rows + seqs * F::kRows - 1) / (seqs * F::kRows) * seqs) * p.c.H;
    tiles *= p.c.H;
    if (tiles > 0x7FFFFFFF) return SHERRY_ERR_UNSUPPORTED;
    // A cluster per row tile, or equal runs and a join.  In pages one after the other, if every sequence is as
    // long as its table: the largest cluster of which all are resident at once, against the runs and about
    // kJoinPages for the join and its launch.  Clusters and runs, us, one new token and 8 heads each: one
    // sequence of 2,048 tokens, heads of 64, 6.6 and 10.9; of 8,192, 10.5 and 14.5; 16 of 2,048, heads of 128,
    // 18.7 and 22.8 (clusters of 2; of 8, in more than one wave, 31.0); 64 of 1,024, heads of 64, clusters of 8
    // in waves 61.9 and 24.7 (of 2, in waves too, 21.0: the rule passes those by).
    const long long slots = (long long)sm_count() * bps, width = p.c.width;
    const long long by_runs = (even * width + slots * kFewWarps - 1) / (slots * kFewWarps) + kJoinPages;
    auto clusters = [&](auto size) {
        constexpr int CL = decltype(size)::value;
        if (width == 1 || even * CL > slots || (width + CL * kFewWarps - 1) / (CL * kFewWarps) > by_runs) return false;
        static OccupancyCache cluster_cache;
        few_blocks_per_sm(attn_few_kernel<D, NT, CL>, F::kSmem, cluster_cache);
        launch_after(attn_few_kernel<D, NT, CL>, dim3((unsigned)(tiles * CL)), kFewThreads, F::kSmem, stream, p, CL);
        return true;
    };
    if (clusters(std::integral_constant<int, 8>{}) || clusters(std::integral_constant<int, 4>{}) ||
        clusters(std::integral_constant<int, 2>{}))
        return launch_status("sherry_attn_kv4");
    const int ctas = std::min(sm_count() * bps, kFewRunsMax / kFewWarps);
    p.grid = ctas * kFewWarps;  // runs
    launch_after(attn_few_kernel<D, NT, 0>, dim3((unsigned)ctas), kFewThreads, F::kSmem, stream, p);
    const sherry_status st = launch_status("sherry_attn_kv4");
    // a table of one page cuts nothing
    if (st != SHERRY_OK || p.c.width == 1) return st;
    // Up to about this many parts a row tile: four warps a row for one long sequence (24 us against 36 at
    // 32,768 tokens, heads of 64), one for many (29 us against 41 for 64 sequences of 1,024).
    const long long parts = std::min<long long>(p.grid / tiles, p.c.width);
    if (parts > 32) launch_after(attn_join_kernel<D, NT, 4>, dim3((unsigned)tiles, NT), 1024, 0, stream, p);
    else launch_after(attn_join_kernel<D, NT, 1>, dim3((unsigned)tiles, NT), 256, 0, stream, p);
    return launch_status("sherry_attn_kv4 (join)");
}

}  // namespace
}  // namespace sherry

namespace sherry {
namespace {

// Which kernel is ahead for sequences of more than kFewRows rows, from what the host knows.  The few-row
// kernel spreads a sequence's pages over the machine but decodes them again for every 16 rows; the tile
// kernel decodes once for 256 rows, one CTA to a key/value head however long the context.  Measured, per
// page of context: 0.25 to 0.35 us for 16 rows of a head on one SM, against 1.0 to 1.2 us for 256 (heads
// of 64 and 128).  E.g. 8 heads, 8,192 tokens, heads of 64: 256 rows 39 us against 135, 1,024 rows 122
// against 136, 2,048 rows 230 against 136.
bool few_is_faster(const sherry_kv4 *c, int g) {
    const long long rows = c->T * g, sms = sm_count();
    const long long few = c->H * (rows / 16 + c->B), tile = c->H * (rows / 256 + c->B);
    return few * 27 < 100 * sms * ((tile + sms - 1) / sms);
}

}  // namespace
}  // namespace sherry

// The parts of the row tiles that the runs of the few-row kernel cut: at most two per run, each
// with 16 rows of D sums, a maximum and a total.
extern "C" size_t sherry_attn_kv4_workspace_bytes(int64_t T, int Hq, int D) {
    if (T < 1 || Hq < 1 || (D != 64 && D != 128)) return 0;
    return (size_t)2 * sherry::kFewRunsMax * 16 * (size_t)(D + 2) * 4;
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
    if (Hq > 65535 || c->T * (Hq / c->H) > 0x7FFFFFFF) return SHERRY_ERR_UNSUPPORTED;
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
    if (most > kFewRows && !few_is_faster(c, p.g)) {
        // a batch may hold both kinds; a lone sequence is one or the other
        p.few_rows = c->B == 1 ? -1 : kFewRows;
        st = attn_tile_launch(p, c->D, s);
        if (st != SHERRY_OK || c->B == 1) return st;
    }
    const bool one = most <= 8;
    if (c->D == 64) return one ? few_launch<64, 1>(p, s) : few_launch<64, 2>(p, s);
    return one ? few_launch<128, 1>(p, s) : few_launch<128, 2>(p, s);
}
