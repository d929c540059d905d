// attn_tile.cu -- causal attention over the 4-bit cache for sequences with many new tokens
// (prompts, chunks of prompts): both products on the tcgen05 tensor cores.
//
// A CTA takes 256 rows of one key/value head, as two tiles of 128, so that each decoded key and
// value serves both (and all query heads of the group: a row is a new token and a query head).
// Per step of 128 tokens:
//     S = Q K^T            fp16 operands, K-major, in shared memory; S (fp32) in tensor memory
//     P = fp16(2^(f S - m + e))  back into S's tensor memory, the A operand of
//     O += P V             V transposed to [D][tokens], so that both operands are K-major
// and l += sum 2^(f S - m) in fp32;  out = O 2^-off / l (e and off: below).
// Precision: decoded values are m + s c rounded once to fp16 (11 bits; bf16's 8 would cost the
// scores of a peaked softmax several percent), after a division by a power of two that brings the
// largest to about 2^-6: there a code's bits are themselves an fp16, c 2^-24, and one FMA makes the
// value.  A page's keys and a step's values share a power where their tokens' sizes lie within 2^7 of
// each other (fp16's subnormals then cost no more than its normal rounding); elsewhere every token has
// its own.  The powers of keys multiply the scores, those of values the probabilities, before these are
// rounded: P = fp16(2^(x - m) 2^(e + off)), e the value's power, m and off the row's own, so that no
// row depends on the size of a token that it does not see or that has no weight in it.
// Queries are bf16: a power of two per row makes them exact in fp16.
// The largest P of a row is 2^9 to 2^16: relative 2^-11 down to 2^-23 of the largest.  References move by
// whole powers of two: nothing that is stored is rounded by them (only what leaves fp16's range below).
// Roles: warps 0-3 and 4-7 the softmax of a tile each (a thread owns a row: no shuffles), warps
// 8-9 decode keys, 10-11 values, warp 12 issues the products, 13 copies pages (codes of keys and
// values of a page are one bulk copy).  The tiles alternate: while one's softmax runs, the tensor
// cores work for the other.
// The bounds, in clocks per 256 rows and 128 tokens (heads of 64; 128): the exponentials 2,048 (16 a clock
// and SM), the products 1,024; 2,048, shared memory 1,150; 2,300 (decoded operands written once and read
// by the products, whose scores alone take all of its bandwidth while they run).  Measured: 3,900; 4,500.
// A tile's softmax (about 2,300 clocks with two of them on the exponentials' unit) and its products (600;
// 1,300) follow each other, and the other tile fills only part of the gap.  4 prompts' chunks of 4,096 tokens
// at 16,384, 32 heads of 128 over 8: 3.8 ms in a graph, 1,010 TFLOP/s (4.0 ms in calls with changing inputs); a
// prompt of 2,048, heads of 64: 47.6 us.
// Tried, in clocks per step with heads of 128 unless said otherwise:
//   codes as operands, steps and low ends applied by the softmax threads from shared memory: 8,000
//   the present operands, code unrolled over the step (four roles' straight-line code does not fit the
//     instruction cache, every role ran at six clocks an instruction): 7,000; a pass of its own for the
//     maximum: 5,000
//   one branch-free step of 128 columns with a test at its end: the same, slower for short prompts
//   two S of 64 columns for each tile, so that neither side waits: 5,000 (products of 64 columns and twice
//     the hand-overs cost more than the waiting)
//   P beside S (there is room for heads of 64), the next scores issued early: 3,900 to 4,200 for heads of 64
//   a share of the exponentials as polynomials on the FMA pipe: 1 in 8 1% slower, 3 in 8 5% slower
#include <algorithm>
#include <cstddef>

#include "attn.cuh"

namespace sherry {
namespace {

constexpr int kRowsTile = 128;
constexpr int kRowsCta = 2 * kRowsTile;
constexpr int kKeys = 128;                 // tokens per step: two pages
// Four warpgroups launched with 128 registers a thread (the last: issue, copies and two idle warps);
// the softmax takes 176, the decoders 96, the last 64: 2 * 176 + 96 + 64 = 4 * 128.
constexpr int kTileThreads = 16 * 32;
constexpr int kInfoSlots = 3;
constexpr int kUp = 10;                    // the largest P of a row is 2^10 when its reference is set
constexpr int kAllSeen = 0x7FFFFFFF - 2 * kKeys;
constexpr int kTmemCols = 512;             // S0, S1 (128 columns each), O0, O1 (D each)
constexpr long long kDrainLimit = 1000000000LL;

template <int D>
struct Tile {
    static constexpr int kQ = kRowsTile * D * 2;      // one tile's queries
    static constexpr int kOp = kKeys * D * 2;         // decoded keys or values of a step
    static constexpr int kPage = 2 * Kv4<D>::kBlock;  // a page of a head, as it is in the cache
    static constexpr int kBars = 1024;
    // One CTA per SM in any case (its tensor memory), so heads of 64 ask for as much as keeps a second
    // one away.  No room is left for aligning the operands: the base is at 1024 (checked).
    static constexpr size_t kUse = 2 * kQ + 4 * kOp + 4 * kPage + kBars;
    static constexpr size_t kSmem = kUse < 120 * 1024 ? 120 * 1024 : kUse;
};

// D = fp32, A and B = fp16, both K-major, 128 x N
template <int N>
constexpr uint32_t kIdesc = (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(kRowsTile >> 4) << 24);

// What the softmax has to know of a step, with kOffset added to every power.
constexpr int kOffset = 120;               // powers are -119 .. 134
constexpr int kApart = 256;                // set in key_exp, value_exp: the tokens have powers of their own
constexpr int kMostExp = 120;              // above it keys are taken token by token too (2^key_exp is a float below)
constexpr int kBad = 255;                  // as a token's value power: the value is NaN
struct alignas(16) StepInfo {
    int key_exp[2];       // a key of the first, second page is its fp16 value times 2^key_exp
    int value_exp;        // a value is its fp16 value times 2^value_exp
    int there;            // bit 0, 1: the first, second page is in the cache
    uint8_t key_of[kKeys], value_of[kKeys];  // the tokens' powers where they have their own
};

static_assert(offsetof(StepInfo, key_of) % 16 == 0 && offsetof(StepInfo, value_of) % 16 == 0, "read 16 bytes at a time");

struct TileBars {
    StepInfo info[kInfoSlots];
    uint64_t q_full, k_full[2], k_empty[2], v_full[2], v_empty[2], info_full[kInfoSlots];
    uint64_t s_full[2], p_full[2], o_full[2], raw_full[2], raw_empty[2], drain;
    uint32_t tmem;
    int abort;
    int there[2];            // of the raw pages
};

template <int N>
__device__ __forceinline__ void regs_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void regs_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

// tmem_ld_wait that the loaded registers depend on: nothing that reads them moves above it.
__device__ __forceinline__ void tmem_ld_wait32(uint32_t (&r)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                   "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]),
                   "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]),
                   "+r"(r[29]), "+r"(r[30]), "+r"(r[31])::"memory");
}

// Power of two to divide by so that magnitudes up to `most` become at most 2^-6.
__device__ __forceinline__ int exp_for(float most) {
    return max((int)(__float_as_uint(most) >> 23) - 127 + 7, -119);  // most >= 0 and finite
}
// Two values m + s c, c the nibbles of x that MASK names, read as fp16 (c 2^-24, or c 2^-20 for the
// nibbles one up): s is the step times 2^24 or 2^20 to match.
template <uint32_t MASK>
__device__ __forceinline__ uint32_t value_pair(uint32_t x, uint32_t s, uint32_t m) {
    uint32_t d;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(x & MASK), "r"(s), "r"(m));
    return d;
}

// A pair (step, low end) whose values are finite and can be ordered: magnitude bound of its values,
// 0 where it is not.
__device__ __forceinline__ float pair_most(uint32_t sm) {
    const float v = fmaxf(fabsf(kv4_low(sm)), fabsf(kv4_low(sm) + 15.0f * kv4_step(sm)));
    return v < INFINITY ? v : 0.0f;
}
__device__ __forceinline__ bool pair_bad(uint32_t sm) {
    return !(fabsf(kv4_low(sm)) < INFINITY && fabsf(kv4_low(sm) + 15.0f * kv4_step(sm)) < INFINITY);
}

// The power that tokens of a warp's sizes `most` share, kOffset added, and kApart where they cannot: `least` is
// the smallest size, any but 0 (those ask for no power: +inf), and 0 for a token that needs a look of its own.
__device__ __forceinline__ int shared_exp(float least, float most) {
    const int hi = (int)__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(most));
    const int lo = (int)__reduce_min_sync(0xFFFFFFFFu, __float_as_uint(least));
    return exp_for(__int_as_float(hi)) + kOffset + (lo < max((hi & 0x7F800000) - (7 << 23), 1) ? kApart : 0);
}

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t one;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xFFFFFFFF;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(one));
    return one != 0;
}

// One k-step of 16.  Operands are low descriptor words (address / 16) and constant offsets, put
// together where they are used: 64-bit descriptors kept ready for 32 k-steps would spill.
constexpr uint32_t kDescHigh = (1024u >> 4) | (1u << 14) | (2u << 29);  // 8-row groups 1024 bytes apart, version 1, 128-byte swizzle
template <int A, int B>
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b32 x, y;\n\t.reg .b64 da, db;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "add.u32 x, %1, %5;\n\tadd.u32 y, %2, %6;\n\t"
        "mov.b64 da, {x, %7};\n\tmov.b64 db, {y, %7};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"(acc), "n"(A), "n"(B), "r"(kDescHigh)
        : "memory");
}
template <int A, int B>
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b32 x, y;\n\t.reg .b64 db;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "add.u32 x, %1, %5;\n\tadd.u32 y, %2, %6;\n\t"
        "mov.b64 db, {y, %7};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [x], db, %3, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"(acc), "n"(A), "n"(B), "r"(kDescHigh)
        : "memory");
}
template <int K, int N, int ROWS>
__device__ __forceinline__ void mma_ss_all(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc) {
    if constexpr (K < N) {
        constexpr int off = ((K / 4) * (ROWS * 128) + (K & 3) * 32) >> 4;
        mma_ss<off, off>(d, a, b, idesc, K != 0);
        mma_ss_all<K + 1, N, ROWS>(d, a, b, idesc);
    }
}
template <int K, int N, int ROWS>
__device__ __forceinline__ void mma_ts_all(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t acc) {
    if constexpr (K < N) {
        mma_ts<8 * K, (((K / 4) * (ROWS * 128) + (K & 3) * 32) >> 4)>(d, a, b, idesc, K != 0 ? 1u : acc);
        mma_ts_all<K + 1, N, ROWS>(d, a, b, idesc, acc);
    }
}

// One arrival for a warp's work: 32 lanes on one barrier are 32 atomics in a row, in the way of the
// products' operand reads (a step of heads of 128 took 7,600 clocks instead of 5,000).
__device__ __forceinline__ void warp_arrive(uint64_t *b) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(b);
}

// mbar_wait by a whole warp; its lanes go on together.
__device__ __forceinline__ bool warp_wait(uint64_t *b, uint32_t parity, volatile int *abort, unsigned int *err,
                                          long long limit) {
    return __all_sync(0xFFFFFFFFu, mbar_wait(b, parity, abort, err, limit));
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

// 32 lanes x 32 bit, 8 or 16 consecutive columns: thread t reads or writes lane (base + t).
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr)
                 : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
                 "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15,"
        " %16};" ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

// A row's state: with x its scores, l = sum 2^(x - m) in two halves, and O is in units of 2^-off of that.
// m and off are whole numbers.
struct RowSums {
    float m;
    int off;
    f2 l;
};

// The factors that bring sums of 2^(x - m), and P and O, to a moved reference.
struct Moved {
    float l, o;
};

// Moves a row's reference: its largest score so far is at least mx (in the part at hand; -inf: none), and the
// part's largest P is 2^(mp - m + off).  The part's largest becomes 2^kUp or what was there keeps its size,
// whichever is lower.
__device__ __forceinline__ Moved move_row(float mx, float mp, RowSums &row) {
    const float up = fmaxf(row.m, ceilf(mx));
    const bool fresh = row.m == -INFINITY;
    if (up == -INFINITY) return {1.0f, 1.0f};
    const float by = fresh ? -INFINITY : row.m - up;                                 // <= 0
    const int keep = fresh ? 100000 : row.off + (int)fminf(-by, 1000.0f);
    const int set = mp == -INFINITY ? 100000 : kUp + (int)floorf(fminf(up - mp, 1000.0f));
    const int off = fresh && mp == -INFINITY ? row.off : min(keep, set);
    const Moved f = {exp2_fast(by), exp2_fast(by + (float)(off - row.off))};
    row.m = up;
    row.off = off;
    row.l = mul2(row.l, pair2(f.l, f.l));
    return f;
}

// Brings the step's P of the parts before column c0 and, past the first step, O to moved references.
template <int D>
__device__ __forceinline__ void rescale(uint32_t s_tmem, uint32_t o_tmem, int c0, bool first, float by) {
    const uint32_t by2 = pack_f16(by, by);
#pragma unroll 1
    for (int c = 0; c < c0; c += 16) {
        uint32_t q[8];
        tmem_ld8(s_tmem + c / 2, q);
        tmem_ld_wait();
#pragma unroll
        for (int k = 0; k < 8; k++) asm volatile("mul.rn.f16x2 %0, %0, %1;" : "+r"(q[k]) : "r"(by2));
        tmem_st8(s_tmem + c / 2, q);
    }
    if (!first) {
        // the products up to the step before are complete: this step's S was issued after them
#pragma unroll 1
        for (int c = 0; c < D; c += 16) {
            uint32_t r[16];
            tmem_ld16(o_tmem + c, r);
            tmem_ld_wait();
#pragma unroll
            for (int k = 0; k < 16; k++) r[k] = __float_as_uint(__uint_as_float(r[k]) * by);
            tmem_st16(o_tmem + c, r);
        }
    }
    tmem_st_wait();
}

// P = 2^(f S - m + e) of the step as fp16 into the tensor memory of S (columns that are read already), with
// e = ve + off for all tokens.  f0, f1 >= 0 scale the pages' scores.  MASK: the row sees the step's first
// `seen` tokens, of pages that are there.  References lag behind the rows' maxima: they move only when 32 P
// add up to more than fp16 holds, or when a row sees its first token.
template <int D, bool MASK>
__device__ __forceinline__ void step_probs(uint32_t s_tmem, uint32_t o_tmem, float f0, float f1, int ve, int seen, int there, bool first,
                                           RowSums &row) {
    uint32_t buf[2][32];
    tmem_ld32(s_tmem, buf[0]);
    // P is 2^(x + nm), and 2^(x - m) is P times un
    float nm = row.m == -INFINITY ? 0.0f : (float)(ve + row.off) - row.m;
    float un = __int_as_float((127 - min(ve + row.off, 126)) << 23);
#pragma unroll 1
    for (int page = 0; page < 2; page++) {
        const float fp = page ? f1 : f0;
        const f2 f = pair2(fp, fp);
#pragma unroll
        for (int half = 0; half < 2; half++) {
            const int c0 = 64 * page + 32 * half;
            uint32_t(&r)[32] = buf[half];
            tmem_ld_wait32(r);
            if (half == 0) tmem_ld32(s_tmem + c0 + 32, buf[1]);  // behind this part's arithmetic
            else if (page == 0) tmem_ld32(s_tmem + c0 + 32, buf[0]);
            const int n = MASK ? (there >> page & 1 ? seen - c0 : 0) : 32;
            uint32_t pk[16];
            f2 sum;
            for (bool moved = false;; moved = true) {
                f2 sum2[2] = {pair2(0.0f, 0.0f), pair2(0.0f, 0.0f)};
#pragma unroll
                for (int i = 0; i < 32; i += 2) {
                    float a, b;
                    split2(fma2(f, pair2u(r[i], r[i + 1]), pair2(nm, nm)), a, b);
                    a = exp2_fast(a);
                    b = exp2_fast(b);
                    if (MASK) {
                        a = i < n ? a : 0.0f;
                        b = i + 1 < n ? b : 0.0f;
                    }
                    sum2[(i / 2) & 1] = add2(sum2[(i / 2) & 1], pair2(a, b));
                    pk[i / 2] = pack_f16(a, b);
                }
                sum = add2(sum2[0], sum2[1]);
                float a, b;
                split2(sum, a, b);
                // once is enough (a row of nothing but NaN has no reference after it either)
                if (moved || !__any_sync(0xFFFFFFFFu, a + b > 60000.0f || (row.m == -INFINITY && n > 0))) break;
                float mx = -INFINITY;
#pragma unroll
                for (int i = 0; i < 32; i++) mx = fmaxf(mx, i < n ? __uint_as_float(r[i]) : -INFINITY);
                mx = mx == -INFINITY ? mx : fp * mx;  // 0 * -inf would be NaN
                const Moved by = move_row(mx, mx + (float)ve, row);
                tmem_ld_wait32(buf[half ^ 1]);
                rescale<D>(s_tmem, o_tmem, c0, first, by.o);
                nm = row.m == -INFINITY ? 0.0f : (float)(ve + row.off) - row.m;
                un = __int_as_float((127 - min(ve + row.off, 126)) << 23);
            }
            row.l = fma2(sum, pair2(un, un), row.l);
            tmem_st16(s_tmem + c0 / 2, pk);
        }
    }
}

// The same where tokens have powers of their own (key_of, value_of, with kOffset added; kBad: a value of NaN)
// or the step's power is far from the row's: one exponential of every score for l, another with its value's power
// for P.  Rare, so a call, out of the usual step's way in the instruction cache (inlined: prompts of 2,048 47.2 us
// against 47.0, chunks of 4,096 at 16,384 3.74 ms against 3.69).  A prompt of 2,048 with one such step for each
// 256 rows takes 55 us, with all of them 96.
template <int D>
__device__ __noinline__ RowSums step_apart(uint32_t s_tmem, uint32_t o_tmem, float row_scale, const StepInfo &info, int seen,
                                           bool first, RowSums row) {
    const int lane = threadIdx.x & 31;
#pragma unroll 1
    for (int c0 = 0; c0 < kKeys; c0 += 32) {
        uint32_t r[32];
        float e[32];
        tmem_ld32(s_tmem + c0, r);
        const int page = info.key_exp[c0 / 64], v = info.value_exp & kApart ? info.value_of[c0 + lane] : info.value_exp;
        const unsigned bad = __ballot_sync(0xFFFFFFFFu, v == kBad);
#pragma unroll
        for (int i = 0; i < 32; i++) e[i] = __shfl_sync(0xFFFFFFFFu, (float)(v - kOffset), i);
        tmem_ld_wait32(r);
        float f = row_scale * __int_as_float(((page & (kApart - 1)) - kOffset + 127) << 23);
        if (page & kApart) {
            // a token's power is a float's up to 2^127: 2^7 of it goes to the row's factor
            f = row_scale * 128.0f;
            const float own = __int_as_float((info.key_of[c0 + lane] - kOffset - 7 + 127) << 23);
#pragma unroll
            for (int i = 0; i < 32; i++) r[i] = __float_as_uint(__uint_as_float(r[i]) * __shfl_sync(0xFFFFFFFFu, own, i));
        }
        const int n = info.there >> (c0 / 64) & 1 ? seen - c0 : 0;
        float mx = -INFINITY, mp = -INFINITY;   // largest score, largest score of a P
#pragma unroll
        for (int i = 0; i < 32; i++) {
            const float x = i < n ? f * __uint_as_float(r[i]) : -INFINITY;
            mx = fmaxf(mx, x);
            mp = fmaxf(mp, x + e[i]);
        }
        const bool far = mx > row.m + 8.0f || mp - row.m + (float)row.off > 14.0f;
        if (__any_sync(0xFFFFFFFFu, far)) {
            const Moved by = far ? move_row(mx, mp, row) : Moved{1.0f, 1.0f};
            rescale<D>(s_tmem, o_tmem, c0, first, by.o);
        }
        const float nm = row.m == -INFINITY ? 0.0f : -row.m, np = nm + (float)row.off;
        float sum[2] = {0.0f, 0.0f};
        uint32_t pk[16];
#pragma unroll
        for (int i = 0; i < 32; i += 2) {
            float p[2];
#pragma unroll
            for (int k = 0; k < 2; k++) {
                const float x = __uint_as_float(r[i + k]), one = exp2_fast(f * x + nm);
                p[k] = exp2_fast(f * x + np + e[i + k]);
                sum[k] += i + k < n ? one : 0.0f;
                p[k] = i + k < n ? p[k] : 0.0f;
            }
            pk[i / 2] = pack_f16(p[0], p[1]);
        }
        if (n > 0 && (bad & (n >= 32 ? 0xFFFFFFFFu : (1u << n) - 1u)) != 0) sum[0] = __int_as_float(0x7FFFFFFF);
        row.l = add2(row.l, pair2(sum[0], sum[1]));
        tmem_st16(s_tmem + c0 / 2, pk);
    }
    return row;
}

template <int D>
__global__ void __launch_bounds__(kTileThreads, 1) attn_tile_kernel(const __grid_constant__ AttnParams p) {
    using T = Tile<D>;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t *sq = smem, *sk = sq + 2 * T::kQ, *sv = sk + 2 * T::kOp, *raw = sv + 2 * T::kOp;
    TileBars *bar = reinterpret_cast<TileBars *>(raw + 4 * T::kPage);
    static_assert(sizeof(TileBars) <= T::kBars && T::kPage % 16 == 0, "barriers");
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
    const int steps = keys > 0 ? (keys - 1) / kKeys + 1 : 0;
    const long long limit = p.wait_limit;
    if (smem_u32(smem) & 1023) {  // the swizzled operands need it
        if (threadIdx.x == 0) atomicCAS(p.err, 0u, (unsigned int)SHERRY_ERR_UNSUPPORTED);
        return;
    }

    if (threadIdx.x == 0) {
        mbar_init(&bar->q_full, 8);
        for (int i = 0; i < 2; i++) {
            mbar_init(&bar->k_full[i], 2);
            mbar_init(&bar->v_full[i], 2);
            mbar_init(&bar->k_empty[i], 1);
            mbar_init(&bar->v_empty[i], 1);
            mbar_init(&bar->s_full[i], 1);
            mbar_init(&bar->p_full[i], 4);
            mbar_init(&bar->o_full[i], 1);
            mbar_init(&bar->raw_full[i], 1);
            mbar_init(&bar->raw_empty[i], 4);
        }
        for (int i = 0; i < kInfoSlots; i++) mbar_init(&bar->info_full[i], 4);
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
        regs_up<176>();
        const int i = warp >> 2, r = threadIdx.x & 127;      // tile, row of the tile
        const int rw = row0 + i * kRowsTile + r;
        const bool live = rw < nrow;
        const int last = live ? pos0 + rw / p.g : kAllSeen;  // a row past the end sees all and is dropped
        const int lo_row = row0 + i * kRowsTile;
        const int last_min = lo_row < nrow ? pos0 + lo_row / p.g : kAllSeen;
        // queries to shared memory (elements of each eight in the order 0 4 1 5 2 6 3 7, as the codes
        // come out of their words), K-major with 128-byte rows swizzled, as fp16 of q 2^-qe
        float row_scale;
        {
            const uint16_t *src = p.q + (long long)(w.first + rw / p.g) * p.q_stride + (long long)(h * p.g + rw % p.g) * D;
            uint8_t *dst = sq + i * T::kQ + r * 128;
            float most = 0.0f;
#pragma unroll 4
            for (int c = 0; c < D / 8; c++) {
                uint4 u = make_uint4(0, 0, 0, 0);
                if (live) u = *reinterpret_cast<const uint4 *>(src + 8 * c);
                const uint32_t e[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                for (int k = 0; k < 4; k++)
                    most = fmaxf(most, fmaxf(fabsf(__uint_as_float(e[k] << 16)), fabsf(__uint_as_float(e[k] & 0xFFFF0000u))));
            }
            const int qe = max((int)(__float_as_uint(fminf(most, 3e38f)) >> 23) - 127 - 7, -120);  // the largest below 2^8
            const float down = copysignf(pow2(-qe), p.scale2);  // scores come out with the scale's sign
            row_scale = fabsf(p.scale2) * pow2(qe);
#pragma unroll 4
            for (int c = 0; c < D / 8; c++) {
                uint4 u = make_uint4(0, 0, 0, 0);
                if (live) u = *reinterpret_cast<const uint4 *>(src + 8 * c);
                const uint32_t lo[2] = {u.x, u.y}, hi[2] = {u.z, u.w};
                uint32_t v[4];
#pragma unroll
                for (int k = 0; k < 2; k++) {
                    v[2 * k] = pack_f16(__uint_as_float(lo[k] << 16) * down, __uint_as_float(hi[k] << 16) * down);
                    v[2 * k + 1] = pack_f16(__uint_as_float(lo[k] & 0xFFFF0000u) * down, __uint_as_float(hi[k] & 0xFFFF0000u) * down);
                }
                *reinterpret_cast<uint4 *>(dst + (c / 8) * (kRowsTile * 128) + (((c & 7) ^ (r & 7)) << 4)) =
                    make_uint4(v[0], v[1], v[2], v[3]);
            }
        }
        fence_proxy_async_smem();
        warp_arrive(&bar->q_full);
        const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t s_tmem = tmem + lane_base + i * kKeys;
        const uint32_t o_tmem = tmem + lane_base + 2 * kKeys + i * D;
        RowSums row = {-INFINITY, 0, pair2(0.0f, 0.0f)};
        bool dead = false;
        int slot = 0;
        uint32_t lap = 0;
        for (int j = 0; j < steps; j++) {
            if (!warp_wait(&bar->info_full[slot], lap, abort, p.err, limit) ||
                !warp_wait(&bar->s_full[i], j & 1, abort, p.err, limit)) {
                dead = true;
                break;
            }
            tc_fence_after();
            const StepInfo &info = bar->info[slot];
            if (++slot == kInfoSlots) slot = 0, lap ^= 1;
            const int4 what = *reinterpret_cast<const int4 *>(info.key_exp);  // key_exp, value_exp, there
            const int there = what.w, t0 = j * kKeys;
            const int seen = min(max(last - t0 + 1, 0), kKeys);
            const int k0 = what.x, k1 = what.y, v = what.z, ve = v - kOffset;
            // (token by token too where a row's P would all be below 2^-40 or above 2^100)
            const bool far = row.m != -INFINITY && (unsigned)(ve + row.off + 40) > 140u;
            if (!__any_sync(0xFFFFFFFFu, far || (k0 | k1 | v) & kApart)) {
                const float f0 = row_scale * __int_as_float((k0 - kOffset + 127) << 23);
                const float f1 = row_scale * __int_as_float((k1 - kOffset + 127) << 23);
                if (there == 3 && t0 + kKeys - 1 <= last_min) step_probs<D, false>(s_tmem, o_tmem, f0, f1, ve, seen, there, j == 0, row);
                else step_probs<D, true>(s_tmem, o_tmem, f0, f1, ve, seen, there, j == 0, row);
            } else {
                row = step_apart<D>(s_tmem, o_tmem, row_scale, info, seen, j == 0, row);
            }
            tmem_st_wait();
            tc_fence_before();
            warp_arrive(&bar->p_full[i]);
        }
        if (!dead && steps > 0)
            dead = !warp_wait(&bar->o_full[i], 0, abort, p.err, limit);
        if (!dead) {
            tc_fence_after();
            float l, l1;
            split2(row.l, l, l1);
            l += l1;
            // out = O 2^-off / l, the power in two halves (values near the ends of fp32's range)
            const float half = pow2(-row.off >> 1), inv = l == 0.0f ? 0.0f : pow2(-row.off - (-row.off >> 1)) / l;
            uint16_t *dst = p.out + (long long)(w.first + rw / p.g) * p.out_stride + (long long)(h * p.g + rw % p.g) * D;
#pragma unroll 1
            for (int c0 = 0; c0 < D; c0 += 32) {
                uint32_t o[32];
                if (steps > 0) {
                    tmem_ld32(o_tmem + c0, o);
                    tmem_ld_wait32(o);
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
                            u[e] = pack_bf16(__uint_as_float(o[k + 2 * e]) * half * inv, __uint_as_float(o[k + 2 * e + 1]) * half * inv);
                        *reinterpret_cast<uint4 *>(dst + c0 + k) = make_uint4(u[0], u[1], u[2], u[3]);
                    }
                }
            }
        }
    } else if (warp < 12) {
        regs_down<96>();
        if (warp < 10) {
            // ---------------- keys: a warp per page, two tokens per thread ----------------
            const int k = warp - 8;
            for (int j = 0, slot = 0; j < steps; j++) {
                const int s = j & 1;
                if (!warp_wait(&bar->raw_full[s], (j >> 1) & 1, abort, p.err, limit)) break;
                const uint8_t *blk = raw + (2 * s + k) * T::kPage;
                const int there = bar->there[s];
                // tokens past the last that a row of this CTA sees may hold anything: they count as zeros
                const int in = there >> k & 1 ? keys - j * kKeys - k * SHERRY_KV4_PAGE : 0;
                const uint32_t *pairs = reinterpret_cast<const uint32_t *>(blk + Kv4<D>::kCodes);
                const uint32_t sm[2] = {lane < in ? pairs[lane] : 0u, lane + 32 < in ? pairs[lane + 32] : 0u};
                const float size[2] = {pair_most(sm[0]), pair_most(sm[1])};
                auto some = [](float v) { return v == 0.0f ? INFINITY : v; };
                int shared = shared_exp(fminf(some(size[0]), some(size[1])), fmaxf(size[0], size[1]));
                if (shared > kOffset + kMostExp) shared |= kApart;
                const int e = (shared & (kApart - 1)) - kOffset;
                int own[2] = {e, e};
                if (!warp_wait(&bar->k_empty[s], ((j >> 1) & 1) ^ 1, abort, p.err, limit)) break;
                // The slot is free: the products of step j - 2 are complete, and their last half was issued after the
                // softmax of step j - 3.
                StepInfo &info = bar->info[slot];
                if (lane == 0) {
                    info.key_exp[k] = shared;
                    if (k == 0) info.there = there;
                }
                if (shared & kApart) {
                    own[0] = exp_for(size[0]), own[1] = exp_for(size[1]);
                    info.key_of[SHERRY_KV4_PAGE * k + lane] = (uint8_t)(own[0] + kOffset);
                    info.key_of[SHERRY_KV4_PAGE * k + lane + 32] = (uint8_t)(own[1] + kOffset);
                }
                warp_arrive(&bar->info_full[slot]);
                if (++slot == kInfoSlots) slot = 0;
#pragma unroll 1
                for (int t = 0; t < 2; t++) {
                    const float down = pow2(-own[t]);
                    const int row = lane + 32 * t, tok = SHERRY_KV4_PAGE * k + row;
                    const float st = kv4_step(sm[t]) * down, lo = kv4_low(sm[t]) * down;
                    const uint32_t s0 = pack_f16(st * 16777216.0f, st * 16777216.0f), s1 = pack_f16(st * 1048576.0f, st * 1048576.0f);
                    const uint32_t m2 = pack_f16(lo, lo);
                    const uint8_t *src = blk + row * Kv4<D>::kRow;
                    uint8_t *dst = sk + s * T::kOp + tok * 128;
#pragma unroll 2
                    for (int q = 0; q < D / 32; q++) {
                        // 16-byte pieces of a row in an order that keeps eight rows out of each other's banks
                        const int qq = (q + (D == 128 ? row >> 1 : row >> 2)) & (D / 32 - 1);
                        uint4 u = *reinterpret_cast<const uint4 *>(src + 16 * qq);
                        if (row >= in) u = make_uint4(0, 0, 0, 0);
                        const uint32_t x[4] = {u.x, u.y, u.z, u.w};
                        uint8_t *half = dst + (qq / 2) * (kKeys * 128);
#pragma unroll
                        for (int i = 0; i < 4; i++) {
                            const int c = (4 * qq + i) & 7;  // 8-element chunk of the 128-byte row
                            const uint32_t y = x[i] >> 8;
                            *reinterpret_cast<uint4 *>(half + ((c ^ (tok & 7)) << 4)) =
                                make_uint4(value_pair<0x000F000F>(x[i], s0, m2), value_pair<0x00F000F0>(x[i], s1, m2),
                                           value_pair<0x000F000F>(y, s0, m2), value_pair<0x00F000F0>(y, s1, m2));
                        }
                    }
                }
                fence_proxy_async_smem();
                warp_arrive(&bar->k_full[s]);
                warp_arrive(&bar->raw_empty[s]);
            }
        } else {
            // ---------------- values: a warp per page, eight tokens per thread, transposed ----------------
            const int k = warp - 10;
            const int grp = lane & 7, qd = lane >> 3;  // tokens 8 grp ... of the page, word qd of each four
            const int odd = grp & 1;                   // these read the tokens of a pair in the other order, for the banks
            for (int j = 0, slot = 0; j < steps; j++) {
                const int s = j & 1;
                if (!warp_wait(&bar->raw_full[s], (j >> 1) & 1, abort, p.err, limit)) break;
                const int there = bar->there[s];
                const uint8_t *blk = raw + 2 * s * T::kPage + Kv4<D>::kBlock;  // the first page's values
                uint32_t pair[4];                                              // of tokens lane + 32 i of the step
                float least = INFINITY, most = 0.0f;
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const bool in = (there >> (i / 2) & 1) && j * kKeys + lane + 32 * i < keys;
                    pair[i] = in ? reinterpret_cast<const uint32_t *>(blk + (i / 2) * T::kPage + Kv4<D>::kCodes)[lane + 32 * (i & 1)] : 0u;
                    const float size = pair_most(pair[i]);
                    least = fminf(least, size != 0.0f ? size : pair_bad(pair[i]) ? 0.0f : INFINITY);
                    most = fmaxf(most, size);
                }
                const int shared = shared_exp(least, most);
                const int ve = (shared & (kApart - 1)) - kOffset;
                const bool apart = shared & kApart;
                blk += k * T::kPage;
                const int in = there >> k & 1 ? keys - j * kKeys - k * SHERRY_KV4_PAGE - 8 * grp : 0;  // tokens of the eight that are there
                uint32_t s0[4], s1[4], m2[4];
                const float down = pow2(-ve);
#pragma unroll
                for (int t = 0; t < 4; t++) {
                    const uint2 u = *reinterpret_cast<const uint2 *>(blk + Kv4<D>::kCodes + 4 * (8 * grp + 2 * t));
                    uint32_t a = 2 * t < in ? u.x : 0u, b = 2 * t + 1 < in ? u.y : 0u;
                    float da = down, db = down;
                    if (apart) {
                        if (pair_bad(a)) a = 0u;
                        if (pair_bad(b)) b = 0u;
                        da = pow2(-exp_for(pair_most(a)));
                        db = pow2(-exp_for(pair_most(b)));
                    }
                    const float sa = kv4_step(a) * da, sb = kv4_step(b) * db;
                    s0[t] = pack_f16(sa * 16777216.0f, sb * 16777216.0f);
                    s1[t] = pack_f16(sa * 1048576.0f, sb * 1048576.0f);
                    m2[t] = pack_f16(kv4_low(a) * da, kv4_low(b) * db);
                }
                if (!warp_wait(&bar->v_empty[s], ((j >> 1) & 1) ^ 1, abort, p.err, limit)) break;
                // The slot is free: the products of step j - 2 are complete, and they were issued after its softmax.
                StepInfo &info = bar->info[slot];
                if (k == 0) {
                    if (lane == 0) info.value_exp = shared;
                    if (apart) {
#pragma unroll
                        for (int i = 0; i < 4; i++)
                            info.value_of[lane + 32 * i] = (uint8_t)(pair_bad(pair[i]) ? kBad : kOffset + exp_for(pair_most(pair[i])));
                    }
                }
                warp_arrive(&bar->info_full[slot]);
                if (++slot == kInfoSlots) slot = 0;
                const uint32_t sel_lo = odd ? 0x1054u : 0x5410u, sel_hi = odd ? 0x3276u : 0x7632u;
                uint8_t *dst = sv + s * T::kOp + k * (D * 128);
                const uint8_t *src = blk + 8 * grp * Kv4<D>::kRow;
#pragma unroll 1
                for (int e = 0; e < D / 32; e++) {
                    const int word = 4 * ((e + (grp >> 1)) & (D / 32 - 1)) + qd;
                    uint32_t lo[4], hi[4];
#pragma unroll
                    for (int t = 0; t < 4; t++) {
                        const uint32_t a = *reinterpret_cast<const uint32_t *>(src + (2 * t + odd) * Kv4<D>::kRow + 4 * word);
                        const uint32_t b = *reinterpret_cast<const uint32_t *>(src + (2 * t + 1 - odd) * Kv4<D>::kRow + 4 * word);
                        lo[t] = prmt(a, b, sel_lo);
                        hi[t] = prmt(a, b, sel_hi);
                    }
                    uint8_t *row = dst + 8 * word * 128;
#pragma unroll
                    for (int i = 0; i < 8; i += 2) {
                        uint32_t y[4];
#pragma unroll
                        for (int t = 0; t < 4; t++) y[t] = (i < 4 ? lo[t] : hi[t]) >> (4 * (i & 2));
                        *reinterpret_cast<uint4 *>(row + i * 128 + ((grp ^ i) << 4)) =
                            make_uint4(value_pair<0x000F000F>(y[0], s0[0], m2[0]), value_pair<0x000F000F>(y[1], s0[1], m2[1]),
                                       value_pair<0x000F000F>(y[2], s0[2], m2[2]), value_pair<0x000F000F>(y[3], s0[3], m2[3]));
                        *reinterpret_cast<uint4 *>(row + (i + 1) * 128 + ((grp ^ (i + 1)) << 4)) =
                            make_uint4(value_pair<0x00F000F0>(y[0], s1[0], m2[0]), value_pair<0x00F000F0>(y[1], s1[1], m2[1]),
                                       value_pair<0x00F000F0>(y[2], s1[2], m2[2]), value_pair<0x00F000F0>(y[3], s1[3], m2[3]));
                    }
                }
                fence_proxy_async_smem();
                warp_arrive(&bar->v_full[s]);
                warp_arrive(&bar->raw_empty[s]);
        }
        }
    } else {
        regs_down<64>();
        if (warp == 13) {
            // ---------------- pages ----------------
            if (lane == 0) {
                int it = 0;
                for (; it < steps; it++) {
                    const int s = it & 1;
                    int page[2], there = 0;
#pragma unroll
                    for (int k = 0; k < 2; k++) {
                        const int t0 = it * kKeys + k * SHERRY_KV4_PAGE;
                        page[k] = t0 < keys ? __ldg(p.c.table + (long long)w.b * p.c.table_stride + t0 / SHERRY_KV4_PAGE) : -1;
                        if (page[k] >= 0 && page[k] < p.c.pages) there |= 1 << k;
                        else if (t0 < keys) atomicCAS(p.err, 0u, (unsigned int)SHERRY_ERR_INDEX);
                    }
                    if (!mbar_wait(&bar->raw_empty[s], ((it >> 1) & 1) ^ 1, abort, p.err, limit)) break;
                    bar->there[s] = there;
                    if (there == 0) {
                        mbar_arrive(&bar->raw_full[s]);
                        continue;
                    }
                    mbar_arrive_expect_tx(&bar->raw_full[s], (there == 3 ? 2 : 1) * T::kPage);
#pragma unroll
                    for (int k = 0; k < 2; k++)
                        if (there >> k & 1)
                            bulk_load(smem_u32(raw + (2 * s + k) * T::kPage), kv4_block<D>(p.c, page[k], h, 0), T::kPage, &bar->raw_full[s]);
                }
                // every copy lands before shared memory is released
                volatile int no_abort = 0;
                for (int j = it < 2 ? 0 : it - 2; j < it; j++) mbar_wait(&bar->raw_full[j & 1], (j >> 1) & 1, &no_abort, p.err, kDrainLimit);
            }
        } else if (warp == 12 && steps > 0) {
            // ---------------- products ----------------
            // The whole warp walks and waits, one elected lane issues.
            const uint32_t q_lo = (smem_u32(sq) >> 4) | (1u << 16), k_lo = (smem_u32(sk) >> 4) | (1u << 16),
                           v_lo = (smem_u32(sv) >> 4) | (1u << 16);
            auto scores = [&](int i, int s) {  // S_i = Q_i K^T
                tc_fence_after();
                if (elect_one()) {
                    mma_ss_all<0, D / 16, 128>(tmem + i * kKeys, q_lo + i * (T::kQ >> 4), k_lo + s * (T::kOp >> 4), kIdesc<kKeys>);
                    umma_commit(&bar->s_full[i]);
                }
                __syncwarp();
            };
            bool ok = warp_wait(&bar->q_full, 0, abort, p.err, limit) && warp_wait(&bar->k_full[0], 0, abort, p.err, limit);
            const bool issued = ok;
            if (ok) {
                scores(0, 0);
                scores(1, 0);
                if (elect_one()) umma_commit(&bar->k_empty[0]);
            }
            for (int j = 0; ok && j < steps; j++) {
                const int s = j & 1, ph = (j >> 1) & 1;
                ok = warp_wait(&bar->v_full[s], ph, abort, p.err, limit);
#pragma unroll
                for (int i = 0; i < 2; i++) {
                    if (!ok) break;
                    ok = warp_wait(&bar->p_full[i], j & 1, abort, p.err, limit);
                    if (!ok) break;
                    tc_fence_after();
                    if (elect_one()) {
                        mma_ts_all<0, kKeys / 16, D>(tmem + 2 * kKeys + i * D, tmem + i * kKeys, v_lo + s * (T::kOp >> 4),
                                                     kIdesc<D>, j != 0);
                        if (j + 1 == steps) umma_commit(&bar->o_full[i]);
                    }
                    __syncwarp();
                    if (j + 1 < steps) {
                        if (i == 0) {
                            ok = warp_wait(&bar->k_full[s ^ 1], ((j + 1) >> 1) & 1, abort, p.err, limit);
                            if (!ok) break;
                        }
                        scores(i, s ^ 1);
                    }
                }
                if (ok && elect_one()) {
                    umma_commit(&bar->v_empty[s]);
                    if (j + 1 < steps) umma_commit(&bar->k_empty[s ^ 1]);
                }
                __syncwarp();
            }
            // every issued product is done before tensor and shared memory are released
            if (issued) {
                if (elect_one()) umma_commit(&bar->drain);
                __syncwarp();
                volatile int no_abort = 0;
                mbar_wait(&bar->drain, 0, &no_abort, p.err, kDrainLimit);
            }
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
