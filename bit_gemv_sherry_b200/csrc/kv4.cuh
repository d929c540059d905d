// kv4.cuh -- the 4-bit key/value cache as the kernels see it (internal).
#pragma once

#include "common.cuh"

namespace sherry {

// A sherry_kv4 in launch-parameter form.
struct Kv4View {
    uint8_t *cache;
    const int *table;   // [B][table_stride], `width` entries used
    const int *lens;    // [B]
    const int *cu;      // [B + 1], or null: one new token per sequence
    long long pages, table_stride;
    int H, width, B;
    int T;
};

template <int D>
struct Kv4 {
    static constexpr int kRow = D / 2;                         // code bytes of a token
    static constexpr int kCodes = SHERRY_KV4_PAGE * kRow;      // code bytes of a block
    static constexpr int kBlock = kCodes + SHERRY_KV4_PAGE * 4;  // + (step, low) pairs
};

// First bad index met by a kernel of the cache or the attention (sherry_device_error).
unsigned int *kv4_error_address();

// bf16 pair (step in the low half, low end in the high half).
__device__ __forceinline__ float kv4_step(uint32_t sm) { return __uint_as_float(sm << 16); }
__device__ __forceinline__ float kv4_low(uint32_t sm) { return __uint_as_float(sm & 0xFFFF0000u); }

// Rows [first, first + count) of sequence b.  Offsets are clamped to [0, T], so a malformed
// cu_q reaches no row outside the tensors.
__device__ __forceinline__ void kv4_rows(const Kv4View &c, int b, int &first, int &count) {
    if (!c.cu) {
        first = b;
        count = b < c.T ? 1 : 0;
        return;
    }
    const int a = min(max(__ldg(c.cu + b), 0), c.T), e = min(max(__ldg(c.cu + b + 1), 0), c.T);
    first = a;
    count = max(e - a, 0);
}

// The sequence of row t and the row's position in it: false for rows behind the last
// sequence.  A position is negative where the sequence is shorter than its new rows.
__device__ __forceinline__ bool kv4_find(const Kv4View &c, int t, int &b, int &pos) {
    if (!c.cu) {
        if (t >= c.B) return false;
        b = t;
        pos = max(__ldg(c.lens + t), 0) - 1;
        return true;
    }
    int lo = 0, hi = c.B;  // the last b with cu[b] <= t
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(c.cu + mid + 1) <= t) lo = mid + 1;
        else hi = mid;
    }
    if (lo >= c.B) return false;
    int first, count;
    kv4_rows(c, lo, first, count);
    if (t < first || t >= first + count) return false;
    b = lo;
    pos = max(__ldg(c.lens + lo), 0) - count + (t - first);
    return true;
}

// Page of position `pos` of sequence b, or -1 (recorded) where the table names none.
__device__ __forceinline__ int kv4_page(const Kv4View &c, int b, int pos, unsigned int *err) {
    const int i = pos / SHERRY_KV4_PAGE;
    const int p = i < c.width ? __ldg(c.table + (long long)b * c.table_stride + i) : -1;
    if (p >= 0 && p < c.pages) return p;
    atomicCAS(err, 0u, (unsigned int)SHERRY_ERR_INDEX);
    return -1;
}

template <int D>
__device__ __forceinline__ uint8_t *kv4_block(const Kv4View &c, int page, int h, int kv) {
    return c.cache + (((long long)page * c.H + h) * 2 + kv) * Kv4<D>::kBlock;
}

// Host: checks shared by the calls that take a sherry_kv4.
sherry_status kv4_check(const sherry_kv4 *c);
Kv4View kv4_view(const sherry_kv4 *c);

}  // namespace sherry
