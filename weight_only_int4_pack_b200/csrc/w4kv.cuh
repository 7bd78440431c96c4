// w4kv.cuh -- what the kernels of the quantized key/value cache share: the
// cache and batch descriptions they get, the search of a row's sequence, and
// the page lookup with its bounds.
#pragma once

#include "w4_half.cuh"
#include "w4_internal.cuh"
#include "w4kv.h"

namespace w4 {
namespace kv {

struct Cache {
    uint8_t *k, *v;
    float *ks, *vs;
    int64_t pages;
    int page, heads, row_bytes;
};

struct Batch {
    const int *table;
    int64_t stride;
    int width;  // pages per sequence the table has room for
    const int *lens, *cu;
    int n;
};

constexpr unsigned kStatusBounds = 2u;  // the bit w4_device_status reports as W4_ERR_BOUNDS

// Sequence of row t (cu[b] <= t < cu[b + 1]), or -1 when it belongs to none.
// All 32 lanes call it with the same t; each step cuts the range by 32.
__device__ __forceinline__ int find_sequence(const int *__restrict__ cu, int n_seq, int t, int lane) {
    int lo = 0, n = n_seq + 1;
    while (n > 32) {
        const int step = (n + 31) / 32, i = lane * step;
        const unsigned le = __ballot_sync(0xffffffffu, i < n && __ldg(cu + lo + i) <= t);
        if (le == 0) return -1;
        const int c = __popc(le) - 1;
        lo += c * step;
        n = min(step, n - c * step);
    }
    const unsigned le = __ballot_sync(0xffffffffu, lane < n && __ldg(cu + lo + lane) <= t);
    const int b = lo + __popc(le) - 1;
    if (b < 0 || b >= n_seq) return -1;
    return __ldg(cu + b) <= t && t < __ldg(cu + b + 1) ? b : -1;
}

// Row index (token of head 0; head h is h * page further) of position p of
// sequence b in the code and scale arrays, or -1 when p or its page number is
// out of range.
__device__ __forceinline__ int64_t row_of(const Cache &c, const Batch &bt, int b, int p) {
    if (p < 0) return -1;
    const int pg = p / c.page;
    if (pg >= bt.width) return -1;
    const int id = __ldg(bt.table + b * bt.stride + pg);
    if (id < 0 || id >= c.pages) return -1;
    return int64_t(id) * c.heads * c.page + (p - pg * c.page);
}

// Scale and zero point of an INT4 row's scale word.
__device__ __forceinline__ float int4_scale(uint32_t w) { return __uint_as_float(w & ~15u); }

// ---- host side ----
// Checks what the entry points share; fills the kernel-side descriptions.
int check_cache(const char *fn, const w4kv_cache *c, Cache *out);
int check_batch(const char *fn, const w4kv_batch *b, const w4kv_cache *c, Batch *out);
// A [rows][heads][dim] 16-bit operand: pointer, strides; outputs must not overlap.
int check_rows(const char *fn, const void *p, int64_t rows, int heads, int dim, int64_t row_stride,
               int64_t head_stride, bool output);

}  // namespace kv
}  // namespace w4
