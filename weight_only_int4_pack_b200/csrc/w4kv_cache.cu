// w4kv_cache.cu -- w4kv_append and w4kv_read: rows of keys and values into the
// quantized paged cache and back (formats and layout: include/w4kv.h).
//
// Both are one pass: 16-bit rows on one side, codes and scale words on the
// other, little arithmetic.  A warp serves one token: D / 8 lanes hold a row (8
// elements a lane, one 16-byte word), so a warp has 32 / (D / 8) rows of the
// token's 2 * kv_heads (keys, then values) at a time and up to kGroups such
// groups in flight.  The token's sequence is found once per warp by a 32-way
// search of cu_rows.
//
// What bounds them: the chain of dependent loads that starts every warp (cu_rows,
// length, page number, row) against the little it then moves, and for the append
// instruction issue.  Measured: appending 2048 tokens of 32 heads as INT4 and
// reading them back 38 us (85 MB), reading 12 sequences to 8192 (INT8, 357 MB)
// 81 us, 4.4 TB/s.  2 row groups a warp: 42 and 99 us (but 6.7 instead of 8.1 us
// for 64 single tokens); 8: 43 and 78; 16 elements a lane when reading: 79; the
// places of a block's tokens looked up first: 42 and 83.

#include <cuda_fp8.h>

#include "w4kv.cuh"

namespace w4 {
namespace kv {
namespace {

constexpr int kThreads = 256;
constexpr int kGroups = 4;  // row groups per warp, loaded together
constexpr float kTinyScale = 0x1p-120f;  // below it a scale's reciprocal is out of range

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}

// Codes of 8 consecutive 16-bit elements w (of a row of LPR lanes) and the row's scale word.
//
// The row's extremes are found on the 16-bit patterns (non-negative floats order
// like integers; NaN > infinity > finite), one shuffle per step.  Codes come from
// the reciprocal: x * fl(1 / s) is within 3 * 2^-24 of fl(x / s), relatively, so a
// code is the exact one unless the quotient lies that near a rounding border; a
// lane that holds such a one, and a scale whose reciprocal is out of range, takes
// the IEEE division.
template <int FMT, int LPR, int XT>
__device__ __forceinline__ uint2 encode8(const uint4 w, uint32_t *word) {
    constexpr uint32_t kInf = XT == W4_F16 ? 0x7C00u : 0x7F80u;
    constexpr float kMagic = 12582912.f;  // 1.5 * 2^23: adding it rounds to an integer, ties to even
    float x[8];
    widen8<XT>(w, x);
    if (FMT == W4KV_INT4) {
        // the largest element, and the largest of the negated ones, at least 0
        uint32_t p = __vmaxs2(__vmaxs2(w.x, w.y), __vmaxs2(w.z, w.w));
        uint32_t q = __vmaxs2(__vmaxs2(w.x ^ 0x80008000u, w.y ^ 0x80008000u),
                              __vmaxs2(w.z ^ 0x80008000u, w.w ^ 0x80008000u));
        uint32_t pq = __vmaxs2(__vmaxs2(__byte_perm(p, q, 0x5410), __byte_perm(p, q, 0x7632)), 0u);
#pragma unroll
        for (int o = LPR / 2; o; o >>= 1) pq = __vmaxu2(pq, __shfl_xor_sync(0xffffffffu, pq, o));
        const float hi = widen1<XT>(static_cast<uint16_t>(pq & 0xFFFFu));
        const float lo = -widen1<XT>(static_cast<uint16_t>(pq >> 16));
        const float range = __fsub_rn(hi, lo);
        const bool bad = (pq & 0xFFFFu) >= kInf || (pq >> 16) >= kInf ||
                         __float_as_uint(range) >= 0x7F800000u;
        const uint32_t sb = (__float_as_uint(__fdiv_rn(range, 15.f)) + 8u) & ~15u;
        if (bad || sb == 0) {
            *word = bad ? 0x7FC00000u : 0u;
            return make_uint2(0, 0);
        }
        const float s = __uint_as_float(sb);
        const float z = rintf(__fdiv_rn(-lo, s));
        *word = sb | static_cast<uint32_t>(z);
        const float r = __frcp_rn(s);
        bool near = s < kTinyScale;
        uint32_t c[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {  // 0 <= code by the choice of z; 15.5 rounds to 16
            const float v = fminf(fmaf(x[i], r, z), 15.f), m = v + kMagic;
            near = near || fabsf(v - (m - kMagic)) > 0.5f - 0x1p-18f;  // 3 * 2^-24 * 16 < 2^-18
            c[i] = __float_as_uint(m);
        }
        if (near) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                c[i] = static_cast<uint32_t>(
                    fminf(fmaxf(rintf(__fadd_rn(__fdiv_rn(x[i], s), z)), 0.f), 15.f));
        }
        // nibble of element i in the little-endian word: 0,4,1,5,2,6,3,7
        uint32_t u = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) u |= (c[i] & 15u) << (4 * ((i >> 1) + 4 * (i & 1)));
        return make_uint2(u, 0);
    }
    uint32_t t = __vmaxu2(__vmaxu2(w.x & 0x7FFF7FFFu, w.y & 0x7FFF7FFFu),
                          __vmaxu2(w.z & 0x7FFF7FFFu, w.w & 0x7FFF7FFFu));
#pragma unroll
    for (int o = LPR / 2; o; o >>= 1) t = __vmaxu2(t, __shfl_xor_sync(0xffffffffu, t, o));
    const uint32_t top = max(t & 0xFFFFu, t >> 16);
    const bool bad = top >= kInf;
    const float s = __fdiv_rn(widen1<XT>(static_cast<uint16_t>(top)), FMT == W4KV_INT8 ? 127.f : 448.f);
    if (bad || s == 0.f) {
        *word = bad ? 0x7FC00000u : 0u;
        return make_uint2(0, 0);
    }
    *word = __float_as_uint(s);
    const float rc = __frcp_rn(s);
    bool near = s < kTinyScale;
    uint2 r;
    if (FMT == W4KV_INT8) {
        uint32_t c[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {  // |x| <= amax: no code beyond 127
            const float v = x[i] * rc, m = v + kMagic;
            near = near || fabsf(v - (m - kMagic)) > 0.5f - 0x1p-15f;  // 3 * 2^-24 * 127 < 2^-15
            c[i] = __float_as_uint(m);
        }
        if (near) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                c[i] = static_cast<uint32_t>(static_cast<int>(
                    fminf(fmaxf(rintf(__fdiv_rn(x[i], s)), -127.f), 127.f)));
        }
        r.x = __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410);
        r.y = __byte_perm(__byte_perm(c[4], c[5], 0x0040), __byte_perm(c[6], c[7], 0x0040), 0x5410);
    } else {
        uint32_t c[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // a code is exact where both ends of the error agree
            const float v0 = x[2 * i] * rc, v1 = x[2 * i + 1] * rc;
            c[i] = e4m3x2(v0 * (1.f - 0x1p-22f), v1 * (1.f - 0x1p-22f));
            near = near || c[i] != e4m3x2(v0 * (1.f + 0x1p-22f), v1 * (1.f + 0x1p-22f));
        }
        if (near) {
#pragma unroll
            for (int i = 0; i < 4; ++i) c[i] = e4m3x2(__fdiv_rn(x[2 * i], s), __fdiv_rn(x[2 * i + 1], s));
        }
        r.x = c[0] | c[1] << 16;
        r.y = c[2] | c[3] << 16;
    }
    return r;
}

// Values of 8 consecutive codes.
template <int FMT>
__device__ __forceinline__ void decode8(const uint2 c, uint32_t word, float y[8]) {
    if (FMT == W4KV_INT4) {
        const float s = int4_scale(word);
        const int z = static_cast<int>(word & 15u);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int u = (c.x >> (4 * ((i >> 1) + 4 * (i & 1)))) & 15;
            y[i] = __fmul_rn(static_cast<float>(u - z), s);
        }
        return;
    }
    const float s = __uint_as_float(word);
    const uint32_t w[2] = {c.x, c.y};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t b = (w[i >> 2] >> (8 * (i & 3))) & 0xFFu;
        float q;
        if (FMT == W4KV_INT8) {
            q = static_cast<float>(static_cast<int8_t>(b));
        } else {
            const __half_raw h = __nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(b), __NV_E4M3);
            q = __half2float(*reinterpret_cast<const __half *>(&h));
        }
        y[i] = __fmul_rn(q, s);
    }
}

struct Rows {
    uint16_t *p[2];  // keys, values
    int64_t row[2], head[2];
};

// READ: cache -> 16-bit rows; else 16-bit rows -> cache.
template <int FMT, int D, int XT, bool READ>
__global__ void __launch_bounds__(kThreads) rows_kernel(const Cache c, const Batch bt, const Rows x,
                                                        int64_t items, int per_token,
                                                        unsigned *__restrict__ status) {
    constexpr int kLpr = D / 8, kRpw = 32 / kLpr;  // lanes per row, rows per warp
    constexpr int kCode = FMT == W4KV_INT4 ? 4 : 8;  // code bytes of a lane's 8 elements
    const int lane = threadIdx.x & 31;
    const int64_t item = (int64_t(blockIdx.x) * kThreads + threadIdx.x) >> 5;
    if (item >= items) return;  // whole warps
    const int t = static_cast<int>(item / per_token);
    const int g0 = static_cast<int>(item - int64_t(t) * per_token) * kGroups;
    const int b = find_sequence(bt.cu, bt.n, t, lane);
    if (b < 0) return;
    const int pos = __ldg(bt.lens + b) - (__ldg(bt.cu + b + 1) - t);
    const int64_t row0 = row_of(c, bt, b, pos);
    if (row0 < 0) {
        if (lane == 0) atomicOr(status, kStatusBounds);
        if (!READ) return;
    }
    const int e = (lane % kLpr) * 8;
    const int n = 2 * c.heads;
    uint4 w16[kGroups];
    uint2 code[kGroups];
    uint32_t word[kGroups];
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {  // all loads first
        const int u = (g0 + g) * kRpw + lane / kLpr;
        if (u < n) {
            const int kv = u >= c.heads, h = u - kv * c.heads;
            if (READ) {
                code[g] = make_uint2(0, 0);
                word[g] = 0;
                if (row0 >= 0) {
                    const int64_t r = row0 + int64_t(h) * c.page;
                    const uint8_t *p = (kv ? c.v : c.k) + r * c.row_bytes + (e / 8) * kCode;
                    if (kCode == 8) code[g] = __ldg(reinterpret_cast<const uint2 *>(p));
                    else code[g].x = __ldg(reinterpret_cast<const uint32_t *>(p));
                    word[g] = __ldg(reinterpret_cast<const uint32_t *>(kv ? c.vs : c.ks) + r);
                }
            } else {
                w16[g] = __ldg(reinterpret_cast<const uint4 *>(x.p[kv] + t * x.row[kv] +
                                                               h * x.head[kv] + e));
            }
        }
    }
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
        const int u = (g0 + g) * kRpw + lane / kLpr;
        const int kv = u >= c.heads, h = u - kv * c.heads;
        if (READ) {
            if (u >= n) continue;
            float f[8];
            decode8<FMT>(code[g], word[g], f);
            uint32_t o[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                o[i] = narrow1<XT>(f[2 * i]) | static_cast<uint32_t>(narrow1<XT>(f[2 * i + 1])) << 16;
            *reinterpret_cast<uint4 *>(x.p[kv] + t * x.row[kv] + h * x.head[kv] + e) =
                make_uint4(o[0], o[1], o[2], o[3]);
        } else {
            // every lane takes part in the row reductions; idle ones carry zeros
            if (u >= n) w16[g] = make_uint4(0, 0, 0, 0);
            uint32_t sw;
            const uint2 cd = encode8<FMT, kLpr, XT>(w16[g], &sw);
            if (u >= n) continue;
            const int64_t r = row0 + int64_t(h) * c.page;
            uint8_t *p = (kv ? c.v : c.k) + r * c.row_bytes + (e / 8) * kCode;
            if (kCode == 8) *reinterpret_cast<uint2 *>(p) = cd;
            else *reinterpret_cast<uint32_t *>(p) = cd.x;
            if (e == 0) reinterpret_cast<uint32_t *>(kv ? c.vs : c.ks)[r] = sw;
        }
    }
}

template <int FMT, int D, bool READ>
void launch_rows(const Cache &c, const Batch &b, const Rows &x, int xt, int64_t items, int per_token,
                 unsigned *status, cudaStream_t s) {
    const unsigned grid = static_cast<unsigned>((items * 32 + kThreads - 1) / kThreads);
    if (xt == W4_F16)
        rows_kernel<FMT, D, W4_F16, READ><<<grid, kThreads, 0, s>>>(c, b, x, items, per_token, status);
    else
        rows_kernel<FMT, D, W4_BF16, READ><<<grid, kThreads, 0, s>>>(c, b, x, items, per_token, status);
}

template <bool READ>
int rows_impl(const char *fn, const w4kv_cache *cache, const w4kv_batch *batch, const void *K,
              const void *V, int xt, int64_t rows, int64_t krs, int64_t khs, int64_t vrs,
              int64_t vhs, void *stream) {
    Cache c;
    Batch b;
    int st;
    if ((st = check_cache(fn, cache, &c)) != W4_OK) return st;
    if ((st = check_batch(fn, batch, cache, &b)) != W4_OK) return st;
    if (xt != W4_F16 && xt != W4_BF16)
        return set_error(W4_ERR_INVALID_ARG, fn, "the rows' type is not W4_F16 or W4_BF16");
    if (rows < 0 || rows > 0x7FFFFFFF)
        return set_error(W4_ERR_INVALID_ARG, fn, "rows must be 0 .. 2^31 - 1");
    if (rows == 0 || b.n == 0) return W4_OK;
    const int D = cache->head_dim;
    if ((st = check_rows(fn, K, rows, c.heads, D, krs, khs, READ)) != W4_OK) return st;
    if ((st = check_rows(fn, V, rows, c.heads, D, vrs, vhs, READ)) != W4_OK) return st;
    const int rpw = 32 / (D / 8);
    const int per_token = (2 * c.heads + rpw * kGroups - 1) / (rpw * kGroups);
    const int64_t items = rows * per_token;
    if (items > (int64_t(0x7FFFFFFF) - 1) * (kThreads / 32))
        return set_error(W4_ERR_INVALID_ARG, fn, "rows * kv_heads too large");
    unsigned *status = device_status_ptr();
    if (!status) return W4_ERR_CUDA;
    Rows x;
    x.p[0] = static_cast<uint16_t *>(const_cast<void *>(K));
    x.p[1] = static_cast<uint16_t *>(const_cast<void *>(V));
    x.row[0] = krs, x.row[1] = vrs, x.head[0] = khs, x.head[1] = vhs;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int key = cache->fmt * 2 + (D == 128);
    switch (key) {
        case W4KV_INT8 * 2: launch_rows<W4KV_INT8, 64, READ>(c, b, x, xt, items, per_token, status, s); break;
        case W4KV_INT8 * 2 + 1: launch_rows<W4KV_INT8, 128, READ>(c, b, x, xt, items, per_token, status, s); break;
        case W4KV_E4M3 * 2: launch_rows<W4KV_E4M3, 64, READ>(c, b, x, xt, items, per_token, status, s); break;
        case W4KV_E4M3 * 2 + 1: launch_rows<W4KV_E4M3, 128, READ>(c, b, x, xt, items, per_token, status, s); break;
        case W4KV_INT4 * 2: launch_rows<W4KV_INT4, 64, READ>(c, b, x, xt, items, per_token, status, s); break;
        default: launch_rows<W4KV_INT4, 128, READ>(c, b, x, xt, items, per_token, status, s); break;
    }
    return cuda_status(cudaGetLastError());
}

}  // namespace

int check_cache(const char *fn, const w4kv_cache *c, Cache *out) {
    if (!c) return set_error(W4_ERR_INVALID_ARG, fn, "null cache");
    if (c->fmt != W4KV_INT8 && c->fmt != W4KV_E4M3 && c->fmt != W4KV_INT4)
        return set_error(W4_ERR_INVALID_ARG, fn, "fmt is not W4KV_INT8, W4KV_E4M3 or W4KV_INT4");
    if (c->num_pages < 1 || c->num_pages > 0x7FFFFFFF)
        return set_error(W4_ERR_INVALID_ARG, fn, "num_pages must be 1 .. 2^31 - 1");
    if (c->kv_heads < 1 || c->kv_heads > 65535)
        return set_error(W4_ERR_INVALID_ARG, fn, "kv_heads must be 1 .. 65535");
    if (c->page_size < 1 || c->head_dim < 1)
        return set_error(W4_ERR_INVALID_ARG, fn, "page_size and head_dim must be positive");
    if (!c->k_codes || !c->v_codes || !c->k_scales || !c->v_scales)
        return set_error(W4_ERR_INVALID_ARG, fn, "null pointer in the cache");
    if (c->page_size % 16 != 0 || c->page_size > 65536)
        return set_error(W4_ERR_UNSUPPORTED, fn, "page_size must be a multiple of 16 up to 65536");
    if (int64_t(c->kv_heads) * c->page_size > 0x7FFFFFFF)
        return set_error(W4_ERR_UNSUPPORTED, fn, "kv_heads * page_size must be below 2^31");
    if (c->head_dim != 64 && c->head_dim != 128)
        return set_error(W4_ERR_UNSUPPORTED, fn, "head_dim must be 64 or 128");
    if (!aligned16(c->k_codes) || !aligned16(c->v_codes) || !aligned16(c->k_scales) ||
        !aligned16(c->v_scales))
        return set_error(W4_ERR_UNSUPPORTED, fn, "cache pointers must be 16-byte aligned");
    out->k = static_cast<uint8_t *>(c->k_codes);
    out->v = static_cast<uint8_t *>(c->v_codes);
    out->ks = c->k_scales;
    out->vs = c->v_scales;
    out->pages = c->num_pages;
    out->page = c->page_size;
    out->heads = c->kv_heads;
    out->row_bytes = c->fmt == W4KV_INT4 ? c->head_dim / 2 : c->head_dim;
    return W4_OK;
}

int check_batch(const char *fn, const w4kv_batch *b, const w4kv_cache *c, Batch *out) {
    if (!b) return set_error(W4_ERR_INVALID_ARG, fn, "null batch");
    if (b->batch < 0 || b->batch > (1 << 20))
        return set_error(W4_ERR_INVALID_ARG, fn, "batch must be 0 .. 2^20");
    // positions are rounded up to units of up to 256 in 31 bits
    if (b->table_width < 1 || b->table_width > (0x7FFFFFFF - 255) / c->page_size)
        return set_error(W4_ERR_INVALID_ARG, fn, "table_width * page_size must be 1 .. 2^31 - 256");
    if (b->batch > 1 && b->table_stride < 0)
        return set_error(W4_ERR_INVALID_ARG, fn, "table_stride must not be negative");
    if (b->batch > 0 && (!b->page_table || !b->kv_lens || !b->cu_rows))
        return set_error(W4_ERR_INVALID_ARG, fn, "null pointer in the batch");
    out->table = b->page_table;
    out->stride = b->table_stride;
    out->width = static_cast<int>(b->table_width);
    out->lens = b->kv_lens;
    out->cu = b->cu_rows;
    out->n = static_cast<int>(b->batch);
    return W4_OK;
}

int check_rows(const char *fn, const void *p, int64_t rows, int heads, int dim, int64_t row_stride,
               int64_t head_stride, bool output) {
    if (!p) return set_error(W4_ERR_INVALID_ARG, fn, "null pointer");
    const int64_t lim = int64_t(1) << 31;
    if (rows == 1) row_stride = 0;  // of no effect
    if (heads == 1) head_stride = 0;
    if (row_stride < 0 || head_stride < 0 || row_stride > lim || head_stride > (int64_t(1) << 40))
        return set_error(W4_ERR_INVALID_ARG, fn, "stride out of range");
    if (output) {
        const bool rows_outer = (heads == 1 || head_stride >= dim) &&
                                (rows == 1 || row_stride >= (heads - 1) * head_stride + dim);
        const bool heads_outer = (rows == 1 || row_stride >= dim) &&
                                 (heads == 1 || head_stride >= (rows - 1) * row_stride + dim);
        if (!rows_outer && !heads_outer)
            return set_error(W4_ERR_INVALID_ARG, fn, "output rows overlap");
    }
    if (!aligned16(p) || row_stride % 8 != 0 || head_stride % 8 != 0)
        return set_error(W4_ERR_UNSUPPORTED, fn,
                         "rows must start on 16-byte boundaries (strides in multiples of 8)");
    return W4_OK;
}

}  // namespace kv
}  // namespace w4

extern "C" {

int w4kv_append(const w4kv_cache *cache, const w4kv_batch *batch, const void *K, const void *V,
                int xt, int64_t rows, int64_t k_row_stride, int64_t k_head_stride,
                int64_t v_row_stride, int64_t v_head_stride, void *stream) {
    return w4::kv::rows_impl<false>("w4kv_append", cache, batch, K, V, xt, rows, k_row_stride,
                                    k_head_stride, v_row_stride, v_head_stride, stream);
}

int w4kv_read(const w4kv_cache *cache, const w4kv_batch *batch, void *K, void *V, int yt,
              int64_t rows, int64_t k_row_stride, int64_t k_head_stride, int64_t v_row_stride,
              int64_t v_head_stride, void *stream) {
    return w4::kv::rows_impl<true>("w4kv_read", cache, batch, K, V, yt, rows, k_row_stride,
                                   k_head_stride, v_row_stride, v_head_stride, stream);
}

}  // extern "C"
