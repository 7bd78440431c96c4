// w4kv_attn.cu -- w4kv_attention: attention of new rows over the quantized
// paged cache (semantics: include/w4kv.h).
//
// One warp per (row, query head): the lanes hold D / 32 elements of the query
// each and walk over the cached tokens with a running maximum and sum.

#include <cuda_fp8.h>
#include <math.h>

#include "w4kv.cuh"

namespace w4 {
namespace kv {
namespace {

template <int FMT, int N>
__device__ __forceinline__ void load_codes(const uint8_t *row, int lane, uint32_t word, float v[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int k = lane * N + i;
        if (FMT == W4KV_INT4) {
            const uint32_t w = reinterpret_cast<const uint32_t *>(row)[k >> 3];
            const int j = k & 7;
            v[i] = static_cast<float>(static_cast<int>((w >> (4 * ((j >> 1) + 4 * (j & 1)))) & 15u) -
                                      static_cast<int>(word & 15u));
        } else if (FMT == W4KV_INT8) {
            v[i] = static_cast<float>(reinterpret_cast<const int8_t *>(row)[k]);
        } else {
            const __half_raw h = __nv_cvt_fp8_to_halfraw(row[k], __NV_E4M3);
            v[i] = __half2float(*reinterpret_cast<const __half *>(&h));
        }
    }
}

template <int FMT, int D, int XT>
__global__ void __launch_bounds__(128)
attention_kernel(const Cache c, const Batch bt, const uint16_t *__restrict__ Q, int64_t qrs, int64_t qhs,
                 uint16_t *__restrict__ O, int64_t ors, int64_t ohs, float *__restrict__ lse,
                 int64_t items, int heads, int64_t max_rows, float scale, int causal, int window,
                 unsigned *__restrict__ status) {
    constexpr int N = D / 32;
    const int lane = threadIdx.x & 31;
    const int64_t item = (int64_t(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
    if (item >= items) return;
    const int t = static_cast<int>(item / heads), h = static_cast<int>(item % heads);
    const int b = find_sequence(bt.cu, bt.n, t, lane);
    if (b < 0) return;
    if (t - __ldg(bt.cu + b) >= max_rows) {
        if (lane == 0) atomicOr(status, kStatusBounds);
        return;
    }
    const int len = __ldg(bt.lens + b);
    const int pos = len - (__ldg(bt.cu + b + 1) - t);
    const int hi = causal ? pos + 1 : len;
    const int lo = window > 0 ? max(0, pos + 1 - window) : 0;
    const int kvh = h / (heads / c.heads);
    float q[N], o[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        q[i] = widen1<XT>(Q[t * qrs + h * qhs + lane * N + i]);
        o[i] = 0.f;
    }
    float m = -INFINITY, l = 0.f;
    for (int j = lo; j < hi; ++j) {
        const int64_t r0 = row_of(c, bt, b, j);
        if (r0 < 0) {
            if (lane == 0) atomicOr(status, kStatusBounds);
            if (j / c.page >= bt.width) break;
            continue;
        }
        const int64_t r = r0 + int64_t(kvh) * c.page;
        const uint32_t kw = __float_as_uint(c.ks[r]), vw = __float_as_uint(c.vs[r]);
        float kk[N], vv[N];
        load_codes<FMT, N>(c.k + r * c.row_bytes, lane, kw, kk);
        load_codes<FMT, N>(c.v + r * c.row_bytes, lane, vw, vv);
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i) s = fmaf(q[i], kk[i], s);
#pragma unroll
        for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
        s *= (FMT == W4KV_INT4 ? int4_scale(kw) : __uint_as_float(kw)) * scale;
        const float vs = FMT == W4KV_INT4 ? int4_scale(vw) : __uint_as_float(vw);
        const float mn = fmaxf(m, s);
        const float f = m == -INFINITY ? 0.f : expf(m - mn);
        const float p = expf(s - mn);
        l = l * f + p;
#pragma unroll
        for (int i = 0; i < N; ++i) o[i] = o[i] * f + p * vs * vv[i];
        m = mn;
    }
    const float inv = l > 0.f || isnan(l) ? 1.f / l : 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) O[t * ors + h * ohs + lane * N + i] = narrow1<XT>(o[i] * inv);
    if (lse && lane == 0) lse[int64_t(t) * heads + h] = l > 0.f || isnan(l) ? m + logf(l) : -INFINITY;
}

}  // namespace
}  // namespace kv
}  // namespace w4

extern "C" {

size_t w4kv_attention_workspace_bytes(const w4kv_cache *cache, int64_t batch, int64_t rows,
                                      int64_t max_rows, int heads) {
    return 0;
}

int w4kv_attention(const w4kv_cache *cache, const w4kv_batch *batch, const void *Q, int xt,
                   int64_t rows, int heads, int64_t q_row_stride, int64_t q_head_stride, void *O,
                   int64_t o_row_stride, int64_t o_head_stride, float *lse, int64_t max_rows,
                   float scale, int causal, int64_t window, void *workspace,
                   size_t workspace_bytes, void *stream) {
    using namespace w4;
    using namespace w4::kv;
    const char *fn = "w4kv_attention";
    Cache c;
    Batch b;
    int st;
    if ((st = check_cache(fn, cache, &c)) != W4_OK) return st;
    if ((st = check_batch(fn, batch, cache, &b)) != W4_OK) return st;
    if (xt != W4_F16 && xt != W4_BF16)
        return set_error(W4_ERR_INVALID_ARG, fn, "xt is not W4_F16 or W4_BF16");
    if (rows < 0 || rows > 0x7FFFFFFF)
        return set_error(W4_ERR_INVALID_ARG, fn, "rows must be 0 .. 2^31 - 1");
    if (heads < 1 || heads % c.heads != 0)
        return set_error(W4_ERR_INVALID_ARG, fn, "heads must be a multiple of kv_heads");
    if (max_rows < 1) return set_error(W4_ERR_INVALID_ARG, fn, "max_rows must be positive");
    if (!isfinite(scale)) return set_error(W4_ERR_INVALID_ARG, fn, "scale is not finite");
    if (window < 0 || (window > 0 && !causal))
        return set_error(W4_ERR_INVALID_ARG, fn, "window must be >= 0, and 0 unless causal");
    if (rows == 0 || b.n == 0) return W4_OK;
    const int D = cache->head_dim;
    if ((st = check_rows(fn, Q, rows, heads, D, q_row_stride, q_head_stride, false)) != W4_OK) return st;
    if ((st = check_rows(fn, O, rows, heads, D, o_row_stride, o_head_stride, true)) != W4_OK) return st;
    if (reinterpret_cast<uintptr_t>(lse) & 3u)
        return set_error(W4_ERR_UNSUPPORTED, fn, "lse must be 4-byte aligned");
    const int64_t items = rows * heads;
    if (items > int64_t(0x7FFFFFFF)) return set_error(W4_ERR_INVALID_ARG, fn, "rows * heads too large");
    unsigned *status = device_status_ptr();
    if (!status) return W4_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const unsigned grid = static_cast<unsigned>((items + 3) / 4);
    const int w = window > 0x7FFFFFFF ? 0 : static_cast<int>(window);
#define RUN(F, DD, X)                                                                              \
    attention_kernel<F, DD, X><<<grid, 128, 0, s>>>(                                               \
        c, b, static_cast<const uint16_t *>(Q), q_row_stride, q_head_stride,                       \
        static_cast<uint16_t *>(O), o_row_stride, o_head_stride, lse, items, heads, max_rows,      \
        scale, causal, w, status)
#define RUN_X(F, DD) if (xt == W4_F16) RUN(F, DD, W4_F16); else RUN(F, DD, W4_BF16)
#define RUN_D(F) if (D == 64) { RUN_X(F, 64); } else { RUN_X(F, 128); }
    if (cache->fmt == W4KV_INT8) { RUN_D(W4KV_INT8) }
    else if (cache->fmt == W4KV_E4M3) { RUN_D(W4KV_E4M3) }
    else { RUN_D(W4KV_INT4) }
    return cuda_status(cudaGetLastError());
}

}  // extern "C"
