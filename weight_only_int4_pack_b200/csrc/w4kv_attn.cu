// w4kv_attn.cu -- w4kv_attention: attention of new rows over the quantized
// paged cache (semantics: include/w4kv.h).
//
// One warp per (row, query head): the lanes hold D / 32 elements of the query
// each and walk over the cached tokens with a running maximum and sum.

#include <cuda_fp8.h>
#include <math.h>

#include "w4kv_attn.cuh"

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
attention_kernel(const Attn a, int64_t items, float scale) {
    const Cache &c = a.c;
    const Batch &bt = a.b;
    const uint16_t *Q = a.q;
    uint16_t *O = a.o;
    float *lse = a.lse;
    const int64_t qrs = a.q_row, qhs = a.q_head, ors = a.o_row, ohs = a.o_head, max_rows = a.max_rows;
    const int heads = a.heads, causal = a.causal, window = a.window;
    unsigned *status = a.status;
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
    const Seq sq = load_seq(a, b);
    if (sq.n == 0) return;
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

// Item that starts in block blockIdx.x and ends in a later one: the weighted
// mean of its blocks' normalized outputs.
template <int XT>
__global__ void __launch_bounds__(256) combine_kernel(const Attn a, int tile, int dim) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int4 d = a.desc[blockIdx.x];
    if (d.z == 0) return;
    const Seq s = load_seq(a, d.x);
    const int64_t r_first = int64_t(d.w) * tile;
    const int R = static_cast<int>(min(static_cast<int64_t>(tile), int64_t(s.n) * a.group - r_first));
    const int64_t slot = slot_floats(tile, dim);
    const float *first = a.slots + (2 * int64_t(blockIdx.x) + 1) * slot;
    const float *rest = a.slots + 2 * int64_t(blockIdx.x) * slot;  // + 2 i slots for block + i
    for (int i = blockIdx.y * 256 + threadIdx.x; i < R * dim / 4; i += 256 * gridDim.y) {
        const int r = i / (dim / 4), e = (i - r * (dim / 4)) * 4;
        float M = first[r];
        for (int q = 1; q < d.z; ++q) M = fmaxf(M, rest[2 * q * slot + r]);
        float L = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int q = 0; q < d.z; ++q) {
            const float *p = q ? rest + 2 * q * slot : first;
            const float w = p[tile + r] * ex2(p[r] - M);
            const float4 v = *reinterpret_cast<const float4 *>(p + 2 * tile + r * dim + e);
            L += w;
            o.x = fmaf(w, v.x, o.x), o.y = fmaf(w, v.y, o.y);
            o.z = fmaf(w, v.z, o.z), o.w = fmaf(w, v.w, o.w);
        }
        const float inv = L == 0.f ? 0.f : 1.f / L;
        const int64_t rr = r_first + r;
        const int64_t t = s.row0 + rr / a.group;
        const int h = d.y * a.group + static_cast<int>(rr % a.group);
        uint2 y;
        y.x = narrow1<XT>(o.x * inv) | static_cast<uint32_t>(narrow1<XT>(o.y * inv)) << 16;
        y.y = narrow1<XT>(o.z * inv) | static_cast<uint32_t>(narrow1<XT>(o.w * inv)) << 16;
        *reinterpret_cast<uint2 *>(a.o + t * a.o_row + h * a.o_head + e) = y;
        if (a.lse && e == 0)
            a.lse[t * a.heads + h] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
    }
}

}  // namespace

int launch_combine(const Attn &a, int grid, int tile, int dim, int xt, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid, max(1, tile * dim / 4 / 1024));
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cuda_status(xt == W4_F16 ? cudaLaunchKernelEx(&cfg, combine_kernel<W4_F16>, a, tile, dim)
                                    : cudaLaunchKernelEx(&cfg, combine_kernel<W4_BF16>, a, tile, dim));
}

namespace {

// Tile of the row kernel for sequences of up to `pairs` (row, head) pairs per
// key/value head: 8 or 16, or 0 when none of the batch can be that small.
struct Plan {
    int rows_tile = 0;  // 8 or 16: the row kernel runs
    bool tiled = false; // the tiled kernel runs
    int grid = 0;
    size_t slots = 0, total = 0;  // bytes: partials per launch, workspace
};

Plan make_plan(const DeviceInfo &d, int dim, int64_t batch, int64_t max_rows, int group) {
    Plan p;
    const int64_t pairs = max_rows * group;
    p.tiled = pairs > 16;
    if (pairs <= 8) p.rows_tile = 8;
    else if (pairs <= 16 || (batch > 1 && group <= 16)) p.rows_tile = 16;
    p.grid = (p.rows_tile == 8 ? 4 : 3) * d.sm_count;
    const size_t desc = (size_t(p.grid) * 16 + 255) & ~size_t(255);
    p.slots = 2 * size_t(p.grid) * slot_floats(p.rows_tile, dim) * 4;
    p.total = p.rows_tile ? desc + ((p.slots + 255) & ~size_t(255)) : 0;
    return p;
}

}  // namespace
}  // namespace kv
}  // namespace w4

extern "C" {

size_t w4kv_attention_workspace_bytes(const w4kv_cache *cache, int64_t batch, int64_t rows,
                                      int64_t max_rows, int heads) {
    using namespace w4;
    using namespace w4::kv;
    Cache c;
    if (check_cache("w4kv_attention_workspace_bytes", cache, &c) != W4_OK) return 0;
    if (batch < 1 || rows < 1 || max_rows < 1 || heads < 1 || heads % c.heads != 0) return 0;
    DeviceInfo d;
    if (device_info(&d) != W4_OK) return 0;
    return make_plan(d, cache->head_dim, batch, max_rows < rows ? max_rows : rows, heads / c.heads).total;
}

int w4kv_attention(const w4kv_cache *cache, const w4kv_batch *batch, const void *Q, int xt,
                   int64_t rows, int heads, int64_t q_row_stride, int64_t q_head_stride, void *O,
                   int64_t o_row_stride, int64_t o_head_stride, float *lse, int64_t max_rows,
                   float scale, int causal, int64_t window, void *workspace,
                   size_t workspace_bytes, void *stream) {
    using namespace w4;
    using namespace w4::kv;
    const char *fn = "w4kv_attention";
    Attn a = {};
    int st;
    if ((st = check_cache(fn, cache, &a.c)) != W4_OK) return st;
    if ((st = check_batch(fn, batch, cache, &a.b)) != W4_OK) return st;
    if (xt != W4_F16 && xt != W4_BF16)
        return set_error(W4_ERR_INVALID_ARG, fn, "xt is not W4_F16 or W4_BF16");
    if (rows < 0 || rows > 0x7FFFFFFF)
        return set_error(W4_ERR_INVALID_ARG, fn, "rows must be 0 .. 2^31 - 1");
    if (heads < 1 || heads % a.c.heads != 0)
        return set_error(W4_ERR_INVALID_ARG, fn, "heads must be a multiple of kv_heads");
    if (max_rows < 1) return set_error(W4_ERR_INVALID_ARG, fn, "max_rows must be positive");
    if (!isfinite(scale)) return set_error(W4_ERR_INVALID_ARG, fn, "scale is not finite");
    if (window < 0 || (window > 0 && !causal))
        return set_error(W4_ERR_INVALID_ARG, fn, "window must be >= 0, and 0 unless causal");
    if (rows == 0 || a.b.n == 0) return W4_OK;
    const int D = cache->head_dim;
    if ((st = check_rows(fn, Q, rows, heads, D, q_row_stride, q_head_stride, false)) != W4_OK) return st;
    if ((st = check_rows(fn, O, rows, heads, D, o_row_stride, o_head_stride, true)) != W4_OK) return st;
    if (reinterpret_cast<uintptr_t>(lse) & 3u)
        return set_error(W4_ERR_UNSUPPORTED, fn, "lse must be 4-byte aligned");
    DeviceInfo d;
    if ((st = device_info(&d)) != W4_OK) return st;
    if (max_rows > rows) max_rows = rows;
    const Plan p = make_plan(d, D, a.b.n, max_rows, heads / a.c.heads);
    if (p.total > 0 && (!workspace || workspace_bytes < p.total ||
                        (reinterpret_cast<uintptr_t>(workspace) & 255u)))
        return set_error(W4_ERR_INVALID_ARG, fn,
                         "workspace missing, misaligned or smaller than w4kv_attention_workspace_bytes");
    if ((a.status = device_status_ptr()) == nullptr) return W4_ERR_CUDA;
    a.q = static_cast<const uint16_t *>(Q);
    a.q_row = q_row_stride, a.q_head = q_head_stride;
    a.o = static_cast<uint16_t *>(O);
    a.o_row = o_row_stride, a.o_head = o_head_stride;
    a.lse = lse;
    a.rows = rows, a.max_rows = max_rows;
    a.heads = heads, a.group = heads / a.c.heads;
    a.scale_log2 = static_cast<float>(scale * 1.4426950408889634);
    a.causal = causal != 0;
    a.window = window > 0x7FFFFFFF ? 0 : static_cast<int>(window);
    a.page_magic = page_magic(a.c.page);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (p.rows_tile) {
        a.min_rows = 0, a.max_served = p.rows_tile;
        a.desc = static_cast<int4 *>(workspace);
        a.slots = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) +
                                            ((size_t(p.grid) * 16 + 255) & ~size_t(255)));
        if ((st = launch_rows_attention(a, cache->fmt, D, xt, p.rows_tile, p.grid, s)) != W4_OK) return st;
        if ((st = launch_combine(a, p.grid, p.rows_tile, D, xt, s)) != W4_OK) return st;
    }
    if (!p.tiled) return W4_OK;
    a.min_rows = p.rows_tile;
    a.max_served = int64_t(1) << 62;
    const int64_t items = rows * heads;
    if (items > int64_t(0x7FFFFFFF)) return set_error(W4_ERR_INVALID_ARG, fn, "rows * heads too large");
    const unsigned grid = static_cast<unsigned>((items + 3) / 4);
#define RUN(F, DD, X) attention_kernel<F, DD, X><<<grid, 128, 0, s>>>(a, items, scale)
#define RUN_X(F, DD) if (xt == W4_F16) RUN(F, DD, W4_F16); else RUN(F, DD, W4_BF16)
#define RUN_D(F) if (D == 64) { RUN_X(F, 64); } else { RUN_X(F, 128); }
    if (cache->fmt == W4KV_INT8) { RUN_D(W4KV_INT8) }
    else if (cache->fmt == W4KV_E4M3) { RUN_D(W4KV_E4M3) }
    else { RUN_D(W4KV_INT4) }
    return cuda_status(cudaGetLastError());
}

}  // extern "C"
