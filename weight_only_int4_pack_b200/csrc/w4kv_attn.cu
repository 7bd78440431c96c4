// w4kv_attn.cu -- w4kv_attention: argument checks, the choice of kernels, and
// the join of partial results (semantics: include/w4kv.h).
//
// Sequences with at most kRowsLimit (row, query head) pairs per key/value head go
// to the row kernel (w4kv_attn_rows.cu), all others to the tiled one
// (w4kv_attn_tiled.cu).  The numbers of rows live on the device, so the host
// launches what max_rows and the batch allow, and each kernel leaves out the
// other's sequences; a batch of one that may pass the limit goes to the tiled
// kernel, whatever its length.

#include <math.h>

#include "w4kv_attn.cuh"

namespace w4 {
namespace kv {
namespace {

// Item that starts in block blockIdx.x and ends in a later one: the weighted
// mean of its blocks' normalized outputs.
template <int XT>
__global__ void __launch_bounds__(256) combine_kernel(const Attn a, int tile, int dim, bool side) {
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
        // `side`: four dims of a row after another, rows side by side
        const int r = side ? i % R : i / (dim / 4), e = (side ? i / R : i - r * (dim / 4)) * 4;
        const int64_t at = 2 * tile + (side ? int64_t(e) * tile + 4 * r : int64_t(r) * dim + e);
        float M = first[r];
        for (int q = 1; q < d.z; ++q) M = fmaxf(M, rest[2 * q * slot + r]);
        float L = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int q = 0; q < d.z; ++q) {
            const float *p = q ? rest + 2 * q * slot : first;
            const float w = p[tile + r] * ex2(p[r] - M);
            const float4 v = *reinterpret_cast<const float4 *>(p + at);
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

int allow_smem(const void *kernel, int bytes, std::atomic<unsigned long long> *ready) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return cuda_fail("cudaGetDevice", e);
    const unsigned long long bit = dev >= 0 && dev < 64 ? 1ull << dev : 0;
    if (ready->load(std::memory_order_acquire) & bit) return W4_OK;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return cuda_fail("cudaFuncSetAttribute(attention kernel)", e);
    ready->fetch_or(bit, std::memory_order_release);
    return W4_OK;
}

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
    const bool side = tile == kTiledRows;
    return cuda_status(xt == W4_F16 ? cudaLaunchKernelEx(&cfg, combine_kernel<W4_F16>, a, tile, dim, side)
                                    : cudaLaunchKernelEx(&cfg, combine_kernel<W4_BF16>, a, tile, dim, side));
}

namespace {

// Which kernels run, and the workspace: per launch its descriptors, then its slots.
struct Launch {
    int tile = 0;  // rows of a slot; 0: the launch is left out
    int grid = 0;
    size_t begin = 0, slots = 0;  // byte offsets of descriptors and slots
};
struct Plan {
    Launch rows, tiled;
    size_t total = 0;
};

// (row, head) pairs per key/value head up to which the row kernel serves a sequence.
constexpr int kRowsLimit = 64;

size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

Plan make_plan(const DeviceInfo &d, int dim, int64_t batch, int64_t max_rows, int group) {
    Plan p;
    const int64_t pairs = max_rows * group;
    if (pairs <= 8) p.rows.tile = 8;
    else if (pairs <= kRowsLimit || (batch > 1 && group <= kRowsLimit)) p.rows.tile = 16;
    if (pairs > kRowsLimit) p.tiled.tile = kTiledRows;
    p.rows.grid = rows_blocks_per_sm(p.rows.tile) * d.sm_count;
    p.tiled.grid = d.sm_count;
    for (Launch *l : {&p.rows, &p.tiled}) {
        if (!l->tile) continue;
        l->begin = p.total;
        l->slots = l->begin + up256(size_t(l->grid) * sizeof(int4));
        p.total = l->slots + up256(2 * size_t(l->grid) * slot_floats(l->tile, dim) * 4);
    }
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
    a.scale_log2 = static_cast<float>(scale * 1.4426950408889634);
    if (!isfinite(a.scale_log2))
        return set_error(W4_ERR_INVALID_ARG, fn, "scale * log2(e) is not finite");
    if (window < 0 || (window > 0 && !causal))
        return set_error(W4_ERR_INVALID_ARG, fn, "window must be >= 0, and 0 unless causal");
    if (rows == 0 || a.b.n == 0) return W4_OK;
    const int D = cache->head_dim;
    if ((st = check_rows(fn, Q, rows, heads, D, q_row_stride, q_head_stride, false)) != W4_OK) return st;
    if ((st = check_rows(fn, O, rows, heads, D, o_row_stride, o_head_stride, true)) != W4_OK) return st;
    if (reinterpret_cast<uintptr_t>(lse) & 3u)
        return set_error(W4_ERR_UNSUPPORTED, fn, "lse must be 4-byte aligned");
    if (max_rows > rows) max_rows = rows;
    if (max_rows * (heads / a.c.heads) > 0x7FFFFFFF - kTiledRows)
        return set_error(W4_ERR_INVALID_ARG, fn, "max_rows * heads / kv_heads too large");
    DeviceInfo d;
    if ((st = device_info(&d)) != W4_OK) return st;
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
    a.causal = causal != 0;
    a.window = window > 0x7FFFFFFF ? 0 : static_cast<int>(window);
    a.page_magic = page_magic(a.c.page);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    auto partials = [&](const Launch &l) {
        a.desc = reinterpret_cast<int4 *>(ws + l.begin);
        a.slots = reinterpret_cast<float *>(ws + l.slots);
    };
    a.min_rows = 0;
    if (p.rows.tile) {
        partials(p.rows);
        a.max_served = p.rows.tile == 8 ? 8 : kRowsLimit;
        if ((st = launch_rows_attention(a, cache->fmt, D, xt, p.rows.tile, p.rows.grid, s)) != W4_OK) return st;
        if ((st = launch_combine(a, p.rows.grid, p.rows.tile, D, xt, s)) != W4_OK) return st;
        a.min_rows = a.max_served;
    }
    if (p.tiled.tile) {
        partials(p.tiled);
        a.max_served = int64_t(1) << 62;
        if ((st = launch_tiled_attention(a, cache->fmt, D, xt, p.tiled.grid, s)) != W4_OK) return st;
        if ((st = launch_combine(a, p.tiled.grid, p.tiled.tile, D, xt, s)) != W4_OK) return st;
    }
    return W4_OK;
}

}  // extern "C"
