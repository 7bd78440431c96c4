// w4kv_attn.cuh -- what the attention kernels over the quantized cache share:
// their arguments, the cut of a call's work into equal contiguous ranges of
// thread blocks, and the layout of the partial results.
//
// Work is counted in units of 128 cached tokens of an item (a key/value head
// of a sequence; in the tiled kernel, of a tile of its rows), plus kItemCost
// per item for its queries and its output: positions kItemCost + u for unit u,
// the first unit standing for the positions before it too.  The positions of
// all items, in the order (sequence, head, tile), are cut into equal ranges, one
// per block; an item that a cut divides is finished by combine_kernel from the
// partial results of its blocks, in block order (deterministic).  The lengths
// live on the device, so every block finds its range itself: a block-wide sum
// over the sequences, then a scan of those, as many as it has threads, that hold
// its first unit.
#pragma once

#include <float.h>

#include <atomic>

#include "w4kv.cuh"

namespace w4 {
namespace kv {

constexpr int kUnit = 128;    // cached tokens per unit of work
// What an item costs beside its units, in units.  Measured on the device with 2, 3, 4 and 8: a
// decode step of 32 sequences to 4096 (INT4) 107, 111, 113 and 122 us, 5 proposals of
// 16 to 8000 (INT8) 72, 69, 69 and 73, chunks and single tokens mixed 208, 202, 207 and 204.
constexpr int kItemCost = 3;

struct Attn {
    Cache c;
    Batch b;
    const uint16_t *q;
    int64_t q_row, q_head;
    uint16_t *o;
    int64_t o_row, o_head;
    float *lse;
    int64_t rows, max_rows;  // rows of the call; rows of a sequence that are served
    int heads, group;        // query heads; query heads per key/value head
    float scale_log2;        // scale * log2(e)
    int causal, window;
    int64_t min_rows, max_served;  // this launch serves min_rows < rows * group <= max_served
    uint32_t page_magic;           // floor(2^32 / (page / 16)), for tile / (page / 16)
    int4 *desc;    // [grid]: the item that starts in a block and ends in a later one
    float *slots;  // [2 * grid] partial results
    unsigned *status;
};

// The first position that a row at `pos` sees through a window: pos + 1 - window, at least 0.
__device__ __forceinline__ int window_from(int pos, int window) {
    return pos >= window ? pos + 1 - window : 0;
}

// The rows that a launch serves of a sequence, and the cached positions they see.
struct Seq {
    int row0, n;  // first row of the call, rows served (0: not served by this launch)
    int first;    // position of row0 (negative: sees nothing)
    int lo, hi;   // cached positions that any of the rows sees: [lo, hi)
};

// Everything is clamped to the call's rows and to the table; what does not fit is reported.
__device__ __forceinline__ Seq load_seq(const Attn &a, int b) {
    Seq s;
    s.row0 = __ldg(a.b.cu + b);
    const int end = __ldg(a.b.cu + b + 1), len = __ldg(a.b.lens + b);
    s.n = end - s.row0;
    s.first = len - s.n;
    s.lo = s.hi = 0;
    if (s.row0 < 0 || end < s.row0 || end > a.rows) {
        atomicOr(a.status, kStatusBounds);
        s.n = 0;
        return s;
    }
    if (s.n > a.max_rows) {
        atomicOr(a.status, kStatusBounds);
        s.n = static_cast<int>(a.max_rows);
    }
    const int64_t tile = int64_t(s.n) * a.group;
    if (tile <= a.min_rows || tile > a.max_served) {
        s.n = 0;
        return s;
    }
    s.hi = max(0, a.causal ? min(len, s.first + s.n) : len);
    const int room = a.b.width * a.c.page;
    if (s.hi > room) {
        atomicOr(a.status, kStatusBounds);
        s.hi = room;
    }
    if (a.window > 0) s.lo = min(s.hi, window_from(s.first, a.window));
    return s;
}

// tile / (page / 16) and the remainder.
__device__ __forceinline__ int page_of_tile(const Attn &a, int tile, int *rest) {
    const uint32_t d = static_cast<uint32_t>(a.c.page) >> 4;
    uint32_t q = __umulhi(static_cast<uint32_t>(tile), a.page_magic), r = tile - q * d;
    if (r >= d) {  // the estimate is at most one short
        ++q;
        r -= d;
    }
    *rest = static_cast<int>(r);
    return static_cast<int>(q);
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float pow2i(int e) {  // 2^e, -126 <= e <= 127
    return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

// The NaN codes (0x7F, 0xFF) of four E4M3 codes: bit 7 of their bytes.
__device__ __forceinline__ uint32_t e4m3_nans(uint32_t w) {
    return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
}

// Zeros in place of the NaN codes of `bytes` bytes (a lane's words from `at` on, 128 apart);
// *found = 1 if there was one.  A call, so that it costs the loop that seldom needs it little.
inline __device__ __noinline__ void zero_nans(uint32_t *at, int bytes, int *found) {
#pragma unroll 1
    for (int i = 0; i < bytes / 4; i += 32) {
        const uint32_t n = e4m3_nans(at[i]);
        if (n) {
            at[i] &= ~((n >> 7) * 255u);
            *found = 1;
        }
    }
    __syncwarp();
}

// a / b, by 32 bits where they do.
__device__ __forceinline__ int64_t div_small(int64_t a, int64_t b) {
    if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
    return a / b;
}

// Range [start, end) of the block in the cost of all items, and the sequence that holds its
// beginning.  units(b) gives the cost of a sequence's items.  All threads of the block
// (kThreads of them) call it and get the same values.
struct Range {
    int64_t total, start, end;
    int blocks;   // blocks that have units: the first min(gridDim.x, total)
    int b;
    int64_t off;  // of `start` within sequence b
};
struct RangeSmem {
    int64_t warp[32], rest[32];
    int64_t off;
    int b;
};

template <int kThreads, class Units>
__device__ __forceinline__ Range block_range(int n_seq, RangeSmem *sm, Units units) {
    constexpr int kWarps = kThreads / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    Range r;
    // The scan of the first kThreads sequences serves for the total of all as well.
    int64_t v = static_cast<int>(threadIdx.x) < n_seq ? units(threadIdx.x) : 0, inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t up = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += up;
    }
    int64_t rest = 0;  // of the sequences behind them
    for (int i = threadIdx.x + kThreads; i < n_seq; i += kThreads) rest += units(i);
    if (n_seq > kThreads) {
#pragma unroll
        for (int o = 16; o; o >>= 1) rest += __shfl_xor_sync(0xffffffffu, rest, o);
    }
    if (lane == 31) {
        sm->warp[warp] = inc;
        sm->rest[warp] = rest;
    }
    __syncthreads();
    int64_t before = 0, p = inc - v;  // units of the first kThreads sequences; those before this thread's
    r.total = 0;
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) p += sm->warp[w];
        before += sm->warp[w];
        r.total += sm->rest[w];
    }
    r.total += before;
    r.b = 0;
    r.off = r.start = r.end = 0;
    r.blocks = static_cast<int>(min(static_cast<int64_t>(gridDim.x), r.total));
    if (static_cast<int>(blockIdx.x) >= r.blocks) return r;
    r.start = div_small(r.total * blockIdx.x, r.blocks);
    r.end = div_small(r.total * (blockIdx.x + 1), r.blocks);
    if (p <= r.start && r.start < p + v) {
        sm->b = threadIdx.x;
        sm->off = r.start - p;
    }
    for (int base = kThreads; before <= r.start && base < n_seq; base += kThreads) {
        const int i = base + threadIdx.x;
        inc = v = i < n_seq ? units(i) : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t up = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += up;
        }
        __syncthreads();
        if (lane == 31) sm->warp[warp] = inc;
        __syncthreads();
        p = before + inc - v;
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) p += sm->warp[w];
            before += sm->warp[w];
        }
        if (p <= r.start && r.start < p + v) {
            sm->b = i;
            sm->off = r.start - p;
        }
    }
    __syncthreads();
    r.b = sm->b;
    r.off = sm->off;
    return r;
}

// The block whose range holds unit u.
__device__ __forceinline__ int block_of_unit(int64_t u, const Range &r) {
    return static_cast<int>(div_small((u + 1) * r.blocks - 1, r.total));
}

// Reference maximum of a row that has seen nothing: the least finite number, so
// that no score is below it and differences of equal maxima are numbers.
constexpr float kNone = -FLT_MAX;

// A partial result: maxima and sums (base 2) and the normalized output of
// `rows` rows: [rows] + [rows] + [rows][dim] floats (the tiled kernel's output:
// [dim / 4][rows][4]).
__host__ __device__ constexpr int64_t slot_floats(int rows, int dim) {
    return int64_t(rows) * (dim + 2);
}

inline uint32_t page_magic(int page) {
    const uint32_t d = static_cast<uint32_t>(page) >> 4;
    return d == 1 ? 0xFFFFFFFFu : static_cast<uint32_t>((uint64_t(1) << 32) / d);
}

// Lets a kernel use `bytes` of dynamic shared memory; once per device.
int allow_smem(const void *kernel, int bytes, std::atomic<unsigned long long> *ready);

// Joins the partial results of items that several blocks share; after each
// attention kernel, with that kernel's grid and `tile` rows per slot.
int launch_combine(const Attn &a, int grid, int tile, int dim, int xt, cudaStream_t stream);

// Items of up to 256 (row, head) pairs on tcgen05 (w4kv_attn_tiled.cu).
constexpr int kTiledRows = 256;
int launch_tiled_attention(const Attn &a, int fmt, int dim, int xt, int grid, cudaStream_t stream);

// Items of 8 or 16 (row, head) pairs, `tile`: warp-level MMA (w4kv_attn_rows.cu).
constexpr int rows_blocks_per_sm(int tile) { return tile == 8 ? 4 : 2; }
int launch_rows_attention(const Attn &a, int fmt, int dim, int xt, int tile, int grid,
                          cudaStream_t stream);

}  // namespace kv
}  // namespace w4
