// w4kv_attn_tiled.cu -- attention of chunks of new rows over the quantized
// cache on the 5th-generation tensor cores.
//
// An item is a key/value head of a sequence and up to 256 (row, query head)
// pairs: two tiles A and B of 128 rows, that share every dequantized key and
// value tile of 128 cached tokens (a step).  Mathematics as in
// w4kv_attn_rows.cu (running maximum that moves by 2^8 at least, weights held
// relative to the largest value scale that the row has seen), with
//     S = Q K^T       tcgen05.mma, both operands in shared memory, fp32 in TMEM
//     O += P V        tcgen05.mma, P (fp16) read from TMEM, V in shared memory
// Codes are widened exactly to fp16 (INT4 as u - z); the scales are applied to
// S's columns and to P's, in fp32.  Tensor memory: S_A, S_B (128 columns each,
// overwritten by P_A, P_B), O_A, O_B.
//
// An item of at most 128 rows runs both streams on the same rows: A takes the
// even steps and B the odd ones, and their results are joined at the end, so
// that the tensor cores and the softmax still alternate.
//
// Warps (20, the last idle): 0-3 softmax of A (a row per thread), 4-7 of B; 8-15 read codes
// from the pages (copied some tiles ahead) and widen them into the swizzled
// operand tiles (three buffers for K and V in turn; V is the MN-major operand,
// so both have the layout of the rows as they lie); 16 and 17 issue the MMAs of
// A and B; 18 prepares the steps' scales.  A stream's MMAs are S(0), then per
// step O, S(next): while its softmax runs the tensor cores work on the other's.
//
// The softmax takes one pass over S in the common case; masks, moving maxima and
// references of the rows' own share a second one, so that the common one's code
// stays small (with the rare paths inside it: 2% on long chunks, 4% on short ones).
//
// What bounds it: a step needs 2048 cycles of tensor cores (2 tiles x 2 x 128 x 128 x
// dim / 4096 a cycle at dim 128) and 2048 of exp2 (16 a cycle), and takes 7500 to 8000,
// the chain scores -> softmax (about half of it; the tensor cores' operand reads
// compete with its loads of the scales) -> MMA warp awake -> O and S issued -> S
// complete, which two streams overlap in part.  The softmax role spills some at 160
// registers.  Measured (device time): 2048 rows at 16384 tokens, 64 / 8 heads x 128,
// INT8: 1.67 ms, 618 TFLOP/s, E4M3 1.75, INT4 1.92; 509 rows at 4096, 32 heads, INT8:
// 106 us.  Widening alone with the MMAs runs at 1300 TFLOP/s.  Every mbarrier wait is
// bounded.

#include <cuda_fp16.h>
#include <math.h>

#include <type_traits>

#include "w4_tc.cuh"
#include "w4kv_attn.cuh"

namespace w4 {
namespace kv {
namespace {

using namespace tc;

constexpr int kM = 128;              // rows of a tile (MMA M, TMEM lanes)
constexpr int kTileRows = kTiledRows;  // rows of an item
static_assert(kTileRows == 2 * kM, "two tiles");
constexpr int kStep = kUnit;         // cached tokens per step (MMA N of S, K of P V)
constexpr int kBuffers = 3;          // operand buffers, taken by K(0) V(0) K(1) V(1) .. in turn
constexpr int kScaleStages = 4;
constexpr int kScaleAhead = 3;       // steps that scale words are copied ahead of use
constexpr int kWidenWarps = 8;
constexpr int kThreads = 32 * (8 + kWidenWarps + 4);  // the last warp only completes a warpgroup
// Registers per thread: launched with 96 x 640 = 61440, and split into
// 160 x 256 (softmax) + 56 x 256 (widening) + 48 x 128 = 61440.
constexpr int kRegSoftmax = 160, kRegWiden = 56, kRegRest = 48;
static_assert(kRegSoftmax * 256 + kRegWiden * 256 + kRegRest * 128 <= 96 * kThreads, "register split");
constexpr int kTmemCols = 512;

// ---- items ------------------------------------------------------------------------------------

struct Walk {
    Seq s;
    int b, h, tile;      // sequence, key/value head, row tile
    int tiles, nu;       // row tiles of the sequence; units of the item
    int r0, R;           // first (row, head) pair of the tile, pairs
    int lo, hi;          // cached positions its rows see; lo a multiple of 16
    int x;               // walked of the item, in cost
    int64_t rem;         // cost of the block's range not yet walked
    int u0, u1;          // units of the current segment
};

__device__ __forceinline__ void tile_bounds(const Attn &a, const Seq &s, int tile, int *lo, int *hi) {
    const int r0 = tile * kTileRows;  // rows * group of a call is below 2^31
    const int r1 = min(s.n * a.group, r0 + kTileRows) - 1;
    *hi = a.causal ? min(s.hi, max(0, s.first + r1 / a.group + 1)) : s.hi;
    *lo = a.window > 0 ? window_from(s.first + r0 / a.group, a.window) : 0;
    *lo = min(*lo, *hi) & ~15;
}

__device__ __forceinline__ int tile_units(const Attn &a, const Seq &s, int tile) {
    int lo, hi;
    tile_bounds(a, s, tile, &lo, &hi);
    return max(1, (hi - lo + kStep - 1) / kStep);
}

__device__ __forceinline__ int seq_tiles(const Attn &a, const Seq &s) {
    return (s.n * a.group - 1) / kTileRows + 1;
}

__device__ __forceinline__ void set_item(const Attn &a, Walk &w) {
    tile_bounds(a, w.s, w.tile, &w.lo, &w.hi);
    w.nu = max(1, (w.hi - w.lo + kStep - 1) / kStep);
    w.r0 = w.tile * kTileRows;
    w.R = min(kTileRows, w.s.n * a.group - w.r0);
}

// Opens the segment (the part of one item in the block's range) at w.x.
__device__ __forceinline__ void open_segment(Walk &w) {
    const int x1 = static_cast<int>(min(static_cast<int64_t>(w.nu + kItemCost), w.x + w.rem));
    w.u0 = max(0, w.x - kItemCost);
    w.u1 = max(0, x1 - kItemCost);
    w.rem -= x1 - w.x;
    w.x = x1;
}

// To the next segment with units; false when the range is walked.
__device__ __forceinline__ bool next_segment(const Attn &a, Walk &w) {
    do {
        if (w.rem == 0) return false;
        w.x = 0;
        if (++w.tile == w.tiles) {
            w.tile = 0;
            if (++w.h == a.c.heads) {
                w.h = 0;
                do {
                    if (w.b + 1 < a.b.n) ++w.b;
                    w.s = load_seq(a, w.b);
                } while (w.s.n == 0 && w.b + 1 < a.b.n);
                w.tiles = max(1, seq_tiles(a, w.s));
            }
        }
        set_item(a, w);
        open_segment(w);
    } while (w.u0 == w.u1);
    return true;
}

__device__ __forceinline__ bool first_segment(const Attn &a, const Range &r, Walk &w) {
    w.b = r.b;
    w.s = load_seq(a, w.b);
    w.tiles = max(1, seq_tiles(a, w.s));
    int64_t per_head = 0;
    for (int t = 0; t < w.tiles; ++t) per_head += kItemCost + tile_units(a, w.s, t);
    w.h = static_cast<int>(div_small(r.off, per_head));
    int64_t x = r.off - w.h * per_head;
    for (w.tile = 0;; ++w.tile) {
        set_item(a, w);
        if (x < w.nu + kItemCost || w.tile + 1 >= w.tiles) break;
        x -= w.nu + kItemCost;
    }
    w.x = static_cast<int>(x);
    w.rem = r.end - r.start;
    open_segment(w);
    return w.u0 < w.u1 || next_segment(a, w);
}

// Steps of the current segment that stream t takes part in: a prefix.
__device__ __forceinline__ int stream_steps(const Attn &a, const Walk &w, int t) {
    const int ns = w.u1 - w.u0;
    if (t == 1 || w.R <= kM || !a.causal) return ns;
    const int hi = min(w.hi, w.s.first + (w.r0 + kM - 1) / a.group + 1);  // tile A sees less
    return min(ns, max(0, (hi - w.lo + kStep - 1) / kStep - w.u0));
}

// Steps of the current segment for which stream t has MMAs of its own.  A
// segment without any (a row tile that sees nothing, or none of the block's
// part) passes none of the stream's barriers, q_full among them: every phase of
// q_full is then followed by an s_full that the softmax waits for, so that it
// cannot complete a second phase before the MMA warp has seen the first (a
// one-bit parity would not show two).
__device__ __forceinline__ int own_steps(const Attn &a, const Walk &w, int t) {
    return w.R <= kM ? (w.u1 - w.u0 + 1 - t) >> 1 : stream_steps(a, w, t);
}

// Positions of the item that all its rows see.
__device__ __forceinline__ void common_bounds(const Attn &a, const Walk &w, int *lo, int *hi) {
    *hi = a.causal ? min(w.hi, w.s.first + w.r0 / a.group + 1) : w.hi;
    *lo = w.s.lo;
    if (a.window > 0) *lo = max(*lo, window_from(w.s.first + (w.r0 + w.R - 1) / a.group, a.window));
}

// The warp's walk in shared memory, moved by lane 0.
__device__ __forceinline__ bool warp_next(const Attn &a, Walk *w) {
    __syncwarp();
    int more = 0;
    if ((threadIdx.x & 31) == 0) more = next_segment(a, *w);
    more = __shfl_sync(0xffffffffu, more, 0);
    __syncwarp();
    return more != 0;
}

// Of a step: the tokens that all rows of the item see, from bits kFrom to kTo; whether it opens a
// segment.
constexpr int kFrom = 8, kTo = 16;
constexpr uint32_t kOpens = 1u << 31;

struct alignas(16) Control {
    float ks[kScaleStages][kStep];  // key scales times scale * log2(e)
    float vs[kScaleStages][kStep];  // value scales times 2^(133 - vexp), or as they are
    uint32_t word[kScaleAhead + 1][2][kStep];  // scale words on their way: keys, values
    uint32_t word_info[kScaleAhead + 1];       // their bad groups; kFrom, kTo; kOpens
    float stat[2][2][kM];           // [stream][maximum, sum][row], to join split streams
    int row_vexp[2][kM];            // [stream][row]: the row's own vexp, while a warp's rows differ
    // Largest exponent field (at least 7) of the value scales of the segment's tokens so far that
    // all rows of the item see; negated if the step has larger ones, that not all see.
    int vexp[kScaleStages];
    uint8_t vgroup[kScaleStages][8];  // then: the largest of each 16 tokens
    uint32_t bad[kScaleStages];     // bit i: tokens 16 i .. 16 i + 15 have no page
    uint64_t q_full[2], s_full[2], p_full[2], pv_done[2];
    uint64_t full[kBuffers], empty[kBuffers];
    uint64_t sc_full[kScaleStages], sc_empty[kScaleStages], joined;
    Walk walk[8 + kWidenWarps + 4];  // of each warp: read by all its lanes, moved by lane 0
    RangeSmem range;
    uint32_t tmem;
    int abort_flag, mma_lock;
    int nans;  // a value's NaN code has been taken out: see zero_nans
};

template <int FMT, int D>
struct Layout {
    static constexpr int kRow = FMT == W4KV_INT4 ? D / 2 : D;  // code bytes of a row
    static constexpr int kBlock = 128 * 128;                   // 128 rows of 64 fp16: the swizzled unit
    static constexpr int kBlocks = D / 64;
    static constexpr int kTile = kBlocks * kBlock;
    // Codes on their way: a warp's 16 rows of a tile, and for INT4 their scale words.
    static constexpr int kRawWarp = 16 * kRow + (FMT == W4KV_INT4 ? 64 : 0);
    static constexpr int kRawTile = kWidenWarps * kRawWarp;
    static constexpr int kRawTiles = kRow == 128 ? 3 : 5;
    static constexpr int kQ = 0, kKV = 2 * kTile, kRaw = kKV + kBuffers * kTile;
    static constexpr int kControl = kRaw + kRawTiles * kRawTile;
    // at least 120 KB, so that one block (all of tensor memory) is on an SM
    static constexpr int kUsed = kControl + static_cast<int>(sizeof(Control)) + 1024;
    static constexpr int kSmem = kUsed < 120 * 1024 ? 120 * 1024 : kUsed;
    static_assert(kSmem <= 227 * 1024 && kControl % 16 == 0, "shared memory");
};

// ---- instructions ------------------------------------------------------------------------------

// Bounded wait (kWaitNs), with the thread suspended between looks at the clock
// and the abort flag, so that waiting warps take no issue slots.
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, volatile int *abort_flag,
                                         unsigned *status) {
    auto attempt = [&]() {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 20000;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(bar), "r"(parity)
            : "memory");
        return ok != 0;
    };
    if (attempt()) return true;
    const unsigned long long t0 = globaltimer();
    while (!attempt()) {
        if (*abort_flag) return false;
        if (globaltimer() - t0 > kWaitNs) {
            *abort_flag = 1;
            atomicOr(status, 1u);
            return false;
        }
    }
    return true;
}

// A lock between the threads that issue MMAs; a wait that runs out goes on without it.
__device__ __forceinline__ void lock(int *word, volatile int *abort_flag, unsigned *status) {
    if (atomicCAS_block(word, 0, 1) == 0) return;
    const unsigned long long t0 = globaltimer();
    while (atomicCAS_block(word, 0, 1) != 0) {
        if (*abort_flag) return;
        if (globaltimer() - t0 > kWaitNs) {
            *abort_flag = 1;
            atomicOr(status, 1u);
            return;
        }
    }
}
__device__ __forceinline__ void unlock(int *word) { atomicExch_block(word, 0); }

// kind::f16, D f32, A and B fp16, M = 128; kTransB: B is MN-major.
template <int N, bool kTransB>
__host__ __device__ constexpr uint32_t instr_desc() {
    return (1u << 4) | (kTransB ? 1u << 16 : 0u) | (static_cast<uint32_t>(N >> 3) << 17) |
           (static_cast<uint32_t>(kM >> 4) << 24);
}

// Shared-memory descriptors, 128-byte swizzle, rows of 128 bytes in groups of 8
// (1024 bytes apart).  The low word holds the address and, for an MN-major
// operand of more than 64 elements, the distance of the next 64 (leading byte
// offset); the high word is the same for all: stride offset, version, swizzle.
constexpr uint32_t kDescHigh = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_low(uint32_t saddr, uint32_t leading) {
    return ((saddr & 0x3FFFF) >> 4) | (leading >> 4) << 16;
}

__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a_low, uint32_t b_low, uint32_t idesc, bool acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "mov.b64 a, {%1, %5};\n\tmov.b64 b, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d),
        "r"(a_low), "r"(b_low), "r"(idesc), "r"(static_cast<uint32_t>(acc)), "r"(kDescHigh)
        : "memory");
}

__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b_low, uint32_t idesc, bool acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "mov.b64 b, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b_low), "r"(idesc), "r"(static_cast<uint32_t>(acc)), "r"(kDescHigh)
        : "memory");
}

__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
        "%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
          "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
          "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr));
}

__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
        "%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15])
        : "r"(addr));
}

__device__ __forceinline__ void tmem_ld8(uint32_t addr, uint32_t (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(addr));
}

__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
        "%15,%16};" ::"r"(addr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

__device__ __forceinline__ void tmem_st8(uint32_t addr, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(addr),
                 "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}

// Waits for the loads issued so far; r depends on it, so that nothing made of r
// comes before.
__device__ __forceinline__ void tmem_wait_ld8(uint32_t (&r)[8]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                   "+r"(r[6]), "+r"(r[7])::"memory");
}

__device__ __forceinline__ void tmem_wait_ld32(uint32_t (&r)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                   "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                   "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]),
                   "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                   "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                   "+r"(r[30]), "+r"(r[31])::"memory");
}

__device__ __forceinline__ void tmem_wait_ld16(uint32_t (&r)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]),
                   "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]),
                   "+r"(r[14]), "+r"(r[15])::"memory");
}

__device__ __forceinline__ void tmem_wait_st() {
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile(
        "{\n\t.reg .pred P;\n\telect.sync _|P, 0xffffffff;\n\tselp.b32 %0, 1, 0, P;\n\t}"
        : "=r"(p));
    return p != 0;
}

// Pairs of fp32 in one 64-bit register.
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t x) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

// Byte offset of 16-byte chunk `chunk` (8 fp16) of row r in a 128-byte-swizzled block.
__device__ __forceinline__ int swz(int r, int chunk) { return r * 128 + ((chunk ^ (r & 7)) << 4); }

// ---- widening -----------------------------------------------------------------------------------

__device__ __forceinline__ uint32_t hsub2u(uint32_t a, uint32_t b) {
    const __half2 r = __hsub2(*reinterpret_cast<const __half2 *>(&a), *reinterpret_cast<const __half2 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&r);
}

// Four codes -> two fp16 pairs.
template <int FMT>
__device__ __forceinline__ uint2 widen4(uint32_t w) {
    uint2 r;
    if (FMT == W4KV_INT8) {  // 1152 + q as fp16 bits 0x64(q ^ 0x80), then - 1152
        const uint32_t x = w ^ 0x80808080u;
        r.x = hsub2u(__byte_perm(x, 0x64646464u, 0x4140), 0x64806480u);
        r.y = hsub2u(__byte_perm(x, 0x64646464u, 0x4342), 0x64806480u);
    } else {
        asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
            "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
            : "=r"(r.x), "=r"(r.y)
            : "r"(w));
    }
    return r;
}

// Dims in which a token of [lo, hi) has an E4M3 NaN code in its value: bit i of nan[c] for dim 32 c + i.
template <int D>
__device__ __forceinline__ void find_nans(const Attn &a, int b, int h, int lo, int hi, uint32_t (&nan)[D / 32]) {
#pragma unroll 1
    for (int at = lo; at < hi; ++at) {
        const int64_t r = row_of(a.c, a.b, b, at);
        if (r < 0) continue;
        const uint4 *code = reinterpret_cast<const uint4 *>(a.c.v + (r + int64_t(h) * a.c.page) * D);
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
            const uint4 v = __ldg(code + i);
            const uint32_t x[4] = {e4m3_nans(v.x) >> 7, e4m3_nans(v.y) >> 7, e4m3_nans(v.z) >> 7, e4m3_nans(v.w) >> 7};
#pragma unroll
            for (int q = 0; q < 4; ++q)
                nan[i / 2] |= ((x[q] | x[q] >> 7 | x[q] >> 14 | x[q] >> 21) & 15u) << (16 * (i & 1) + 4 * q);
        }
    }
}

// Eight INT4 codes -> u - z in dim order; zb = 1024 + z in both halves.
__device__ __forceinline__ uint4 widen8_int4(uint32_t w, uint32_t zb) {
    uint4 r;
    r.x = hsub2u((w & 0x000F000Fu) | 0x64006400u, zb);
    r.y = hsub2u(((w >> 4) & 0x000F000Fu) | 0x64006400u, zb);
    r.z = hsub2u(((w >> 8) & 0x000F000Fu) | 0x64006400u, zb);
    r.w = hsub2u(((w >> 12) & 0x000F000Fu) | 0x64006400u, zb);
    return r;
}

template <int FMT, int D, int XT>
__global__ void __launch_bounds__(kThreads, 1) tiled_kernel(const Attn a) {
    using L = Layout<FMT, D>;
    constexpr int kRow = L::kRow;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                ~static_cast<uintptr_t>(1023));
    Control *sm = reinterpret_cast<Control *>(base + L::kControl);
    volatile int *abort_flag = &sm->abort_flag;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (threadIdx.x == 0) {
        for (int t = 0; t < 2; ++t) {
            mbar_init(smem_u32(&sm->q_full[t]), kM);
            mbar_init(smem_u32(&sm->s_full[t]), 1);
            mbar_init(smem_u32(&sm->p_full[t]), kM);
            mbar_init(smem_u32(&sm->pv_done[t]), 1);
        }
        for (int i = 0; i < kBuffers; ++i) {
            mbar_init(smem_u32(&sm->full[i]), 32 * kWidenWarps);
            mbar_init(smem_u32(&sm->empty[i]), 2);  // both streams
        }
        for (int i = 0; i < kScaleStages; ++i) {
            mbar_init(smem_u32(&sm->sc_full[i]), 1);
            mbar_init(smem_u32(&sm->sc_empty[i]), 8);
        }
        mbar_init(smem_u32(&sm->joined), 2 * kM);
        sm->abort_flag = 0;
        sm->mma_lock = 0;
        sm->nans = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    const Range range = block_range<kThreads>(a.b.n, &sm->range, [&](int b) -> int64_t {
        const Seq s = load_seq(a, b);
        if (s.n == 0) return 0;
        const int tiles = seq_tiles(a, s);
        int64_t cost = 0;
        for (int t = 0; t < tiles; ++t) cost += kItemCost + tile_units(a, s, t);
        return cost * a.c.heads;
    });
    if (threadIdx.x == 0) a.desc[blockIdx.x] = make_int4(0, 0, 0, 0);
    if (range.start == range.end) return;  // the whole block
    if (warp == 16) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_u32(&sm->tmem)),
                     "n"(kTmemCols));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm->tmem;
    const uint32_t tS = tmem, tO = tmem + 2 * kStep;  // + 128 t

    Walk &w = sm->walk[warp];
    bool more;
    {
        int first = 0;
        if (lane == 0) first = first_segment(a, range, w);
        more = __shfl_sync(0xffffffffu, first, 0) != 0;
        __syncwarp();
    }

    if (warp < 8) {
        // =============================== softmax ===============================
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegSoftmax) : "memory");
        const int t = warp >> 2, row = threadIdx.x & (kM - 1);
        const uint32_t lane_bits = static_cast<uint32_t>(warp & 3) << 21;  // TMEM lane quarter
        const uint32_t s_col = tS + t * kStep + lane_bits, o_col = tO + t * 128 + lane_bits;
        uint32_t step_no = 0, own_no = 0, joins = 0;
        bool ok = true;
        auto join = [&]() {  // both streams' warps, bounded like every wait
            mbar_arrive(smem_u32(&sm->joined));
            ok = __all_sync(0xffffffffu, bar_wait(smem_u32(&sm->joined), joins & 1, abort_flag, a.status));
            ++joins;
        };
        for (; more && ok; more = warp_next(a, &w)) {
            const bool split = w.R <= kM;
            const int r = split ? row : t * kM + row;  // of the item
            const bool live = r < w.R;
            const int rr = w.r0 + r;
            const int token = rr / a.group, head = w.h * a.group + rr - token * a.group;
            // ---- the query row: scaled by a power of two, fp16, swizzled ----
            // D / 8 lanes read a row together; lane i keeps the factor of row i of the warp.
            float fr = 1.f;
            if (own_steps(a, w, t) > 0) {
                constexpr int kLanes = D / 8, kAtOnce = 32 / kLanes, kBatch = 8;
                const int part = lane % kLanes, sub = lane / kLanes;
                uint8_t *qs = base + L::kQ + t * L::kTile + (part >> 3) * L::kBlock;
#pragma unroll 1
                for (int i = 0; i < 32; i += kBatch * kAtOnce) {
                    uint4 v[kBatch];
#pragma unroll
                    for (int q = 0; q < kBatch; ++q) {  // all loads first
                        const int lr = i + q * kAtOnce + sub, x = (row & ~31) + lr + (split ? 0 : t * kM);
                        const int y = w.r0 + x, tok = y / a.group;
                        v[q] = x < w.R ? __ldg(reinterpret_cast<const uint4 *>(
                                                   a.q + int64_t(w.s.row0 + tok) * a.q_row +
                                                   (w.h * a.group + y - tok * a.group) * a.q_head) + part)
                                       : make_uint4(0, 0, 0, 0);
                    }
#pragma unroll
                    for (int q = 0; q < kBatch; ++q) {
                        const int lr = i + q * kAtOnce + sub;
                        const uint32_t x = __vmaxu2(__vmaxu2(v[q].x & 0x7FFF7FFFu, v[q].y & 0x7FFF7FFFu),
                                                    __vmaxu2(v[q].z & 0x7FFF7FFFu, v[q].w & 0x7FFF7FFFu));
                        uint32_t top = max(x & 0xFFFFu, x >> 16);
#pragma unroll
                        for (int o = 1; o < kLanes; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
                        int sh = 0;  // the row times 2^sh has its largest element in [2^4, 2^5)
                        const uint32_t t32 = __float_as_uint(widen1<XT>(static_cast<uint16_t>(top)));
                        if (t32 != 0 && t32 < 0x7F800000u) sh = min(120, 131 - static_cast<int>(t32 >> 23));
                        const float up = pow2i(sh);
                        float e[8];
                        widen8<XT>(v[q], e);
                        uint32_t h[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const __half2 p = __floats2half2_rn(e[2 * j] * up, e[2 * j + 1] * up);
                            h[j] = *reinterpret_cast<const uint32_t *>(&p);
                        }
                        *reinterpret_cast<uint4 *>(qs + swz((row & ~31) + lr, part & 7)) = make_uint4(h[0], h[1], h[2], h[3]);
#pragma unroll
                        for (int o = 0; o < kAtOnce; ++o) {
                            const int s2 = __shfl_sync(0xffffffffu, sh, o * kLanes);
                            if (lane == i + q * kAtOnce + o) fr = pow2i(-s2);
                        }
                    }
                }
                fence_proxy_async();
                mbar_arrive(smem_u32(&sm->q_full[t]));
            }
            // ---- what the row sees: [clo, chi); what all rows of the warp see: [all_lo, all_hi) ----
            const int pos = w.s.first + token;
            int clo = w.lo, chi = w.hi;
            if (a.window > 0) clo = max(clo, window_from(pos, a.window));
            if (a.causal) chi = min(chi, pos + 1);
            if (!live) clo = w.lo, chi = w.hi;
            clo = max(clo, w.s.lo);
            const int all_lo = __reduce_max_sync(0xffffffffu, clo);
            const int all_hi = __reduce_min_sync(0xffffffffu, chi);
            const bool any_live = __any_sync(0xffffffffu, live);

            float m = kNone, l = 0.f;
            // Weights are p * scale * 2^(133 - e), e the exponent field of the largest value scale
            // that the row has seen (at least 7): vcur, or row_vexp where that is -1.
            int vcur = 7, own = 0;
            const int ns = w.u1 - w.u0, mine = stream_steps(a, w, t), kv_base = w.lo + w.u0 * kStep;
            for (int j = 0; j < ns && ok; ++j, ++step_no) {
                const int sc = step_no % kScaleStages;
                ok = __all_sync(0xffffffffu, bar_wait(smem_u32(&sm->sc_full[sc]),
                                                       (step_no / kScaleStages) & 1, abort_flag, a.status));
                if (!ok) break;
                if (split ? (j & 1) == t : j < mine) {
                    ok = __all_sync(0xffffffffu, bar_wait(smem_u32(&sm->s_full[t]), own_no & 1, abort_flag, a.status));
                    if (!ok) break;
                    tc_fence_after();
                    if (any_live) {
                        const int kv0 = kv_base + j * kStep;
                        const uint32_t bad = sm->bad[sc];
                        const bool cut = bad != 0 || kv0 < all_lo || kv0 + kStep > all_hi;
                        auto seen = [&](int c) {  // bits of the 16 tokens from kv0 + 16 c
                            const int lo = clo - (kv0 + 16 * c), hi = chi - (kv0 + 16 * c);
                            if (lo >= 16 || hi <= 0 || ((bad >> c) & 1)) return 0u;
                            return (0xFFFFu << max(lo, 0)) & (0xFFFFu >> (16 - min(hi, 16)));
                        };
                        const ulonglong2 *ks2 = reinterpret_cast<const ulonglong2 *>(sm->ks[sc]);
                        const ulonglong2 *vs2 = reinterpret_cast<const ulonglong2 *>(sm->vs[sc]);
                        const uint64_t fr2 = pack2(fr, fr);
                        // Eight pairs of scores over m, of the chunk being loaded; then `next`.
                        auto bases = [&](uint32_t (&s)[16], int c, uint64_t (&y)[8], auto next) {
                            ulonglong2 k[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i) k[i] = ks2[4 * c + i];
                            const uint64_t m2 = pack2(-m, -m);
                            tmem_wait_ld16(s);
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                y[2 * i] = fma2(mul2(pack2(__uint_as_float(s[4 * i]), __uint_as_float(s[4 * i + 1])), k[i].x), fr2, m2);
                                y[2 * i + 1] = fma2(mul2(pack2(__uint_as_float(s[4 * i + 2]), __uint_as_float(s[4 * i + 3])), k[i].y), fr2, m2);
                            }
                            next();
                        };
                        // Eight pairs of scores over m -> weights; the unscaled ones' sum to l2.
                        // g: the row's reference over the step's, where they may differ.
                        auto weights = [&](const uint64_t (&y)[8], int c, uint64_t &l2, uint32_t (&p)[8], auto g) {
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                ulonglong2 v = vs2[4 * c + i];
                                if constexpr (std::is_same_v<decltype(g), float>)
                                    v.x = mul2(v.x, pack2(g, g)), v.y = mul2(v.y, pack2(g, g));
                                const float2 y0 = unpack2(y[2 * i]), y1 = unpack2(y[2 * i + 1]);
                                const uint64_t p0 = pack2(ex2(y0.x), ex2(y0.y)), p1 = pack2(ex2(y1.x), ex2(y1.y));
                                l2 = add2(l2, p0);
                                l2 = add2(l2, p1);
                                const float2 w0 = unpack2(mul2(p0, v.x)), w1 = unpack2(mul2(p1, v.y));
                                const __half2 h0 = __floats2half2_rn(w0.x, w0.y), h1 = __floats2half2_rn(w1.x, w1.y);
                                p[2 * i] = *reinterpret_cast<const uint32_t *>(&h0);
                                p[2 * i + 1] = *reinterpret_cast<const uint32_t *>(&h1);
                            }
                        };
                        // O, and P's first `cols` columns, times f.
                        auto rescale = [&](float f, int cols) {
                            if (own > 0) {
                                if (!__all_sync(0xffffffffu, bar_wait(smem_u32(&sm->pv_done[t]), (own_no - 1) & 1,
                                                                      abort_flag, a.status)))
                                    return false;
                                tc_fence_after();
#pragma unroll 1
                                for (int c = 0; c < D / 16; ++c) {
                                    uint32_t o[16];
                                    tmem_ld16(o_col + 16 * c, o);
                                    tmem_wait_ld16(o);
#pragma unroll
                                    for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                                    tmem_st16(o_col + 16 * c, o);
                                }
                            }
                            tmem_wait_st();
#pragma unroll 1
                            for (int c = 0; c < cols; c += 8) {
                                uint32_t p[8];
                                tmem_ld8(s_col + c, p);
                                tmem_wait_ld8(p);
#pragma unroll
                                for (int i = 0; i < 8; ++i) {  // (in fp32: f may be below fp16's range)
                                    const float2 x = __half22float2(*reinterpret_cast<const __half2 *>(&p[i]));
                                    const __half2 y = __floats2half2_rn(x.x * f, x.y * f);
                                    p[i] = *reinterpret_cast<const uint32_t *>(&y);
                                }
                                tmem_st8(s_col + c, p);
                            }
                            tmem_wait_st();
                            return true;
                        };
                        // The value scales' reference moves with the step's, or where that is none with
                        // what each row sees.  (One reference for all rows would let tokens that a
                        // row does not see shift its weights out of fp16's range.)
                        const int ve = sm->vexp[sc];
                        bool own_ref = false;  // rows' references differ from the step's
                        if (ve != vcur || ve < 0) {
                            const int old = vcur < 0 ? sm->row_vexp[t][row] : vcur;
                            int e = max(old, abs(ve));
                            if (ve < 0) {
#pragma unroll 1
                                for (int c = 0; c < 8; ++c) {
                                    const uint32_t bits = live ? seen(c) : 0u;
                                    if (bits == 0xFFFFu) e = max(e, static_cast<int>(sm->vgroup[sc][c]));
                                    if (__any_sync(0xffffffffu, bits != 0u && bits != 0xFFFFu)) {
#pragma unroll
                                        for (int i = 0; i < 16; ++i) {
                                            const int x = (__float_as_uint(sm->vs[sc][16 * c + i]) >> 23) & 255;
                                            if (((bits >> i) & 1) && x != 255) e = max(e, x);
                                        }
                                    }
                                }
                            }
                            if (__any_sync(0xffffffffu, e != old)) {
                                ok = rescale(pow2i(max(-126, old - e)), 0);
                                if (!ok) break;
                            }
                            const int first = __shfl_sync(0xffffffffu, e, 0);
                            vcur = __all_sync(0xffffffffu, !live || e == first) ? first : -1;
                            sm->row_vexp[t][row] = e;
                            own_ref = ve < 0 || vcur != ve;
                        }
                        if (__any_sync(0xffffffffu, m == kNone)) {
                            // Rows that have seen nothing yet start from their largest score.
                            float top = -INFINITY;
#pragma unroll 1
                            for (int c = 0; c < 8; ++c) {
                                uint32_t s[16];
                                tmem_ld16(s_col + 16 * c, s);
                                tmem_wait_ld16(s);
                                float x[16];
#pragma unroll
                                for (int i = 0; i < 4; ++i) {
                                    const float4 k = reinterpret_cast<const float4 *>(sm->ks[sc])[4 * c + i];
                                    x[4 * i] = __uint_as_float(s[4 * i]) * k.x;
                                    x[4 * i + 1] = __uint_as_float(s[4 * i + 1]) * k.y;
                                    x[4 * i + 2] = __uint_as_float(s[4 * i + 2]) * k.z;
                                    x[4 * i + 3] = __uint_as_float(s[4 * i + 3]) * k.w;
                                }
                                if (cut) {
                                    const uint32_t bits = seen(c);
#pragma unroll
                                    for (int i = 0; i < 16; ++i) x[i] = (bits >> i) & 1 ? x[i] : -INFINITY;
                                }
#pragma unroll
                                for (int i = 0; i < 8; ++i) x[i] = fmaxf(x[i], x[i + 8]);
#pragma unroll
                                for (int i = 0; i < 4; ++i) x[i] = fmaxf(x[i], x[i + 4]);
                                top = fmaxf(top, fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])));
                                __syncwarp();
                            }
                            if (m == kNone) m = fmaxf(m, top * fr);
                        }
                        // One pass with the maximum as it is, where the warp's rows see the whole step and
                        // have its reference.
                        float lsum = 0.f;
                        int c0 = 0;  // chunks of 16 tokens done
                        if (!cut && !own_ref) {
                            uint32_t s[16];
                            tmem_ld16(s_col, s);
#pragma unroll
                            for (int c = 0; c < 8; ++c) {
                                uint64_t y[8], l2 = 0;
                                uint32_t p[8];
                                bases(s, c, y, [&] {
                                    if (c < 7) tmem_ld16(s_col + 16 * (c + 1), s);
                                });
                                weights(y, c, l2, p, std::false_type());
                                const float sum = unpack2(l2).x + unpack2(l2).y;
                                if (__any_sync(0xffffffffu, sum > 256.f)) {  // seldom
                                    if (c < 7) tmem_wait_ld16(s);
                                    break;
                                }
                                lsum += sum;
                                tmem_st8(s_col + 8 * c, p);
                                c0 = c + 1;
                            }
                        }
                        // The rest, and steps with masks or references of the rows' own.  Where a score
                        // exceeds the maximum by more than 2^8, it moves by a whole number, so that what
                        // is done already (sums, weights, O) is rescaled exactly; from far below (where
                        // that leaves nothing of it) to the largest score itself, whose distance has few
                        // bits for the fraction.  (A sum of weights up to 2^8 has none above it.)
                        if (c0 < 8) {
                            const float g = own_ref ? pow2i(max(-126, (ve < 0 ? 133 : ve) - sm->row_vexp[t][row])) : 1.f;
                            int tries = 0;
                            bool far = false;
#pragma unroll 1
                            for (int c = c0; c < 8; ++c) {
                                uint32_t s[16];
                                tmem_ld16(s_col + 16 * c, s);
                                uint64_t y[8], l2 = 0;
                                uint32_t p[8];
                                bases(s, c, y, [] {});
                                const uint32_t bits = seen(c);
#pragma unroll
                                for (int i = 0; i < 8; ++i) {
                                    const float2 z = unpack2(y[i]);
                                    y[i] = pack2((bits >> (2 * i)) & 1 ? z.x : -INFINITY,
                                                 (bits >> (2 * i)) & 2 ? z.y : -INFINITY);
                                }
                                weights(y, c, l2, p, g);
                                const float sum = unpack2(l2).x + unpack2(l2).y;
                                if (__any_sync(0xffffffffu, far || sum > 256.f) && tries < 4) {
                                    float top = kNone;
#pragma unroll
                                    for (int i = 0; i < 8; ++i) top = fmaxf(top, fmaxf(unpack2(y[i]).x, unpack2(y[i]).y));
                                    const bool over = !far && sum > 256.f;
                                    const float up = over ? ceilf(top) : 0.f, f = ex2(-up);
                                    m = far ? top : m + up;
                                    far = up >= 1024.f;
                                    if (far) m = 0.f;  // the chunk's bases are its scores then
                                    l *= f;
                                    lsum *= f;
                                    ok = rescale(f, 8 * c);
                                    if (!ok) break;
                                    ++tries;
                                    --c;  // the chunk again
                                    continue;
                                }
                                tries = 0;
                                // unseen: exactly zero, whatever the value row's scale is
#pragma unroll
                                for (int i = 0; i < 8; ++i) {
                                    const uint32_t two = (bits >> (2 * i)) & 3u;
                                    p[i] &= (two & 1u ? 0xFFFFu : 0u) | (two & 2u ? 0xFFFF0000u : 0u);
                                }
                                lsum += sum;
                                __syncwarp();
                                tmem_st8(s_col + 8 * c, p);
                            }
                        }
                        l += lsum;
                        if (!ok) break;
                        tmem_wait_st();
                    }
                    tc_fence_before();
                    mbar_arrive(smem_u32(&sm->p_full[t]));
                    ++own;
                    ++own_no;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&sm->sc_empty[sc]));
            }
            if (!ok) break;
            // ---- the result ----
            if (own > 0) {
                ok = __all_sync(0xffffffffu, bar_wait(smem_u32(&sm->pv_done[t]), (own_no - 1) & 1, abort_flag, a.status));
                if (!ok) break;
                tc_fence_after();
            }
            const bool from_start = w.u0 == 0, to_end = w.u1 == w.nu, whole = from_start && to_end;
            float *slot = a.slots + (2 * int64_t(blockIdx.x) + (from_start ? 1 : 0)) * slot_floats(kTileRows, D);
            if (!whole && from_start && threadIdx.x == 0) {
                const int64_t last = range.end - w.rem + (w.nu - w.u1) - 1;  // its last unit
                a.desc[blockIdx.x] = make_int4(w.b, w.h, block_of_unit(last, range) - static_cast<int>(blockIdx.x) + 1, w.tile);
            }
            float M = m, Lsum = l, weight;
            float *joined = reinterpret_cast<float *>(base + L::kQ);  // [D][128], over both query tiles
            if (split) {
                sm->stat[t][0][row] = m;
                sm->stat[t][1][row] = l;
                join();
                if (!ok) break;
                const float m2 = sm->stat[1 - t][0][row], l2 = sm->stat[1 - t][1][row];
                M = fmaxf(m, m2);
                Lsum = l * ex2(m - M) + l2 * ex2(m2 - M);
                weight = Lsum == 0.f ? 0.f : ex2(m - M) / Lsum;
            } else {
                weight = l == 0.f ? 0.f : 1.f / l;
            }
            uint32_t nan[D / 32] = {};
            if (FMT == W4KV_E4M3 && __any_sync(0xffffffffu, own > 0 && *static_cast<volatile int *>(&sm->nans))) {
                int all_lo, all_hi;  // outside them, to multiples of 16, NaN codes count as zeros in the MMAs
                common_bounds(a, w, &all_lo, &all_hi);
                const int from = max(clo, kv_base), to = min(chi, kv_base + ns * kStep);
                all_lo = (all_lo + 15) & ~15;
                all_hi = max(all_lo, all_hi & ~15);
                if (live) {
                    find_nans<D>(a, w.b, w.h, from, min(to, all_lo), nan);
                    find_nans<D>(a, w.b, w.h, max(from, all_hi), to, nan);
                }
                __syncwarp();
            }
            const float vback = pow2i((vcur < 0 ? sm->row_vexp[t][row] : vcur) - 133);
            auto value = [&](int d, uint32_t o) {
                if (FMT == W4KV_E4M3 && ((nan[d / 32] >> (d % 32)) & 1)) return __uint_as_float(0x7FC00000u);
                return __uint_as_float(o) * weight * vback;
            };
            auto output = [&](auto add) {  // the row's normalized output, in chunks of 32 dims
#pragma unroll
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t o[32];
                    if (own > 0) {
                        tmem_ld32(o_col + 32 * c, o);
                        tmem_wait_ld32(o);
                    }
                    float x[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        x[i] = add(32 * c + i, own > 0 ? value(32 * c + i, o[i]) : 0.f);
                    if (live && whole) {
                        uint16_t *op = a.o + int64_t(w.s.row0 + token) * a.o_row + head * a.o_head + 32 * c;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            uint32_t h[4];
#pragma unroll
                            for (int q = 0; q < 4; ++q)
                                h[q] = narrow1<XT>(x[8 * i + 2 * q]) |
                                       static_cast<uint32_t>(narrow1<XT>(x[8 * i + 2 * q + 1])) << 16;
                            reinterpret_cast<uint4 *>(op)[i] = make_uint4(h[0], h[1], h[2], h[3]);
                        }
                    } else if (live) {
                        // four dims of a row after another, rows side by side
                        float4 *sp = reinterpret_cast<float4 *>(slot + 2 * kTileRows) + 8 * c * kTileRows + r;
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            sp[i * kTileRows] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
                    }
                    __syncwarp();
                }
                if (live) {
                    if (!whole) {
                        slot[r] = M;
                        slot[kTileRows + r] = Lsum;
                    } else if (a.lse) {
                        a.lse[int64_t(w.s.row0 + token) * a.heads + head] =
                            Lsum == 0.f ? -INFINITY : (M + log2f(Lsum)) * 0.6931471805599453f;
                    }
                }
            };
            if (!split) {
                output([](int, float x) { return x; });
            } else {
                if (t == 1) {
#pragma unroll
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t o[32];
                        if (own > 0) {
                            tmem_ld32(o_col + 32 * c, o);
                            tmem_wait_ld32(o);
                        }
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            joined[(32 * c + i) * kM + row] = own > 0 ? value(32 * c + i, o[i]) : 0.f;
                    }
                }
                join();
                if (!ok) break;
                if (t == 0) output([&](int d, float x) { return x + joined[d * kM + row]; });
                join();  // before the next item's queries
            }
            tc_fence_before();
        }
    } else if (warp < 8 + kWidenWarps) {
        // =============================== widening ===============================
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegWiden) : "memory");
        // A warp serves 16 rows of every tile: one page, and one run of bytes in it.
        // It copies them (cp.async) kRawTiles tiles ahead, and reads page numbers one
        // step before that.
        const int wr = (warp - 8) * 16;  // its first row
        uint8_t *ring = base + L::kRaw + (warp - 8) * L::kRawWarp;
        int pj = 0, id = -1, kv0 = 0, hi = 0, lo = 0, h = 0;
        int all_lo = 0, all_hi = 0;  // positions that all rows of the item see
        uint32_t part_mask = 0;      // per tile on its way: values that not all rows see
        bool fetched = more;  // a step's page number is at hand
        auto fetch_page = [&]() {
            kv0 = w.lo + (w.u0 + pj) * kStep + wr;
            lo = w.s.lo, hi = w.hi, h = w.h;
            if (FMT == W4KV_E4M3 && pj == 0) common_bounds(a, w, &all_lo, &all_hi);
            int rest;
            const int pg = page_of_tile(a, kv0 >> 4, &rest);
            id = pg < a.b.width && kv0 < hi ? __ldg(a.b.table + w.b * a.b.stride + pg) : -1;
            if (++pj == w.u1 - w.u0) {
                pj = 0;
                more = warp_next(a, &w);
            }
        };
        uint32_t issued = 0;  // tiles
        int put = 0;
        auto issue = [&]() {  // the next tile: K of a step, then its V
            if (fetched) {
                const bool is_v = issued & 1;
                const uint32_t dst = smem_u32(ring + put * L::kRawTile);
                const bool live = static_cast<uint32_t>(id) < static_cast<uint32_t>(a.c.pages);
                int rest;
                page_of_tile(a, kv0 >> 4, &rest);
                const int64_t rr = live ? (int64_t(id) * a.c.heads + h) * a.c.page + rest * 16 : 0;
                const uint8_t *src = (is_v ? a.c.v : a.c.k) + rr * kRow + lane * 16;
                const int v0 = live ? lo - kv0 : 16, v1 = hi - kv0;  // rows in use
#pragma unroll
                for (int i = 0; i < (kRow + 31) / 32; ++i) {  // 512 bytes each
                    const int row = (lane * 16 + i * 512) / kRow;
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + lane * 16 + i * 512),
                                 "l"(src + i * 512), "r"(row >= v0 && row < v1 ? 16 : 0) : "memory");
                }
                if (FMT == W4KV_INT4 && lane < 16)
                    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst + 16 * kRow + lane * 4),
                                 "l"((is_v ? a.c.vs : a.c.ks) + rr + lane), "r"(lane >= v0 && lane < v1 ? 4 : 0) : "memory");
                ++issued;
                if (FMT == W4KV_E4M3) {
                    const bool part = is_v && (kv0 < all_lo || kv0 + 16 > all_hi);
                    part_mask = (part_mask & ~(1u << put)) | static_cast<uint32_t>(part) << put;
                }
                if (is_v) {
                    fetched = more;
                    if (fetched) fetch_page();
                }
            }
            put = put + 1 == L::kRawTiles ? 0 : put + 1;
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        if (fetched) fetch_page();
        for (int i = 0; i < L::kRawTiles; ++i) issue();
        // Eight codes make one 16-byte chunk; the lanes of a phase write the chunks of
        // one row, which lie in different banks.
        constexpr int kRowChunks = D / 8, kRowsAtOnce = 32 / kRowChunks, kN = 16 / kRowsAtOnce;
        const int chunk = lane % kRowChunks, r0 = lane / kRowChunks;
        const int st_off = (chunk >> 3) * L::kBlock;
        int get = 0;
        uint32_t buf = 0, phase = 1;
        for (uint32_t n = 0; n < issued; ++n) {
            asm volatile("cp.async.wait_group %0;" ::"n"(L::kRawTiles - 1) : "memory");
            __syncwarp();
            const uint8_t *src = ring + get * L::kRawTile;
            // A weight of zero times a NaN is a NaN: among values that not all rows see, NaN codes
            // count as zeros, and the softmax warps look which rows see them at the item's end.
            if (FMT == W4KV_E4M3 && ((part_mask >> get) & 1))
                zero_nans(reinterpret_cast<uint32_t *>(ring + get * L::kRawTile) + lane, 16 * kRow, &sm->nans);
            uint2 raw[kN];
            uint32_t z[kN];
#pragma unroll
            for (int i = 0; i < kN; ++i) {
                const int row = r0 + i * kRowsAtOnce;
                if (FMT == W4KV_INT4) {
                    raw[i].x = *reinterpret_cast<const uint32_t *>(src + row * kRow + chunk * 4);
                    z[i] = *reinterpret_cast<const uint32_t *>(src + 16 * kRow + row * 4);
                } else {
                    raw[i] = *reinterpret_cast<const uint2 *>(src + row * kRow + chunk * 8);
                }
            }
            get = get + 1 == L::kRawTiles ? 0 : get + 1;
            __syncwarp();
            issue();
            if (!__all_sync(0xffffffffu, bar_wait(smem_u32(&sm->empty[buf]), phase, abort_flag, a.status))) break;
            uint8_t *tile = base + L::kKV + buf * L::kTile + st_off + wr * 128;
#pragma unroll
            for (int i = 0; i < kN; ++i) {
                uint4 x;
                if (FMT == W4KV_INT4) {
                    x = widen8_int4(raw[i].x, 0x64006400u | (z[i] & 15u) * 0x10001u);
                } else {
                    const uint2 h0 = widen4<FMT>(raw[i].x), h1 = widen4<FMT>(raw[i].y);
                    x = make_uint4(h0.x, h0.y, h1.x, h1.y);
                }
                *reinterpret_cast<uint4 *>(tile + swz(r0 + i * kRowsAtOnce, chunk & 7)) = x;
            }
            fence_proxy_async();
            mbar_arrive(smem_u32(&sm->full[buf]));
            if (++buf == kBuffers) {
                buf = 0;
                phase ^= 1;
            }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
    } else {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegRest) : "memory");
      if (warp < 18) {
        // =============================== MMA ===============================
        // One warp per stream, so that the waits and commits of one (100 cycles
        // and more each) pass while the other's MMAs run.  The whole warp walks,
        // one elected thread issues.
        const int t = warp - 16;
        constexpr uint32_t id_s = instr_desc<kStep, false>(), id_o = instr_desc<D, true>();
        const uint32_t q = desc_low(smem_u32(base + L::kQ + t * L::kTile), 16);
        const uint32_t k0 = desc_low(smem_u32(base + L::kKV), 16);
        const uint32_t v0 = desc_low(smem_u32(base + L::kKV), L::kBlock);
        const uint32_t d_s = tS + t * kStep, d_o = tO + t * 128;
        uint32_t step0 = 0, n_q = 0, n_p = 0;
        bool ok = true;
        auto wait = [&](uint64_t *bar, uint32_t parity) {
            ok = __all_sync(0xffffffffu, ok && bar_wait(smem_u32(bar), parity, abort_flag, a.status));
            return ok;
        };
        for (; more && ok; more = warp_next(a, &w)) {
            const bool split = w.R <= kM;
            const int ns = w.u1 - w.u0, mine = stream_steps(a, w, t);
            if (own_steps(a, w, t) > 0 && !wait(&sm->q_full[t], n_q++ & 1)) break;
            auto filled = [&](uint32_t n) { return wait(&sm->full[n % kBuffers], (n / kBuffers) & 1); };
            auto let_go = [&](uint32_t n) {
                if (lane == 0) mbar_arrive(smem_u32(&sm->empty[n % kBuffers]));
            };
            auto score = [&](uint32_t n) {  // S from the keys in tile n (one thread)
                const uint32_t k = k0 + (n % kBuffers) * (L::kTile >> 4);
#pragma unroll
                for (int x = 0; x < D / 16; ++x) {
                    const uint32_t off = ((x / 4) * L::kBlock + (x % 4) * 32) >> 4;
                    mma_ss(d_s, q + off, k + off, id_s, x > 0);
                }
                mma_commit(smem_u32(&sm->s_full[t]));
                mma_commit(smem_u32(&sm->empty[n % kBuffers]));
            };
            auto output = [&](uint32_t n, bool first) {  // O from the values in tile n (one thread)
                const uint32_t v = v0 + (n % kBuffers) * (L::kTile >> 4);
#pragma unroll
                for (int x = 0; x < kStep / 16; ++x)
                    mma_ts(d_o, d_s + 8 * x, v + x * (2048 >> 4), id_o, !(first && x == 0));
                mma_commit(smem_u32(&sm->pv_done[t]));
                mma_commit(smem_u32(&sm->empty[n % kBuffers]));
            };
            // Tiles are taken, or let go, in the order they are widened.
            if (split) {
                bool first = true;
                for (int j = 0; j < ns && ok; ++j) {
                    const bool own = (j & 1) == t;
                    const uint32_t n = 2 * (step0 + j);
                    if (!filled(n)) break;
                    if (!own) {
                        let_go(n);
                    } else {
                        tc_fence_after();
                        if (elect_one()) score(n);
                        __syncwarp();
                    }
                    if (!filled(n + 1)) break;
                    if (!own) {
                        let_go(n + 1);
                    } else {
                        if (!wait(&sm->p_full[t], n_p++ & 1)) break;
                        tc_fence_after();
                        if (elect_one()) output(n + 1, first);
                        __syncwarp();
                        first = false;
                    }
                }
            } else {
                // O(j) and S(j + 1) go to the tensor cores together: the streams' MMAs do
                // not mix, so that the first one's softmax starts while the other's run.
                if (mine > 0) {
                    if (!filled(2 * step0)) break;
                    tc_fence_after();
                    if (elect_one()) score(2 * step0);
                    __syncwarp();
                }
                for (int j = 0; j < mine && ok; ++j) {
                    const uint32_t n = 2 * (step0 + j) + 1;
                    const bool next = j + 1 < mine;
                    if (!filled(n) || (next && !filled(n + 1))) break;
                    if (!wait(&sm->p_full[t], n_p++ & 1)) break;
                    tc_fence_after();
                    if (elect_one()) {
                        lock(&sm->mma_lock, abort_flag, a.status);
                        output(n, j == 0);
                        if (next) score(n + 1);
                        unlock(&sm->mma_lock);
                    }
                    __syncwarp();
                }
                for (int j = mine; j < ns && ok; ++j) {  // steps that tile A does not see
                    if (!filled(2 * (step0 + j))) break;
                    let_go(2 * (step0 + j));
                    if (!filled(2 * (step0 + j) + 1)) break;
                    let_go(2 * (step0 + j) + 1);
                }
            }
            step0 += ns;
        }
      } else if (warp == 18) {
        // =============================== scales ===============================
        // Page numbers are read one step before the words' copies are issued, and
        // those (cp.async, each lane its own words) kScaleAhead steps before use.
        int pj = 0, kv0 = 0, lo = 0, hi = 0, h = 0, id[4];
        uint32_t vexp = 7, flags = 0;
        int all_lo = 0, all_hi = 0;  // positions that all rows of the item see
        bool fetched = more;  // a step's page numbers are at hand
        uint32_t issued = 0;
        auto fetch_pages = [&]() {
            kv0 = w.lo + (w.u0 + pj) * kStep, lo = w.s.lo, hi = w.hi, h = w.h;
            flags = 0;
            if (pj == 0) {
                flags = kOpens;
                common_bounds(a, w, &all_lo, &all_hi);
            }
            flags |= static_cast<uint32_t>(min(max(all_lo - kv0, 0), kStep)) << kFrom;
            flags |= static_cast<uint32_t>(min(max(all_hi - kv0, 0), kStep)) << kTo;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int tile = (kv0 + 32 * i + lane) >> 4;
                int rest;
                const int pg = page_of_tile(a, tile, &rest);
                id[i] = pg < a.b.width && tile * 16 < hi ? __ldg(a.b.table + w.b * a.b.stride + pg) : -1;
            }
            if (++pj == w.u1 - w.u0) {
                pj = 0;
                more = warp_next(a, &w);
            }
        };
        auto issue = [&]() {
            if (fetched) {
                const int rs = issued++ % (kScaleAhead + 1);
                uint32_t badbits = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int at = kv0 + 32 * i + lane;
                    int rest;
                    page_of_tile(a, at >> 4, &rest);
                    const bool good = static_cast<uint32_t>(id[i]) < static_cast<uint32_t>(a.c.pages);
                    const uint32_t b = __ballot_sync(0xffffffffu, !good && (at & ~15) < hi);
                    badbits |= ((b & 1u) | (b >> 31 << 1)) << (2 * i);
                    const int n = good && at >= lo && at < hi ? 4 : 0;  // else a word of zeros
                    const int64_t rr = n ? (int64_t(id[i]) * a.c.heads + h) * a.c.page + rest * 16 + (at & 15) : 0;
                    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(
                                     smem_u32(&sm->word[rs][0][32 * i + lane])), "l"(a.c.ks + rr), "r"(n) : "memory");
                    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(
                                     smem_u32(&sm->word[rs][1][32 * i + lane])), "l"(a.c.vs + rr), "r"(n) : "memory");
                }
                if (lane == 0) sm->word_info[rs] = badbits | flags;
                fetched = more;
                if (fetched) fetch_pages();
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        if (fetched) fetch_pages();
        for (int i = 0; i < kScaleAhead; ++i) issue();
        for (uint32_t step_no = 0;; ++step_no) {
            issue();
            if (step_no == issued) break;  // all steps are done
            const int sc = step_no % kScaleStages, rs = step_no % (kScaleAhead + 1);
            asm volatile("cp.async.wait_group %0;" ::"n"(kScaleAhead) : "memory");
            __syncwarp();
            const uint32_t info = sm->word_info[rs];
            const int from = (info >> kFrom) & 255u, to = (info >> kTo) & 255u;
            uint32_t kw[4], vw[4], e[4], top = 7, common = 7;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                kw[i] = sm->word[rs][0][32 * i + lane];
                vw[i] = sm->word[rs][1][32 * i + lane];
                e[i] = (vw[i] >> 23) & 255u;
                if (e[i] == 255u) e[i] = 0;
                top = max(top, e[i]);
                if (32 * i + lane >= from && 32 * i + lane < to) common = max(common, e[i]);
            }
            vexp = max(info & kOpens ? 7u : vexp, __reduce_max_sync(0xffffffffu, common));
            const bool own_ref = __reduce_max_sync(0xffffffffu, top) > vexp;
            const float vmul = own_ref ? 1.f : pow2i(133 - static_cast<int>(vexp));
            if (own_ref) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int o = 1; o < 16; o <<= 1) e[i] = max(e[i], __shfl_xor_sync(0xffffffffu, e[i], o));
            }
            if (!__all_sync(0xffffffffu, bar_wait(smem_u32(&sm->sc_empty[sc]),
                                                   ((step_no / kScaleStages) & 1) ^ 1, abort_flag, a.status)))
                break;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float k = FMT == W4KV_INT4 ? int4_scale(kw[i]) : __uint_as_float(kw[i]);
                const float v = FMT == W4KV_INT4 ? int4_scale(vw[i]) : __uint_as_float(vw[i]);
                sm->ks[sc][32 * i + lane] = k * a.scale_log2;
                sm->vs[sc][32 * i + lane] = v * vmul;
                if ((lane & 15) == 0) sm->vgroup[sc][2 * i + (lane >> 4)] = static_cast<uint8_t>(e[i]);
            }
            if (lane == 0) {
                sm->vexp[sc] = own_ref ? -static_cast<int>(vexp) : static_cast<int>(vexp);
                sm->bad[sc] = info & 255u;
                if (info & 255u) atomicOr(a.status, kStatusBounds);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sm->sc_full[sc]));
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
      }
    }
    // MMAs in flight are waited for by the softmax warps (pv_done of the last
    // step); after an abort nothing reads them, and the wait below is bounded.
    if (*abort_flag && warp == 16 && lane == 0) {
        const unsigned long long t0 = globaltimer();
        while (globaltimer() - t0 < 1000000ull) {
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 16) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(kTmemCols));
    }
}

template <int FMT, int D, int XT>
int run(const Attn &a, int grid, cudaStream_t stream) {
    auto kernel = tiled_kernel<FMT, D, XT>;
    static std::atomic<unsigned long long> ready{0};  // a bit per device
    const int st = allow_smem(reinterpret_cast<const void *>(kernel), Layout<FMT, D>::kSmem, &ready);
    if (st != W4_OK) return st;
    kernel<<<grid, kThreads, Layout<FMT, D>::kSmem, stream>>>(a);
    return cuda_status(cudaGetLastError());
}

template <int FMT, int D>
int run_x(const Attn &a, int xt, int grid, cudaStream_t s) {
    return xt == W4_F16 ? run<FMT, D, W4_F16>(a, grid, s) : run<FMT, D, W4_BF16>(a, grid, s);
}

}  // namespace

int launch_tiled_attention(const Attn &a, int fmt, int dim, int xt, int grid, cudaStream_t stream) {
    if (dim == 64) {
        if (fmt == W4KV_INT8) return run_x<W4KV_INT8, 64>(a, xt, grid, stream);
        if (fmt == W4KV_E4M3) return run_x<W4KV_E4M3, 64>(a, xt, grid, stream);
        return run_x<W4KV_INT4, 64>(a, xt, grid, stream);
    }
    if (fmt == W4KV_INT8) return run_x<W4KV_INT8, 128>(a, xt, grid, stream);
    if (fmt == W4KV_E4M3) return run_x<W4KV_E4M3, 128>(a, xt, grid, stream);
    return run_x<W4KV_INT4, 128>(a, xt, grid, stream);
}

}  // namespace kv
}  // namespace w4
