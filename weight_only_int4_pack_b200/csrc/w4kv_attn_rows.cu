// w4kv_attn_rows.cu -- attention of few rows over the quantized cache: decode
// steps and short proposals, up to 64 (row, query head) pairs per key/value
// head, in tiles of 8 or 16.
//
// Mathematics: one pass over the cache with a running maximum m, sum l and
// output O per row; a score is q . codes times the key row's scale, a weight
// is p = 2^(score - m) times the value row's scale.  The codes enter the MMAs
// exactly: INT8 and E4M3 are fp16 numbers, and so are u - z and 16 (u - z) of
// INT4, which saves half of the shifts.  (The fp16 subnormals u * 2^-24, with the
// zero points taken off the sums, would save the subtraction, but the MMA aligns
// them as if they were 2^-14: errors of 2^-14 of the largest product.)  m moves
// only when a score exceeds it by 8 (2^8 in the weights), so that O is rarely
// rescaled; p <= 2^8 then, and the value scales are taken relative to 2^k > the
// running maximum / 2^7 of those that the row sees, so that a weight fits fp16
// (below 2^15) with 21 bits of range under the largest one.
//
// HBM bounds it: a token of a head is 2 (dim + 4) bytes (INT8) and a few
// thousand multiplications.  The layout keeps the shared-memory and register
// work off that path:
//   * S^T = K Q^T and O^T = V^T P^T with mma.sync m16n8k16, cached tokens (or
//     dims) as the 16 rows and query rows as the 8 columns: a decode step of
//     8 heads per key/value head fills the tile; tcgen05's 128 rows would be
//     15/16 padding.
//   * a tile of 16 tokens is copied (cp.async) as it lies, whole lines, into
//     swizzled shared memory, and every lane reads its own fragments' bytes:
//     contiguous pieces of a row.  Which dim a fragment index stands for is
//     free (the contraction index of S, the row index of O^T), so a lane's
//     piece of a row becomes consecutive fragments.
//   * value fragments pair two tokens of one dim: bytes of two rows'
//     words, merged with byte permutations.
//   * P^T needs one 8x8 transpose per 8 tokens (movmatrix).
// A block of 4 warps takes an item's 16-token tiles round robin, joins its warps'
// results in shared memory at the item's end, and prefetches across items; 16
// warps an SM (8 with tiles of 16 query rows) hide the chain of a tile.
//
// Measured (device time): 64 sequences to 16384 tokens, 64 / 8 heads x 128, E4M3:
// 178 us, 5.6 TB/s (0.86 of a copy's rate; the loads alone take 155 us); 32 sequences
// to 4096, 32 heads, INT4: 110 us, bound by about 400 instructions per tile at half the
// bytes (two tiles at a time per warp took the same time); 5 proposals of 16 sequences
// to 8000, 8 heads per key/value head, INT8: 70 us.  1 sequence at 1000 tokens: 9.5 us,
// and 4 for the join.

#include <cuda_fp16.h>
#include <math.h>

#include "w4kv_attn.cuh"

namespace w4 {
namespace kv {
namespace {

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kTile = 16;  // tokens per MMA tile

template <int FMT, int D, int NT>
struct Shape {
    static constexpr int kRow = FMT == W4KV_INT4 ? D / 2 : D;  // code bytes of a row
    static constexpr int kKB = kRow / 4, kVB = kRow / 8;       // a lane's bytes of a key / value row
    static constexpr int kStage = 2 * kTile * kRow + 128;      // codes, then 32 scale words
    static constexpr int kBlocks = rows_blocks_per_sm(8 * NT);
    static constexpr int kStages = kRow == 128 ? (NT == 1 ? 3 : 5) : (NT == 1 ? 5 : 8);
    static constexpr int kSteps = D / 16;  // k steps of S, row tiles of O^T
    static constexpr int kTileRows = 8 * NT;
    static constexpr int kPhase = 32;  // dims joined at a time
    static constexpr int kPad = kPhase + 8;
    static constexpr int kRing = kWarps * kStages * kStage;
    static constexpr int kJoin = kWarps * kTileRows * kPad * 4;
    static constexpr int kStats = kWarps * kTileRows * 2 * 4;
    static constexpr int kSmem = kRing + kJoin + kStats + static_cast<int>(sizeof(RangeSmem)) + 32;
    // the grid is one wave: kBlocks of them (and 1 KB each) fit an SM's 228 KB
    static_assert(kBlocks * (kSmem + 1024) <= 228 * 1024, "shared memory");
};

__device__ __forceinline__ uint32_t smem_u32(const void *p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

// Copies 16 bytes; with kCut, or writes 16 zeros.
template <bool kCut>
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool live) {
    if (kCut)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
    else
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// Where the 16-byte piece p of row r of a tile lies in a stage: the pieces that
// the lanes of a fragment load read together fall into different banks.
template <int ROW>
__device__ __forceinline__ int piece_at(int r, int p) {
    if (ROW == 128) return r * 128 + ((p ^ (r & 7)) << 4);
    if (ROW == 64) return r * 64 + ((p ^ ((r >> 1) & 3)) << 4);
    return r * 32 + ((p ^ ((r >> 2) & 1)) << 4);
}

// A tile's codes (16 rows one after the other: whole lines per instruction)
// and scale words into a stage.  kp, vp, sp point to the lane's first piece.
// With kCut only rows [v0, v1) are read, the others are zeros.
template <class S, bool kCut>
__device__ __forceinline__ void copy_tile(uint32_t stage, const uint8_t *kp, const uint8_t *vp,
                                          const float *sp, int lane, int v0, int v1) {
    constexpr int kPieces = S::kRow / 16;
    const int r0 = lane / kPieces;
#pragma unroll
    for (int i = 0; i < S::kRow / 32; ++i) {  // 512 bytes each
        const int r = r0 + i * (32 / kPieces);
        const uint32_t at = piece_at<S::kRow>(r, lane % kPieces);
        const bool live = !kCut || (r >= v0 && r < v1);
        copy16<kCut>(stage + at, kp + i * 512, live);
        copy16<kCut>(stage + kTile * S::kRow + at, vp + i * 512, live);
    }
    const int r = lane & 15;
    const uint32_t at = stage + 2 * kTile * S::kRow + lane * 4;
    if (kCut)
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(at), "l"(sp), "r"(r >= v0 && r < v1 ? 4 : 0) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(at), "l"(sp) : "memory");
}

__device__ __forceinline__ void mma(float c[4], const uint32_t a[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
    return __byte_perm(a, b, sel);
}

// Four code bytes -> two fp16 pairs (bytes 0, 1 and 2, 3).
template <int FMT>
__device__ __forceinline__ void widen4(uint32_t w, uint32_t *lo, uint32_t *hi) {
    if (FMT == W4KV_INT8) {  // 1152 + q as fp16 bits 0x64(q ^ 0x80), then - 1152
        const uint32_t x = w ^ 0x80808080u;
        const __half2 bias = __half2half2(__ushort_as_half(0x6480));
        const uint32_t l = prmt(x, 0x64646464u, 0x4140), h = prmt(x, 0x64646464u, 0x4342);
        const __half2 a = __hsub2(*reinterpret_cast<const __half2 *>(&l), bias);
        const __half2 b = __hsub2(*reinterpret_cast<const __half2 *>(&h), bias);
        *lo = *reinterpret_cast<const uint32_t *>(&a);
        *hi = *reinterpret_cast<const uint32_t *>(&b);
    } else {
        asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
            "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
            : "=r"(*lo), "=r"(*hi)
            : "r"(w));
    }
}

// The dims of k step s of lane c: fragment k 2c, 2c + 1 are d, d + 1 and
// k 2c + 8, 2c + 9 are d + 2, d + 3.
template <int FMT, int D>
__device__ __forceinline__ int key_dim(int c, int s) {
    constexpr int kKB = (FMT == W4KV_INT4 ? D / 2 : D) / 4;
    if (FMT == W4KV_INT4) return 2 * (c * kKB + 4 * (s >> 1)) + 4 * (s & 1);
    return c * kKB + 4 * s;
}

// Where a walk over the block's units stands: an item and its tiles.
struct Walk {
    Seq s;
    int b, h, tile;   // sequence, key/value head, tile of its (row, head) pairs
    int lo, hi;       // cached positions that the tile's rows see
    int x, nu;        // walked of the item, in cost; its units
    int64_t rem;      // cost of the block's range not yet walked
    int u0, u1;       // units of the current segment (the item's part in the block's range)
    int next, end;    // its 16-token tiles: this warp's next one, the first behind it
};

template <int FMT, int D, int XT, int NT>
__global__ void __launch_bounds__(kThreads, Shape<FMT, D, NT>::kBlocks) rows_kernel(const Attn a) {
    using S = Shape<FMT, D, NT>;
    extern __shared__ __align__(128) uint8_t smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, c = lane & 3;
    uint8_t *ring = smem + warp * S::kStages * S::kStage;
    const uint32_t ring_u = smem_u32(ring);
    float *join = reinterpret_cast<float *>(smem + S::kRing);
    float *stat_m = reinterpret_cast<float *>(smem + S::kRing + S::kJoin);  // [warps][rows]
    float *stat_l = stat_m + kWarps * S::kTileRows;
    RangeSmem *rsm = reinterpret_cast<RangeSmem *>(
        smem + ((S::kRing + S::kJoin + S::kStats + 15) & ~15));
    int *nans = reinterpret_cast<int *>(rsm + 1);  // a value's NaN code has been taken out: see zero_nans
    if (FMT == W4KV_E4M3 && threadIdx.x == 0) *nans = 0;  // (barriers follow)

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    auto tiles_of = [&](const Seq &s) { return (s.n * a.group - 1) / S::kTileRows + 1; };
    auto tile_range = [&](const Seq &s, int tile, int *lo, int *hi) {
        const int r0 = tile * S::kTileRows, r1 = min(s.n * a.group, r0 + S::kTileRows) - 1;
        *hi = a.causal ? min(s.hi, max(0, s.first + r1 / a.group + 1)) : s.hi;
        *lo = a.window > 0 ? min(*hi, window_from(s.first + r0 / a.group, a.window)) : 0;
        return max(1, ((*hi + 15) / 16 - *lo / 16 + kUnit / 16 - 1) / (kUnit / 16));  // units
    };
    const Range range = block_range<kThreads>(a.b.n, rsm, [&](int b) -> int64_t {
        const Seq s = load_seq(a, b);
        if (s.n == 0) return 0;
        const int tiles = tiles_of(s);
        int cost = 0, lo, hi;
        for (int t = 0; t < tiles; ++t) cost += kItemCost + tile_range(s, t, &lo, &hi);
        return int64_t(cost) * a.c.heads;
    });
    if (threadIdx.x == 0) a.desc[blockIdx.x] = make_int4(0, 0, 0, 0);
    if (range.start == range.end) return;

    // Opens the segment (the part of one item in this block's range) at w.b, w.h, w.x.
    auto open = [&](Walk &w) {
        const int x1 = static_cast<int>(min(static_cast<int64_t>(w.nu + kItemCost), w.x + w.rem));
        w.u0 = max(0, w.x - kItemCost);
        w.u1 = max(0, x1 - kItemCost);
        w.rem -= x1 - w.x;
        w.x = x1;
        const int t0 = w.lo / 16;
        w.next = t0 + w.u0 * (kUnit / 16) + warp;
        w.end = min((w.hi + 15) / 16, t0 + w.u1 * (kUnit / 16));
    };
    auto next_item = [&](Walk &w) {  // only while w.rem > 0: a later item exists
        w.x = 0;
        if (++w.tile == tiles_of(w.s)) {
            w.tile = 0;
            ++w.h;
        }
        if (w.h == a.c.heads) {
            w.h = 0;
            do {
                if (w.b + 1 < a.b.n) ++w.b;
                w.s = load_seq(a, w.b);
            } while (w.s.n == 0 && w.b + 1 < a.b.n);
        }
        w.nu = tile_range(w.s, w.tile, &w.lo, &w.hi);
    };
    Walk w;
    w.b = range.b;
    w.s = load_seq(a, w.b);
    {
        const int tiles = tiles_of(w.s);
        int per_head = 0;
        for (int t = 0; t < tiles; ++t) per_head += kItemCost + tile_range(w.s, t, &w.lo, &w.hi);
        w.h = static_cast<int>(div_small(range.off, per_head));
        w.x = static_cast<int>(range.off - int64_t(w.h) * per_head);
        for (w.tile = 0;; ++w.tile) {
            w.nu = tile_range(w.s, w.tile, &w.lo, &w.hi);
            if (w.x < w.nu + kItemCost || w.tile + 1 >= tiles) break;
            w.x -= w.nu + kItemCost;
        }
    }
    w.rem = range.end - range.start;
    open(w);
    Walk p = w;  // the producer's walk, ahead of the consumer's

    // ---- producer: fragment bytes of one tile per stage ----
    int p_id = 0, p_rest = 0;
    bool p_live = true;  // a tile is left to issue
    auto fetch_page = [&]() {
        while (p.next >= p.end) {  // to the next segment that has a tile for this warp
            if (p.rem == 0) {
                p_live = false;
                return;
            }
            next_item(p);
            open(p);
        }
        const int pg = page_of_tile(a, p.next, &p_rest);
        p_id = pg < a.b.width ? __ldg(a.b.table + p.b * a.b.stride + pg) : -1;
    };
    fetch_page();
    uint32_t bad_mask = 0;  // per stage: the tile's page number was out of range
    const uint8_t *k_lane = a.c.k + lane * 16, *v_lane = a.c.v + lane * 16;
    const float *s_lane = (lane < 16 ? a.c.ks : a.c.vs) + (lane & 15);
    const int page_rows = a.c.heads * a.c.page;
    int put = 0;  // stage that is filled next
    auto issue = [&]() {
        if (p_live) {
            const uint32_t dst = ring_u + put * S::kStage;
            const bool ok = static_cast<uint32_t>(p_id) < static_cast<uint32_t>(a.c.pages);
            const int64_t r0 = int64_t(ok ? p_id : 0) * page_rows + (p.h * a.c.page + p_rest * kTile);
            const int v0 = p.lo - p.next * kTile, v1 = p.hi - p.next * kTile;  // rows in use
            if (ok && v0 <= 0 && v1 >= kTile) {
                bad_mask &= ~(1u << put);
                copy_tile<S, false>(dst, k_lane + r0 * S::kRow, v_lane + r0 * S::kRow, s_lane + r0, lane, 0, 0);
            } else {
                bad_mask = ok ? bad_mask & ~(1u << put) : bad_mask | (1u << put);
                if (!ok && lane == 0) atomicOr(a.status, kStatusBounds);
                copy_tile<S, true>(dst, k_lane + r0 * S::kRow, v_lane + r0 * S::kRow, s_lane + r0, lane,
                                   ok ? v0 : kTile, v1);
            }
            p.next += kWarps;
            fetch_page();
        }
        put = put + 1 == S::kStages ? 0 : put + 1;
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll 1
    for (int i = 0; i < S::kStages; ++i) issue();
    int get = 0;  // stage that is read next

    while (true) {  // segments
        if (w.u0 == w.u1) {  // none of the item's units
            if (w.rem == 0) break;
            next_item(w);
            open(w);
            continue;
        }
        // ---- the item's query rows as B fragments, and what each column sees ----
        uint32_t bq[NT][S::kSteps][2];
        float f[NT][2];  // scale * log2(e) without the row's power of two
        int qpos[NT][2];  // position of the column's row
        const int r0 = w.tile * S::kTileRows, R = min(S::kTileRows, w.s.n * a.group - r0);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int r = nt * 8 + g;
            const bool live = r < R;
            const int i = (r0 + r) / a.group;
            const uint16_t *qp = a.q + int64_t(w.s.row0 + i) * a.q_row +
                                 (w.h * a.group + r0 + r - i * a.group) * a.q_head;
            uint2 raw[S::kSteps];
            uint32_t top = 0;
#pragma unroll
            for (int s = 0; s < S::kSteps; ++s) {
                raw[s] = live ? __ldg(reinterpret_cast<const uint2 *>(qp + key_dim<FMT, D>(c, s)))
                              : make_uint2(0, 0);
                const uint32_t x = raw[s].x & 0x7FFF7FFFu, y = raw[s].y & 0x7FFF7FFFu;
                const uint32_t z = __vmaxu2(x, y);
                top = max(top, max(z & 0xFFFFu, z >> 16));
            }
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
            // the row times 2^sh has its largest element in [2^4, 2^5)
            int sh = 0;
            {
                const uint32_t t32 = __float_as_uint(widen1<XT>(static_cast<uint16_t>(top)));
                if (t32 != 0 && t32 < 0x7F800000u) sh = min(120, 131 - static_cast<int>(t32 >> 23));
            }
            const float up = pow2i(sh);
#pragma unroll
            for (int s = 0; s < S::kSteps; ++s) {
                const float e0 = widen1<XT>(raw[s].x & 0xFFFF) * up, e1 = widen1<XT>(raw[s].x >> 16) * up;
                float e2 = widen1<XT>(raw[s].y & 0xFFFF) * up, e3 = widen1<XT>(raw[s].y >> 16) * up;
                if (FMT == W4KV_INT4) {  // the second pair's codes come 16-fold
                    e2 *= 0.0625f;
                    e3 *= 0.0625f;
                }
                const __half2 h0 = __floats2half2_rn(e0, e1), h1 = __floats2half2_rn(e2, e3);
                bq[nt][s][0] = *reinterpret_cast<const uint32_t *>(&h0);
                bq[nt][s][1] = *reinterpret_cast<const uint32_t *>(&h1);
            }
            // this lane's score columns are 2c, 2c + 1: their rows' values live in lanes 8c, 8c + 4
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int s2 = __shfl_sync(0xffffffffu, sh, 8 * c + 4 * e);
                f[nt][e] = pow2i(-s2) * a.scale_log2;
                const int rr = nt * 8 + 2 * c + e;
                const int pos = w.s.first + (r0 + rr) / a.group;
                qpos[nt][e] = pos;
            }
        }
        // tiles inside [all_lo, all_hi) are seen whole by every row
        const int all_hi = a.causal ? min(w.hi, w.s.first + r0 / a.group + 1) : w.hi;
        const int all_lo = a.window > 0 ? max(w.lo, window_from(w.s.first + (r0 + R - 1) / a.group, a.window)) : w.lo;

        float m[NT][2], l[NT][2], o[NT][S::kSteps][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                m[nt][e] = kNone;
                l[nt][e] = 0.f;
            }
#pragma unroll
            for (int t = 0; t < S::kSteps; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[nt][t][i] = 0.f;
        }
        // A weight is fed as p * scale * vref, vref = 2^(133 - e) with e the exponent field of the
        // largest value scale that the column's row has seen (at least 7).  Each column has its
        // own: one for the tile would let tokens that a row does not see shift its weights out of
        // fp16's range.  For the same reason a column's maximum moves only by its own scores
        // where other columns' may be of tokens that it does not see.
        float vref[NT][2], vmax = pow2i(126);  // vmax: the lane's largest
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) vref[nt][0] = vref[nt][1] = vmax;

        auto consume = [&]() {
            asm volatile("cp.async.wait_group %0;" ::"n"(S::kStages - 1) : "memory");
            __syncwarp();
            uint32_t kw[2][S::kKB / 4], ksw[2], vsw[2];
            const uint8_t *st = ring + get * S::kStage;
            const uint32_t *sw = reinterpret_cast<const uint32_t *>(st + 2 * kTile * S::kRow);
            const bool bad = (bad_mask >> get) & 1;
#pragma unroll
            for (int i = 0; i < 2; ++i) {  // rows g, g + 8: the same piece offsets, 8 rows on
                if (S::kKB >= 16) {
#pragma unroll
                    for (int j = 0; j < S::kKB / 16; ++j) {
                        const uint4 v = *reinterpret_cast<const uint4 *>(
                            st + piece_at<S::kRow>(g, c * (S::kKB / 16) + j) + i * 8 * S::kRow);
                        kw[i][4 * j] = v.x, kw[i][4 * j + 1] = v.y;
                        kw[i][4 * j + 2] = v.z, kw[i][4 * j + 3] = v.w;
                    }
                } else {
                    const uint2 v = *reinterpret_cast<const uint2 *>(
                        st + piece_at<S::kRow>(g, c >> 1) + (c & 1) * 8 + i * 8 * S::kRow);
                    kw[i][0] = v.x, kw[i][1] = v.y;
                }
            }
            ksw[0] = sw[g], ksw[1] = sw[g + 8];
            vsw[0] = sw[16 + g], vsw[1] = sw[24 + g];
            // ---- S^T = K Q^T ----
            float sc[NT][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i) sc[nt][i] = 0.f;
#pragma unroll
            for (int s = 0; s < S::kSteps; ++s) {
                uint32_t fa[4];
                if (FMT == W4KV_INT4) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) {  // u - z, then 16 (u - z), of rows g, g + 8
                        const uint32_t x = kw[q & 1][s >> 1] >> (8 * (s & 1));
                        const uint32_t u = (x & (q & 2 ? 0x00F000F0u : 0x000F000Fu)) | 0x64006400u;
                        const uint32_t z = (ksw[q & 1] & 15u) * (q & 2 ? 0x100010u : 0x10001u) | 0x64006400u;
                        const __half2 r = __hsub2(*reinterpret_cast<const __half2 *>(&u),
                                                  *reinterpret_cast<const __half2 *>(&z));
                        fa[q] = *reinterpret_cast<const uint32_t *>(&r);
                    }
                } else {
                    widen4<FMT>(kw[0][s], &fa[0], &fa[2]);
                    widen4<FMT>(kw[1][s], &fa[1], &fa[3]);
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) mma(sc[nt], fa, bq[nt][s][0], bq[nt][s][1]);
            }
            // ---- scores in base 2, masked ----
            bool grow = false;
            const int kv0 = w.next * kTile;
            const bool cut = bad || kv0 < all_lo || kv0 + kTile > all_hi;  // warp-uniform
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int e = i & 1;
                    const uint32_t kw_ = ksw[i >> 1];
                    float x = sc[nt][i];
                    x *= FMT == W4KV_INT4 ? int4_scale(kw_) : __uint_as_float(kw_);
                    sc[nt][i] = x * f[nt][e];
                }
            if (cut) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int j = kv0 + g + 8 * (i >> 1), pos = qpos[nt][i & 1];
                        if (bad || j < w.lo || j >= w.hi || (a.causal && j > pos) ||
                            (a.window > 0 && j < window_from(pos, a.window)))
                            sc[nt][i] = -INFINITY;
                    }
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i) grow = grow || sc[nt][i] > m[nt][i & 1] + 8.f;
            // ---- new reference maxima and value exponent, if they moved ----
            if (cut) {  // scales of rows out of use may be anything
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int j = kv0 + g + 8 * i;
                    if (bad || j < w.lo || j >= w.hi) vsw[i] = 0;
                }
            }
            auto exponent = [](uint32_t scale) {  // its field; none for infinities and NaN
                const uint32_t e = (scale >> 23) & 255u;
                return e == 255u ? 0u : e;
            };
            const uint32_t ve = __reduce_max_sync(0xffffffffu, max(max(exponent(vsw[0]), exponent(vsw[1])), 7u));
            const float vtile = pow2i(133 - static_cast<int>(ve));
            if (__any_sync(0xffffffffu, grow || vtile < vmax)) {
                // (without a window, cut tiles are an item's last)
                const bool own_moves = cut || a.window > 0;
                vmax = 0.f;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float fo[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float x = fmaxf(sc[nt][e], sc[nt][e + 2]), v = vtile;
#pragma unroll
                        for (int d = 4; d < 32; d <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
                        x = !own_moves || x > m[nt][e] + 8.f ? fmaxf(x, m[nt][e]) : m[nt][e];
                        if (cut) {  // of the tokens that the row sees
                            uint32_t t = 7;
#pragma unroll
                            for (int i = 0; i < 2; ++i)
                                if (sc[nt][2 * i + e] != -INFINITY) t = max(t, exponent(vsw[i]));
#pragma unroll
                            for (int d = 4; d < 32; d <<= 1) t = max(t, __shfl_xor_sync(0xffffffffu, t, d));
                            v = pow2i(133 - static_cast<int>(t));
                        }
                        v = fminf(v, vref[nt][e]);
                        fo[e] = ex2(m[nt][e] - x);
                        m[nt][e] = x;
                        l[nt][e] *= fo[e];
                        fo[e] *= pow2i(max(-126, static_cast<int>(__float_as_uint(v) - __float_as_uint(vref[nt][e])) >> 23));
                        vref[nt][e] = v;
                        vmax = fmaxf(vmax, v);
                    }
#pragma unroll
                    for (int t = 0; t < S::kSteps; ++t)
#pragma unroll
                        for (int i = 0; i < 4; ++i) o[nt][t][i] *= fo[i & 1];
                }
            }
            // ---- weights, transposed into B fragments ----
            // For fp16 outputs a weight is fed as the sum of two fp16 numbers: one alone would
            // err as much as the output's own rounding (0.0003 instead of 0.0002 in all).
            constexpr int kParts = XT == W4_F16 ? 2 : 1;
            uint32_t pb[kParts][NT][2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {  // tokens g, g + 8
                const float vs = FMT == W4KV_INT4 ? int4_scale(vsw[i]) : __uint_as_float(vsw[i]);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float pw[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float x = sc[nt][2 * i + e];
                        const float pe = ex2(x - m[nt][e]);
                        l[nt][e] += pe;
                        pw[e] = pe * (vs * vref[nt][e]);
                        // unseen: exactly zero, whatever the value row's scale is
                        if (cut && x == -INFINITY) pw[e] = 0.f;
                    }
                    __half2 h = __floats2half2_rn(pw[0], pw[1]);
                    pb[0][nt][i] = transpose8(*reinterpret_cast<const uint32_t *>(&h));
                    if (kParts == 2) {
                        const float2 r = __half22float2(h);
                        h = __floats2half2_rn(pw[0] - r.x, pw[1] - r.y);
                        pb[kParts - 1][nt][i] = transpose8(*reinterpret_cast<const uint32_t *>(&h));
                    }
                }
            }
            // ---- O^T += V^T P^T ----
            // A weight of zero times a NaN is a NaN: in cut tiles, whose tokens not all rows see, NaN
            // codes count as zeros, and at the item's end each row looks for those it sees.
            if (FMT == W4KV_E4M3 && cut)
                zero_nans(reinterpret_cast<uint32_t *>(ring + get * S::kStage + kTile * S::kRow) + lane,
                          kTile * S::kRow, nans);
            uint32_t vw[4][S::kVB / 4];
            uint32_t vz[2];  // zero points of the value rows 2c, 2c + 1 and 2c + 8, 2c + 9
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint8_t *vp = st + kTile * S::kRow + (i >> 1) * 8 * S::kRow +
                                    piece_at<S::kRow>(2 * c + (i & 1), g * S::kVB / 16) +
                                    (g * S::kVB) % 16;
                if (S::kVB == 16) {
                    const uint4 v = *reinterpret_cast<const uint4 *>(vp);
                    vw[i][0] = v.x, vw[i][1] = v.y, vw[i][2] = v.z, vw[i][3] = v.w;
                } else if (S::kVB == 8) {
                    const uint2 v = *reinterpret_cast<const uint2 *>(vp);
                    vw[i][0] = v.x, vw[i][1] = v.y;
                } else {
                    vw[i][0] = *reinterpret_cast<const uint32_t *>(vp);
                }
            }
            if (FMT == W4KV_INT4) {
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const uint2 z = *reinterpret_cast<const uint2 *>(sw + 16 + 2 * c + 8 * q);
                    vz[q] = (z.x & 15u) | (z.y & 15u) << 16;
                }
            }
            __syncwarp();
            issue();
            if (FMT == W4KV_INT4) {
#pragma unroll
                for (int j = 0; j < S::kVB / 4; ++j) {
                    uint32_t x[2][2];  // [low, high nibbles' halves][tokens 2c.., 2c + 8..]
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        x[0][q] = prmt(vw[2 * q][j], vw[2 * q + 1][j], 0x5410);
                        x[1][q] = prmt(vw[2 * q][j], vw[2 * q + 1][j], 0x7632);
                    }
#pragma unroll
                    for (int t = 0; t < 4; ++t) {  // dims 8j + 2t, 8j + 2t + 1; 16-fold for odd t
                        // 1024 + u as fp16 bits 0x6400 | u (or 16 u), then - (1024 + z)
                        const uint32_t mask = t & 1 ? 0x00F000F0u : 0x000F000Fu;
                        const int sh = t & 2 ? 8 : 0;
                        uint32_t fa[4];
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const uint32_t u = ((x[q & 1][q >> 1] >> sh) & mask) | 0x64006400u;
                            const uint32_t z = (vz[q >> 1] << (t & 1 ? 4 : 0)) | 0x64006400u;
                            const __half2 r = __hsub2(*reinterpret_cast<const __half2 *>(&u),
                                                      *reinterpret_cast<const __half2 *>(&z));
                            fa[q] = *reinterpret_cast<const uint32_t *>(&r);
                        }
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int q = 0; q < kParts; ++q)
                                mma(o[nt][4 * j + t], fa, pb[q][nt][0], pb[q][nt][1]);
                    }
                }
            } else {
#pragma unroll
                for (int j = 0; j < S::kVB / 4; ++j) {
                    uint32_t fa[2][4];  // dims 4j, 4j + 1 and 4j + 2, 4j + 3
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const uint32_t x = prmt(vw[2 * q][j], vw[2 * q + 1][j], 0x5140);
                        const uint32_t y = prmt(vw[2 * q][j], vw[2 * q + 1][j], 0x7362);
                        widen4<FMT>(x, &fa[0][2 * q], &fa[0][2 * q + 1]);
                        widen4<FMT>(y, &fa[1][2 * q], &fa[1][2 * q + 1]);
                    }
#pragma unroll
                    for (int t = 0; t < 2; ++t)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int q = 0; q < kParts; ++q)
                                mma(o[nt][2 * j + t], fa[t], pb[q][nt][0], pb[q][nt][1]);
                }
            }
            get = get + 1 == S::kStages ? 0 : get + 1;
            w.next += kWarps;
        };
        while (w.next < w.end) consume();

        // ---- the warps' results together ----
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) {
                    l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], d);
                }
                if (g == 0) {
                    const int r = warp * S::kTileRows + nt * 8 + 2 * c + e;
                    stat_m[r] = m[nt][e];
                    stat_l[r] = l[nt][e];
                }
            }
        __syncthreads();
        float wgt[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = nt * 8 + 2 * c + e;
                float M = kNone, L = 0.f;
#pragma unroll
                for (int q = 0; q < kWarps; ++q) M = fmaxf(M, stat_m[q * S::kTileRows + r]);
#pragma unroll
                for (int q = 0; q < kWarps; ++q)
                    L += stat_l[q * S::kTileRows + r] * ex2(stat_m[q * S::kTileRows + r] - M);
                wgt[nt][e] = L == 0.f ? 0.f : ex2(m[nt][e] - M) / L;
                vref[nt][e] = __uint_as_float((254u << 23) - __float_as_uint(vref[nt][e]));  // 1 / vref
            }
        // where the item's units lie among the blocks
        const bool from_start = w.u0 == 0;
        const bool to_end = w.u1 == w.nu;
        const bool whole = from_start && to_end;
        float *slot = a.slots + (2 * int64_t(blockIdx.x) + (from_start ? 1 : 0)) *
                                    slot_floats(S::kTileRows, D);
        if (!whole && from_start && threadIdx.x == 0) {
            const int64_t last = range.end - w.rem + (w.nu - w.u1) - 1;  // its last unit
            a.desc[blockIdx.x] =
                make_int4(w.b, w.h, block_of_unit(last, range) - static_cast<int>(blockIdx.x) + 1, w.tile);
        }
        if (threadIdx.x < S::kTileRows) {
            const int r = threadIdx.x;
            float M = kNone, L = 0.f;
            for (int q = 0; q < kWarps; ++q) M = fmaxf(M, stat_m[q * S::kTileRows + r]);
            for (int q = 0; q < kWarps; ++q)
                L += stat_l[q * S::kTileRows + r] * ex2(stat_m[q * S::kTileRows + r] - M);
            if (!whole) {
                slot[r] = M;
                slot[S::kTileRows + r] = L;
            } else if (a.lse && r < R) {
                const int i = (r0 + r) / a.group;
                a.lse[int64_t(w.s.row0 + i) * a.heads + w.h * a.group + r0 + r - i * a.group] =
                    L == 0.f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
            }
        }
#pragma unroll
        for (int ph = 0; ph < D / S::kPhase; ++ph) {
            constexpr int kT = S::kPhase / 16;  // row tiles of O^T per phase
            if (ph) __syncthreads();            // the previous phase has been read
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int t = 0; t < kT; ++t)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float x = o[nt][ph * kT + t][e], y = o[nt][ph * kT + t][e + 2];
                        if (FMT == W4KV_INT4 && ((ph * kT + t) & 1)) {  // 16-fold codes
                            x *= 0.0625f;
                            y *= 0.0625f;
                        }
                        *reinterpret_cast<float2 *>(
                            join + (warp * S::kTileRows + nt * 8 + 2 * c + e) * S::kPad + t * 16 + 2 * g) =
                            make_float2(x * wgt[nt][e] * vref[nt][e], y * wgt[nt][e] * vref[nt][e]);
                    }
            __syncthreads();
            for (int i = threadIdx.x; i < S::kTileRows * S::kPhase / 2; i += kThreads) {
                const int r = i / (S::kPhase / 2), j = i - r * (S::kPhase / 2);
                if (r >= R) break;
                float x = 0.f, y = 0.f;
#pragma unroll
                for (int q = 0; q < kWarps; ++q) {
                    const float2 v = *reinterpret_cast<const float2 *>(
                        join + (q * S::kTileRows + r) * S::kPad + 2 * j);
                    x += v.x;
                    y += v.y;
                }
                const int d = (D / 8) * (j & 7) + 2 * (ph * kT + (j >> 3));
                if (FMT == W4KV_E4M3 && *nans) {  // the row's NaN codes in cut tiles
                    const int pos = w.s.first + (r0 + r) / a.group;
                    const int from = max(a.window > 0 ? window_from(pos, a.window) : 0, (w.lo / 16 + w.u0 * (kUnit / 16)) * 16);
                    const int to = min(min(w.hi, a.causal ? pos + 1 : w.hi), (w.lo / 16 + w.u1 * (kUnit / 16)) * 16);
                    for (int at = max(from, w.lo); at < to; ++at) {
                        if (at >= ((all_lo + 15) & ~15) && at < (all_hi & ~15)) at = all_hi & ~15;
                        const int64_t row = at < to ? row_of(a.c, a.b, w.b, at) : -1;
                        if (row < 0) continue;
                        const uint32_t code = __ldg(reinterpret_cast<const uint16_t *>(
                            a.c.v + (row + int64_t(w.h) * a.c.page) * D + d));
                        if (e4m3_nans(code) & 0x80u) x = __uint_as_float(0x7FC00000u);
                        if (e4m3_nans(code) & 0x8000u) y = __uint_as_float(0x7FC00000u);
                    }
                }
                if (whole) {
                    const int t = (r0 + r) / a.group;
                    *reinterpret_cast<uint32_t *>(a.o + int64_t(w.s.row0 + t) * a.o_row +
                                                  (w.h * a.group + r0 + r - t * a.group) * a.o_head + d) =
                        narrow1<XT>(x) | static_cast<uint32_t>(narrow1<XT>(y)) << 16;
                } else {
                    *reinterpret_cast<float2 *>(slot + 2 * S::kTileRows + r * D + d) = make_float2(x, y);
                }
            }
        }
        if (w.rem == 0) break;
        next_item(w);
        open(w);
        __syncthreads();  // join and the statistics are read before they are written again
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
}

template <int FMT, int D, int XT, int NT>
int run(const Attn &a, int grid, cudaStream_t stream) {
    using S = Shape<FMT, D, NT>;
    auto kernel = rows_kernel<FMT, D, XT, NT>;
    static std::atomic<unsigned long long> ready{0};  // a bit per device
    const int st = allow_smem(reinterpret_cast<const void *>(kernel), S::kSmem, &ready);
    if (st != W4_OK) return st;
    kernel<<<grid, kThreads, S::kSmem, stream>>>(a);
    return cuda_status(cudaGetLastError());
}

template <int FMT, int D>
int run_x(const Attn &a, int xt, int tile, int grid, cudaStream_t s) {
    if (xt == W4_F16)
        return tile == 8 ? run<FMT, D, W4_F16, 1>(a, grid, s) : run<FMT, D, W4_F16, 2>(a, grid, s);
    return tile == 8 ? run<FMT, D, W4_BF16, 1>(a, grid, s) : run<FMT, D, W4_BF16, 2>(a, grid, s);
}

}  // namespace

int launch_rows_attention(const Attn &a, int fmt, int dim, int xt, int tile, int grid,
                          cudaStream_t stream) {
    if (dim == 64) {
        if (fmt == W4KV_INT8) return run_x<W4KV_INT8, 64>(a, xt, tile, grid, stream);
        if (fmt == W4KV_E4M3) return run_x<W4KV_E4M3, 64>(a, xt, tile, grid, stream);
        return run_x<W4KV_INT4, 64>(a, xt, tile, grid, stream);
    }
    if (fmt == W4KV_INT8) return run_x<W4KV_INT8, 128>(a, xt, tile, grid, stream);
    if (fmt == W4KV_E4M3) return run_x<W4KV_E4M3, 128>(a, xt, tile, grid, stream);
    return run_x<W4KV_INT4, 128>(a, xt, tile, grid, stream);
}

}  // namespace kv
}  // namespace w4
