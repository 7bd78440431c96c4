/*
 * w4kv.h -- C ABI of libw4a16.so, third workload: a paged key/value cache kept
 * in 8 or 4 bits, and the attention that reads it, on NVIDIA B200 (sm_100a).
 * Beside quantized weights (w4a16.h) and activations (w8a8.h) the cache is the
 * remaining large array that a decode step streams.
 *
 * Method source (cited by page title and section):
 *   [LQ]  "LLM quantization methods: principles and implementation"
 *         (zhiyuanblog.org/blog/llm-quantization): §2.2 symmetric and
 *         asymmetric quantization (scale, zero point, round, clamp),
 *         §4.6 FP8 E4M3 (scale = max|x| / 448, cast).
 *
 * Conventions are those of w4a16.h (device pointers owned by the caller,
 * 16-byte aligned; `stream` a cudaStream_t as void*; calls only enqueue;
 * arguments validated on the host before anything is enqueued; status codes
 * w4_status; w4_last_error() describes a failure).  The two structs are HOST
 * structs, read during the call only.
 *
 * The cache.  A row is one token of one key/value head: head_dim numbers x,
 * kept as codes and one 32-bit scale word.
 *   W4KV_INT8  s = fl32(amax / 127), q = clamp(rne(fl32(x / s)), -127, 127);
 *              the row stands for q * s.
 *   W4KV_E4M3  s = fl32(amax / 448), q = the nearest E4M3 value (ties to even,
 *              saturating) of fl32(x / s); the row stands for q * s.  (The NaN
 *              codes 0x7F and 0xFF, which w4kv_append does not write, stand for
 *              NaN in their element.)
 *   W4KV_INT4  lo = min(0, min x), hi = max(0, max x); s = fl32(fl32(hi - lo) / 15)
 *              with its bit pattern rounded to a multiple of 16 (ties up);
 *              z = rne(fl32(-lo / s)), u = clamp(rne(fl32(fl32(x / s) + z)), 0, 15).
 *              The scale word is the bit pattern of s with z (0 .. 15) in the
 *              four low bits that the rounding freed; the row stands for
 *              (u - z) * s.  The range contains 0, so z needs no clamp.
 *   s = 0 stores zero codes (and z = 0).  A row with a NaN or an infinity, or
 *   whose hi - lo overflows (W4KV_INT4), stores zero codes and a NaN scale: it
 *   reads back as NaN and turns the attention rows that see it into NaN, and
 *   no others.
 *   Codes: [num_pages][kv_heads][page_size][head_dim] bytes, head_dim / 2 for
 *   W4KV_INT4 in the nibble order of w4_quantize; scale words:
 *   [num_pages][kv_heads][page_size].  page_size is a multiple of 16; head_dim
 *   is 64 or 128.
 *
 * The batch.  Sequence b has kv_lens[b] tokens, position p of it in page
 * page_table[b * table_stride + p / page_size] at offset p % page_size.  The
 * rows cu_rows[b] .. cu_rows[b + 1] - 1 of a call belong to sequence b and are
 * its LAST tokens: row r has position kv_lens[b] - (cu_rows[b + 1] - r).  So
 * kv_lens already counts the rows that a call appends.  cu_rows starts at 0 and does not decrease;
 * a sequence may have no rows.  Rows from cu_rows[batch] on belong to no
 * sequence: nothing of them is read or written.  These arrays live on the
 * device and are read by the kernels, so that one captured graph serves
 * changing lengths.
 *   table_width * page_size is at most 2^31 - 256.
 *   A position below 0 or beyond table_width pages and a page number outside
 *   [0, num_pages) are never dereferenced: the row is not stored (append),
 *   reads as zeros (read) or counts as unseen (attention), and the device status word
 *   reports W4_ERR_BOUNDS (w4_device_status).  A negative position is an
 *   error for append and read; for attention that row sees nothing.
 */
#ifndef W4KV_H
#define W4KV_H

#include <stddef.h>
#include <stdint.h>

#include "w4a16.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { W4KV_INT8 = 0, W4KV_E4M3 = 1, W4KV_INT4 = 2 } w4kv_format;

typedef struct {
    void *k_codes;
    float *k_scales;
    void *v_codes;
    float *v_scales;
    int64_t num_pages;
    int page_size; /* tokens per page: a multiple of 16 */
    int kv_heads;
    int head_dim; /* 64 or 128 */
    int fmt;      /* w4kv_format */
} w4kv_cache;

typedef struct {
    const int32_t *page_table; /* [batch][table_width], rows table_stride apart */
    int64_t table_stride;
    int64_t table_width;
    const int32_t *kv_lens; /* [batch] */
    const int32_t *cu_rows; /* [batch + 1] */
    int64_t batch;
} w4kv_batch;

/*
 * w4kv_append -- quantizes the keys and values of new tokens into the cache.
 *   K, V  [rows][kv_heads][head_dim] fp16 or bf16 (xt); the strides count
 *         elements, are multiples of 8 and need not be those of a dense array
 *         (slices of a fused projection's output work as they are).  The
 *         stride of a single row or head is not looked at.
 *   Positions that two rows of one call name (pages shared between sequences)
 *   hold one or the other row, or a mixture: pages that are written belong to
 *   one sequence.
 *   One kernel; each row is read once and its codes written once.
 */
int w4kv_append(const w4kv_cache *cache, const w4kv_batch *batch, const void *K, const void *V,
                int xt, int64_t rows, int64_t k_row_stride, int64_t k_head_stride,
                int64_t v_row_stride, int64_t v_head_stride, void *stream);

/*
 * w4kv_read -- the values of cached rows: fl16(fl32(q * s)) into K, V
 * [rows][kv_heads][head_dim] fp16 or bf16 (yt), each row of the batch the
 * cached token of its position (with cu_rows counting whole sequences: all of
 * them).  Strides as for w4kv_append; the rows of an output must not overlap.
 */
int w4kv_read(const w4kv_cache *cache, const w4kv_batch *batch, void *K, void *V, int yt,
              int64_t rows, int64_t k_row_stride, int64_t k_head_stride, int64_t v_row_stride,
              int64_t v_head_stride, void *stream);

/*
 * w4kv_attention_workspace_bytes -- device scratch bytes w4kv_attention needs
 * for these sizes on the current device (0 for sizes it rejects): partial
 * results of rows whose cached tokens are split between thread blocks, up to
 * 5 MB for decode steps and 44 MB where chunks are served.
 */
size_t w4kv_attention_workspace_bytes(const w4kv_cache *cache, int64_t batch, int64_t rows,
                                      int64_t max_rows, int heads);

/*
 * w4kv_attention -- O = softmax(scale * Q K^T) V over the cached rows.
 *   Q, O   [rows][heads][head_dim] fp16 or bf16 (xt), strides as above;
 *          heads is a multiple of kv_heads, query head h reads key/value head
 *          h / (heads / kv_heads).
 *   causal != 0: the row of position p sees the positions 0 .. p, or with
 *          window > 0 the last `window` of them (p - window + 1 .. p).
 *   causal == 0: every row sees all kv_lens[b] positions (window must be 0).
 *   A row that sees nothing gets zeros (and lse = -infinity).  What a row does
 *   not see has no influence on it, whatever it holds.
 *   lse    nullable [rows][heads] fp32 (dense): log of the sum of
 *          exp(scale * q k) over what the row sees, for joining with the
 *          attention over other keys.
 *   max_rows  at least the largest cu_rows[b + 1] - cu_rows[b] (1 for a plain
 *          decode step); it selects the kernels.  Of a longer sequence the
 *          rows beyond the first max_rows are left as they were and the device
 *          status word reports W4_ERR_BOUNDS.
 *   Numerics: codes enter the tensor cores unrounded (they are exact in fp16);
 *   scores, maxima, sums and outputs are fp32; the probabilities times the
 *   value scales are rounded to fp16 (relative to a running power of two of
 *   each row, so that no scale leaves the range: a token loses at most 2^-31,
 *   W4KV_INT4 2^-30, of the largest value that the row sees); the output is
 *   rounded once.  Queries enter as fp16, each row scaled by a power of two:
 *   exact for elements down to 2^-14 of the row's largest, smaller ones carry
 *   an error of at most 2^-25 of it.
 *   Q and what the cache's visible rows stand for must be finite for a finite
 *   result, and keys below 1e34.  Deterministic: repeated calls give the same bits.
 *   Sequences with at most 64 (row, query head) pairs per key/value head run on
 *   warp-level MMAs, bound by reading the cache; longer chunks on tcgen05.  Two
 *   kernels, or four where max_rows allows both kinds; no host synchronization;
 *   a captured call follows changed lengths, pages and row counts (up to
 *   max_rows).
 *   workspace: at least w4kv_attention_workspace_bytes(...) bytes, 256-byte
 *   aligned, contents irrelevant (clobbered); one per call in flight.
 */
int w4kv_attention(const w4kv_cache *cache, const w4kv_batch *batch, const void *Q, int xt,
                   int64_t rows, int heads, int64_t q_row_stride, int64_t q_head_stride, void *O,
                   int64_t o_row_stride, int64_t o_head_stride, float *lse, int64_t max_rows,
                   float scale, int causal, int64_t window, void *workspace,
                   size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* W4KV_H */
