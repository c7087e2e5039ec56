/*
 * entmaxkv_kv4.h -- C ABI of libentmaxkv.so: a paged K/V cache held in 4 bits,
 * and the decode attention that reads it.  Same conventions as entmaxkv.h
 * (device pointers owned by the caller, work enqueued on `stream`, host-side
 * checks before anything is launched, device-side errors in the status word,
 * kv-head ranges), same page tables, lengths, page metadata and selections:
 * entmaxkv_score_pages and entmaxkv_select run on a 4-bit cache's metadata as
 * they are.
 *
 * The 4-bit cache
 * ---------------
 * One buffer for keys and one for values, each entmaxkv_kv4_bytes(shape)
 * long.  Every (token, kv head, 64 consecutive coordinates) is quantised by
 * itself, every fl() a rounding to fp32:
 *   lo   = min x                           (a bf16 value)
 *   s    = bf16(fl(fl(max x - lo) / 15)),  0 when below 2^-126
 *   code = clamp(rint(fl(fl(x - lo) * fl(1 / s))), 0, 15),  0 when s = 0
 * and stands for  value = fl(s * code + lo),  so |value - x| is at most half a
 * step s plus rounding.  A group that holds a NaN or an infinity, or whose
 * max - min overflows fp32, gets s = lo = NaN: every value of it reads as NaN.
 * 4.5 bits a value: codes, and 2 bf16 for 64 of them.
 *
 * Layout: cache[block][kv head][P / 16 tiles][9 d bytes].  A tile holds 16
 * consecutive tokens: 8 d bytes of codes, then for each token and each group
 * of 64 coordinates a 32-bit word, s in the low and lo in the high half.
 * Codes lie in 32-bit words:
 *   keys    token t, coordinate j = 64 g + 16 c + 8 i + n: word
 *           t d/8 + c d/32 + 2 g + i, bits 16 (n & 1) + 4 (n >> 1)
 *   values  token t, coordinate j = 64 g + 8 r + 4 i + n: word
 *           (t >> 1) d/4 + (r ^ x) d/32 + 2 g + i, bits 16 (t & 1) + 4 n,
 *           x = 2 ((t >> 1) & 3) for d = 128, 4 ((t >> 2) & 1) for d = 64
 *           (keeps the eight-token reads of the attention kernel on distinct
 *           shared-memory banks)
 */
#ifndef ENTMAXKV_KV4_H
#define ENTMAXKV_KV4_H

#include "entmaxkv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* element type of rows that entmaxkv_kv4_read writes */
enum { ENTMAXKV_ROWS_BF16 = 0, ENTMAXKV_ROWS_F32 = 1 };

/* Bytes of one 4-bit cache (keys or values): num_blocks * Hkv * P * 9 d / 16.
 * 0 for an invalid shape. */
ENTMAXKV_API size_t entmaxkv_kv4_bytes(const entmaxkv_shape *shape);

/*
 * Write new tokens.  Sequence b gains n_b tokens, at positions
 * seq_lens[b] - n_b .. seq_lens[b] - 1 (seq_lens already counts them).  Their
 * key and value rows are rows row_start[b] .. row_start[b+1] - 1 of k_new and
 * v_new (n_b = row_start[b+1] - row_start[b]; row_start int32 [B+1], device,
 * ascending: where it is not, ENTMAXKV_STATUS_BAD_LENGTH is set and rows of
 * other sequences may be left out too);
 * row_start NULL: one row a sequence, row b, n_rows = B.  Row i, kv head h
 * starts at element i * row_stride + h * d (bf16; row_stride >= Hkv d, a
 * multiple of 8, so rows may sit inside a fused projection's output).  With
 * meta (nullable) the metadata record of every page that got a row is rebuilt
 * from the values its codes stand for, in the layout of entmaxkv_meta_bytes:
 * kmin rounded down and kmax up to bf16, so that the page bound of
 * entmaxkv_score_pages bounds the scores of the 4-bit keys; mean and var as
 * in entmaxkv_build_meta (sums in fp64: partial sums of every 1024/d-th token,
 * added in order).
 * Sequences with n_b = 0 or a length <= 0 are skipped.  A sequence with
 * n_b < 0, n_b > seq_lens[b], rows outside [0, n_rows) or a length above
 * max_pages * P is skipped and sets ENTMAXKV_STATUS_BAD_LENGTH; a page with a
 * bad table entry is skipped and sets ENTMAXKV_STATUS_BAD_PAGE.  k_new and
 * v_new may be pinned host memory.  One launch; no workspace.
 */
ENTMAXKV_API int entmaxkv_kv4_write(const entmaxkv_shape *shape, const void *k_new, const void *v_new,
                       int64_t row_stride, const int32_t *row_start, int32_t n_rows,
                       const int32_t *page_table, const int32_t *seq_lens, void *k4, void *v4,
                       void *meta, void *stream);

/*
 * Read the last n_b tokens of every sequence back: the inverse of
 * entmaxkv_kv4_write, with the same rows (row_start, n_rows, row_stride) and
 * the same refusals.  k_out / v_out receive the values the codes stand for,
 * as fp32, or rounded once to bf16 (rows: ENTMAXKV_ROWS_*, else
 * ENTMAXKV_ERR_POLICY); row_stride counts their elements, a multiple of 8.
 */
ENTMAXKV_API int entmaxkv_kv4_read(const entmaxkv_shape *shape, const void *k4, const void *v4,
                      int64_t row_stride, const int32_t *row_start, int32_t n_rows,
                      const int32_t *page_table, const int32_t *seq_lens, int32_t rows,
                      void *k_out, void *v_out, void *stream);

/* Workspace bytes of entmaxkv_kv4_decode; (size_t)-1 for an invalid shape.
 * Conventions of entmaxkv_workspace_size. */
ENTMAXKV_API size_t entmaxkv_kv4_workspace_size(const entmaxkv_shape *shape);

/*
 * Decode attention over the 4-bit cache: for each (b, h), over the tokens T
 * of the pages sel[b][h][0..cnt[b][h]) (ascending, as entmaxkv_select writes
 * them; anything else sets ENTMAXKV_STATUS_BAD_SELECTION or counts once), or
 * over every token of the sequence when sel and cnt are both NULL,
 *   alpha > 1:  out = sum_T p_t v_t with the exact alpha-entmax weights of
 *               entmaxkv_decode_sparse; value rows without weight are not
 *               read; tau_out (nullable) gets tau
 *   alpha == 1: out = sum_T softmax(s)_t v_t; tau_out gets log sum_T exp(s_t)
 * with k_t, v_t the values the codes stand for.  out fp32 [B][Hq][d] (may be
 * pinned host memory), tau_out fp32 [B][Hq].  Scores are held in fp32 in the
 * units of a query whose largest coordinate is near 2^13, softmax weights in
 * units of the values' steps: beyond magnitudes of 2^100, keys may overflow
 * and values lose their smallest weights.  Near alpha = 1 entmax weights are
 * powers of 1/(alpha - 1) > 100, which the rounding of z - tau is multiplied
 * by: out is off by 5e-6 (relative) at alpha = 1.01, 5e-5 at 1.001 and 6e-4 at
 * 1.0001.  A head without tokens gets
 * out = 0, tau = NaN; a non-finite query row NaN, and
 * ENTMAXKV_STATUS_NONFINITE.  NaN values that carry weight, and NaN keys,
 * make out NaN.  Results do not depend on the order in which CTAs run.
 * max_pages <= 196608 with sel.
 */
ENTMAXKV_API int entmaxkv_kv4_decode(const entmaxkv_shape *shape, const void *q, const void *k4,
                        const void *v4, const int32_t *page_table, const int32_t *seq_lens,
                        const int32_t *sel, const int32_t *cnt, float alpha, float *out,
                        float *tau_out, void *workspace, size_t ws_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* ENTMAXKV_KV4_H */
