/*
 * entmaxkv_pages.h -- C ABI of libentmaxkv.so: copying, forking, growing,
 * compacting and freeing the pages of a paged cache (bf16 or 4-bit, any
 * number of layers that share one page table).  Conventions of entmaxkv.h.
 *
 * There is no allocator state.  A block is in use when a row of the page
 * table reaches it (its first ceil(seq_lens[b] / P) entries), or when
 * hold[block] > 0 (int32 [num_blocks], nullable: blocks that the caller keeps
 * for itself, a cached prefix for instance).  Every other block is free, so a
 * sequence is freed by setting its length to 0 (or by forking its row away),
 * and nothing can leak.  Rows may share full pages.  A partial last page
 * belongs to one row: new tokens are written into it.  New blocks are always
 * the free ones with the lowest numbers, so every result is a function of
 * its inputs.
 *
 * kv_begin and kv_count of the shape must be 0 (a page holds every head).
 * page_table entries outside [0, num_blocks) inside a row set
 * ENTMAXKV_STATUS_BAD_PAGE and are treated as holding no block; over-long
 * sequences set ENTMAXKV_STATUS_BAD_LENGTH and count as max_pages * P tokens.
 */
#ifndef ENTMAXKV_PAGES_H
#define ENTMAXKV_PAGES_H

#include "entmaxkv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* bits of the device status word, beside those of entmaxkv.h */
enum {
    ENTMAXKV_STATUS_NO_BLOCK = 64, /* fewer free blocks than a call needed */
    ENTMAXKV_STATUS_BAD_ROW = 128  /* a parent outside [-1, B), or one that an in-place fork overwrites */
};

/* Buffers that share one page table: base[i], i < count (a host array of
 * device pointers, 16-byte aligned; entmaxkv_pages_copy also takes pinned
 * host memory), each block_bytes (a multiple of 16) for every block.
 * count <= ENTMAXKV_MAX_BUFFERS; the struct is read during the call only. */
#define ENTMAXKV_MAX_BUFFERS 256
typedef struct entmaxkv_buffers {
    int32_t count;
    int64_t block_bytes;
    void *const *base;
} entmaxkv_buffers;

/* Workspace bytes of the calls below; (size_t)-1 for an invalid shape.
 * Conventions of entmaxkv_workspace_size. */
ENTMAXKV_API size_t entmaxkv_pages_workspace_size(const entmaxkv_shape *shape);

/* refs[block] (int32 [num_blocks], nullable) = rows that reach the block +
 * max(hold, 0); n_free (int32 [1], nullable) = blocks with refs 0.  Both NULL:
 * ENTMAXKV_ERR_NULL. */
ENTMAXKV_API int entmaxkv_pages_refs(const entmaxkv_shape *shape, const int32_t *page_table,
                        const int32_t *seq_lens, const int32_t *hold, int32_t *refs,
                        int32_t *n_free, void *workspace, size_t ws_bytes, void *stream);

/*
 * Row b of the new table continues row parent[b] of the old one (int32 [B];
 * -1: an empty row, its sequence is freed).  lens_out[b] =
 * lens_in[parent[b]]; full pages are shared.  Of the rows with the same
 * parent p, row p itself keeps a partial last page if it is among them
 * (parent[p] == p), else the first of them; each other one gets a copy
 * of it in a new block (the free blocks of the OLD table, in ascending order
 * of b), in every buffer of bufs.  Entries past a row's pages become -1.
 * When the free blocks run out, the rows left over lose their partial page
 * (lens_out rounded down to whole pages) and ENTMAXKV_STATUS_NO_BLOCK is set.
 * meta_in / meta_out (nullable, together): metadata buffers
 * (entmaxkv_meta_bytes each) whose records follow their rows.
 * In place (table_out == table_in, then also lens_out == lens_in and each
 * meta_out == meta_in, and only then): rows with parent[b] == b stay as they
 * are, and a row may be the parent of another only if it is its own
 * parent; a row that breaks this, and any row with a parent outside
 * [-1, B), sets ENTMAXKV_STATUS_BAD_ROW and is left as it is in place, or
 * becomes empty.
 */
ENTMAXKV_API int entmaxkv_pages_fork(const entmaxkv_shape *shape, const int32_t *parent,
                        const int32_t *table_in, const int32_t *lens_in, const int32_t *hold,
                        int32_t *table_out, int32_t *lens_out, const entmaxkv_buffers *bufs,
                        const entmaxkv_buffers *meta_in, const entmaxkv_buffers *meta_out,
                        void *workspace, size_t ws_bytes, void *stream);

/*
 * Sequence b grows by n_add[b] tokens (int32 [B]; <= 0: none), in place: its
 * new pages get free blocks in ascending order of (b, page).  A sequence that
 * would grow past max_pages * P (ENTMAXKV_STATUS_BAD_LENGTH), and every
 * sequence for which the free blocks do not suffice, counting all needs
 * before it (ENTMAXKV_STATUS_NO_BLOCK), keeps its length and row.
 */
ENTMAXKV_API int entmaxkv_pages_grow(const entmaxkv_shape *shape, const int32_t *n_add, const int32_t *hold,
                        int32_t *page_table, int32_t *seq_lens, void *workspace, size_t ws_bytes,
                        void *stream);

/*
 * Move the blocks in use to the numbers below n_live, their count: the i-th
 * used block with a number >= n_live goes to the i-th free number below it,
 * in every buffer; the others stay.  table_out (may be table_in) gets the
 * rows with the new numbers and -1 past their pages; remap int32 [num_blocks]
 * the new number of every used block, -1 for free ones (holders follow it);
 * n_live int32 [1].
 */
ENTMAXKV_API int entmaxkv_pages_compact(const entmaxkv_shape *shape, const int32_t *table_in,
                           const int32_t *seq_lens, const int32_t *hold, int32_t *table_out,
                           const entmaxkv_buffers *bufs, int32_t *remap, int32_t *n_live,
                           void *workspace, size_t ws_bytes, void *stream);

/*
 * Block dst_ids[i] of every `dst` buffer := block src_ids[i] of the `src`
 * buffer of the same number, i < n (device int32; same count and block_bytes).
 * src_blocks / dst_blocks: blocks each side holds; pairs with a number
 * outside set ENTMAXKV_STATUS_BAD_PAGE and are skipped.  The dst blocks must
 * be distinct, and none may be a src block of the same buffer.  No workspace.
 */
ENTMAXKV_API int entmaxkv_pages_copy(const entmaxkv_buffers *src, int32_t src_blocks,
                        const entmaxkv_buffers *dst, int32_t dst_blocks, const int32_t *src_ids,
                        const int32_t *dst_ids, int32_t n, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* ENTMAXKV_PAGES_H */
