/*
 * loopq_kv.h -- paged key-value cache of a looped transformer and the
 * attention over it, the part of a block between its q|k|v linear and its
 * output linear (include/loopq.h), for AMD Instinct MI355X (gfx950).
 *
 * The pages give the shapes: each token passes through the same layers several
 * times ("LoopQ 4-bit quantization of Ouro-1.4B -- raw artifacts", 24 layers
 * four times), so every (layer, loop) has keys and values of its own for every
 * token.  One (layer, loop) is a "slab" here (slab = layer * T + t); the page
 * table is shared by all slabs, since they grow, fork and shrink together.
 *
 * The cache:
 *   pool   bf16 [num_pages][slabs][2][heads][page_size][head_dim], contiguous;
 *          index 0 of the third axis holds keys, 1 values.  A page is one
 *          contiguous run, so forking or moving it is one copy for all slabs.
 *   table  int32 [rows][max_pages]: entry k of row b is the page that holds the
 *          row's tokens k * page_size .. k * page_size + page_size - 1.  An entry
 *          outside [0, num_pages) (-1 by custom) is no page.
 *   lens   int32 [rows]: tokens of each row (0: an empty row).
 *   refs   int32 [num_pages]: holders of each page (table entries, and whatever
 *          the caller pins); 0 is a free page.
 * Lengths, tables and reference counts live on the device and are read there,
 * so a sequence of calls needs no host synchronization and can be captured
 * into a HIP graph.  Their values are never trusted with an address: an entry
 * outside the pool is no page, a length counts as between 0 and max_pages *
 * page_size.
 *
 * Limits (LOOPQ_ERR_UNSUPPORTED outside them): head_dim 64, 96 or 128;
 * page_size a power of two in 8 .. 256; a page below 2 GiB; num_pages <= 2^22;
 * rows <= 8192; max_pages <= 2^22 and rows * max_pages < 2^31; heads_q a
 * multiple of heads.
 *
 * The conventions of loopq.h hold: device pointers unless the name ends in
 * _host, work is enqueued on `stream` and the call returns, the caller owns
 * every buffer, arguments are checked on the host before any HIP call.  rows
 * or a query count of 0 is a no-op.  Buffers must not overlap unless a call
 * says so.
 */
#ifndef LOOPQ_KV_H
#define LOOPQ_KV_H

#include "loopq.h"

#ifdef __cplusplus
extern "C" {
#endif

/* The pool's shape and memory.  data is 16-byte aligned. */
typedef struct {
  void* data;
  int32_t num_pages, slabs, heads, page_size, head_dim;
} loopq_kv_pool;

/* Page table, lengths and reference counts (4-byte aligned device memory). */
typedef struct {
  int32_t* table; /* [rows][max_pages] */
  int32_t* lens;  /* [rows] */
  int32_t* refs;  /* [num_pages] */
  int32_t rows, max_pages, num_pages;
} loopq_kv_table;

/* Values of info[0] (int32, device) after reserve and fork. */
typedef enum {
  LOOPQ_KV_DONE = 0,
  LOOPQ_KV_NO_PAGES = 1, /* fewer free pages than needed: nothing was changed */
  LOOPQ_KV_ROW_FULL = 2  /* a row would need more than max_pages pages: nothing was changed */
} loopq_kv_info;

/* Bytes of a pool's data (host only). */
int32_t loopq_kv_pool_bytes(int32_t num_pages, int32_t slabs, int32_t heads, int32_t page_size,
                            int32_t head_dim, size_t* bytes_host);

/* Workspace of reserve, fork and compact for tables of up to `rows` rows (the
 * larger of in and out) over num_pages pages; a multiple of 256 (host only). */
int32_t loopq_kv_workspace_bytes(int32_t rows, int32_t num_pages, size_t* bytes_host);

/* Room for grow[b] (device int32 [rows], negative counts as 0) more tokens in
 * each row: lens grow by it and the pages the rows then lack are taken from the
 * free ones, lowest index first, in the order of rows and of positions, with
 * one reference each.  All or nothing: if the free pages do not suffice, or a
 * row would pass max_pages, out is a copy of in and info says so.  info[1] is
 * the number of pages taken, or needed.  A row's last partial page must not be
 * shared (loopq_kv_fork never leaves one shared).  out may be in itself (all
 * three buffers); the shapes of in and out are the same. */
int32_t loopq_kv_reserve(const loopq_kv_table* in_host, int32_t page_size, const int32_t* grow,
                         const loopq_kv_table* out_host, int32_t* info, void* workspace,
                         size_t workspace_bytes, void* stream);

/* Keys and values of new tokens into one slab.  cu (device int32 [rows + 1],
 * ascending from 0) gives row b the tokens cu[b] .. cu[b+1] - 1 of k and v; they
 * are the last tokens of the row (lens counts them already, see reserve).
 * k, v [tokens][heads][head_dim] in `dtype`, tokens ldk and ldv elements apart
 * (slices of a fused q|k|v row qualify), 16-byte aligned rows; fp32 is rounded
 * to bf16, to nearest, ties to even.  A token whose position has no page is
 * dropped; tokens past cu[rows] are not read.  tokens * heads * head_dim is at most
 * 2^35 - 2048 (LOOPQ_ERR_UNSUPPORTED). */
int32_t loopq_kv_write(const loopq_kv_pool* pool_host, int32_t slab, const loopq_kv_table* table_host,
                       const int32_t* cu, const void* k, int64_t ldk, const void* v, int64_t ldv,
                       int32_t dtype, int32_t tokens, void* stream);

/* Fork, reorder and free rows in one call: row i of out takes the tokens of row
 * parent[i] of in (device int32 [out rows]; a value outside [0, in rows) makes
 * an empty row).  Full pages are shared.  A partial last page is kept by the
 * first child, if in's row is its only holder; every other child gets a copy
 * of it in a free page, lowest index first, in the order of the rows.  Every
 * reference of in is given up and every one of out taken: refs of out = refs of
 * in - entries in in's table + entries in out's table.  Pages that this frees
 * are not used for the copies, and their contents stay.  If the free pages do
 * not suffice, out has empty rows and in's refs, nothing is copied and in goes
 * on being valid.  info[1] is the number of pages copied, or needed.  in and
 * out must not overlap; max_pages and num_pages are the same. */
int32_t loopq_kv_fork(const loopq_kv_pool* pool_host, const loopq_kv_table* in_host, const int32_t* parent,
                      const loopq_kv_table* out_host, int32_t* info, void* workspace,
                      size_t workspace_bytes, void* stream);

/* Free what a sliding window (window >= 1) leaves behind: the entries of pages
 * none of whose tokens a query at position lens[b] or later can see (all of them
 * before lens[b] - window + 1 and at or past sinks) become -1, and their pages
 * lose a reference.  out may be in itself. */
int32_t loopq_kv_trim(const loopq_kv_table* in_host, int32_t page_size, int32_t window, int32_t sinks,
                      const loopq_kv_table* out_host, void* stream);

/* Close the holes: with L pages in use (refs > 0), the k-th used page at index
 * L or above moves to the k-th free page below L, so that pages L and above
 * are free; table and refs follow (an entry whose page has no holder by refs
 * becomes -1).  page_map (int32 [num_pages]) receives each
 * used page's new index, -1 for a free one, for holders outside the table.
 * info = {L, pages moved}.  out may be in itself. */
int32_t loopq_kv_compact(const loopq_kv_pool* pool_host, const loopq_kv_table* in_host,
                         const loopq_kv_table* out_host, int32_t* page_map, int32_t* info,
                         void* workspace, size_t workspace_bytes, void* stream);

/* Page contents from one pool to another, or within one: dst page dst[i] = src
 * page src[i] for i < count (device int32 lists).  The pools differ at most in
 * num_pages.  A pair with an index outside its pool is skipped.  A page must not
 * be in both lists if the pools are the same, nor twice in dst. */
int32_t loopq_kv_copy_pages(const loopq_kv_pool* src_pool_host, const int32_t* src,
                            const loopq_kv_pool* dst_pool_host, const int32_t* dst, int32_t count,
                            void* stream);

/* Workspace of the attention calls (host only): queries is the number of query
 * tokens (rows for decode).  Enough for both calls; a multiple of 256. */
int32_t loopq_attn_workspace_bytes(int32_t queries, int32_t heads_q, int32_t rows,
                                   int32_t head_dim, size_t* bytes_host);

/* Attention of one new token per row over the row's cached tokens in one slab.
 * q, out [rows][heads_q][head_dim] in `dtype` (fp32 or bf16), rows ldq and ldo
 * elements apart, 16-byte aligned rows (with ldq = ldo also columns of the same
 * wider rows); query head h reads key head h / (heads_q / heads).  The query of
 * row b is its token lens[b] - 1 (already in the cache); key j is visible to a
 * query at position p if 0 <= j <= p, the table has a page for j, and window == 0
 * or p - j < window or j < sinks.
 * out = sum_j exp(s_j - m) v_j / sum_j exp(s_j - m) over the visible keys,
 * s_j = scale * (q . k_j), m their maximum; 0 where no key is visible.  Keys and
 * values at hidden positions are not used, whatever they hold.  scale is finite;
 * window, sinks >= 0.
 *
 * Precision: sums are held in fp32.  fp32 queries and the weights they give
 * enter the products with 24 bits, weights of bf16 queries with 16 (see prefill).
 * Range: the magnitudes of the values that a query sees add up to less than 2^119
 * in every column; past that, results may be infinite (weights are taken against
 * a reference that their maximum may exceed by 2^8).
 * Infinities and NaN: a value that is infinite or NaN makes its column infinite or
 * NaN (either of them) for every query that sees it, however small its weight,
 * and reaches no other query.  A score of -infinity is a weight of 0, and out is 0
 * if all are; a score of +infinity or NaN makes the whole head's result NaN. */
int32_t loopq_attn_decode(const loopq_kv_pool* pool_host, int32_t slab, const loopq_kv_table* table_host,
                          const void* q, int64_t ldq, int32_t dtype, int32_t heads_q, float scale,
                          int32_t window, int32_t sinks, void* out, int64_t ldo, void* workspace,
                          size_t workspace_bytes, void* stream);

/* The same for several new tokens a row: row b has the queries cu[b] ..
 * cu[b+1] - 1 of q (device int32 [rows + 1], ascending from 0), the last of the
 * row's lens[b] tokens, query i of n at position lens[b] - n + i (nothing is
 * visible at a negative position).  q, out [queries][heads_q][head_dim]; rows of
 * out past cu[rows] are not written.  Weights of bf16 queries are rounded to one
 * bf16 (8 bits) before they meet the values, and the sum is that of the rounded
 * weights; they keep 16 bits where window < 256 (and not 0) or the queries lie
 * among the first 255 tokens.  fp32 queries keep 24 bits throughout. */
int32_t loopq_attn_prefill(const loopq_kv_pool* pool_host, int32_t slab, const loopq_kv_table* table_host,
                           const int32_t* cu, const void* q, int64_t ldq, int32_t dtype, int32_t queries,
                           int32_t heads_q, float scale, int32_t window, int32_t sinks, void* out,
                           int64_t ldo, void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* LOOPQ_KV_H */
