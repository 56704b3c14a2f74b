/*
 * spec_sparse.h — C ABI of what keeps a long paged cache (spec_cache.h) affordable:
 * reading few of its pages, and holding few of its tokens.
 *
 * Sparse attention over the pages that a cheap score selects for each new token:
 *
 *   spec_cache_bounds          the least and the largest key of every channel, for each
 *                              page and kv head, after the keys were written;
 *   spec_cache_score           for each new token, kv head and page an upper bound of the
 *                              page's scores, from the bounds alone;
 *   spec_cache_select          the pages of the highest scores, beside the first and the
 *                              last ones;
 *   spec_cache_attend_selected attention of the new tokens over those pages.
 *
 * Eviction by accumulated attention weight:
 *
 *   spec_cache_weigh           add to every cached token the softmax weights that the new
 *                              tokens gave it;
 *   spec_cache_evict           keep the tokens of the highest weights of each request and
 *                              kv head, beside the first and the last ones, close the gaps
 *                              and give pages back.
 *
 * Conventions, layouts of pages and tables, status words and return codes are those of
 * spec_cache.h. A page column c of a request is entry c of its row of block_table; it holds
 * the tokens c * page_size .. c * page_size + page_size - 1. New token i of request r with
 * n_r = cu_q[r + 1] - cu_q[r] new tokens stands at position kv_lens[r] - n_r + i, and a
 * column is visible to it if the column's first token is at that position or before.
 * Rows of the new tokens that belong to no request (before cu_q[0], past cu_q[B]) are given
 * -inf (scores), -1 (columns) or 0 (outputs). A request whose length cannot be sees nothing;
 * offsets that cannot be (negative, falling, past the last row) make the outputs of the call
 * meaningless. Both set SPEC_CACHE_BAD_LENGTHS.
 * Page sizes are powers of two from 8 to 2^20, dim is a multiple of 8 up to 128 and a kv head has
 * up to 128 query heads (SPEC_ERR_UNSUPPORTED). Addresses and strides (of more than one element)
 * of 16-bit arrays are multiples of 16 bytes. What a call writes overlaps none of its other
 * arguments. Results are the same to the bit in every call with the same arguments.
 * spec_cache_score writes, and spec_cache_select and spec_cache_evict choose their forms by, the
 * width that they are given (columns of scores or block_table), not the requests' lengths: pass the
 * columns that the longest request may have, as the first ones of a wider table (table_stride). 64
 * requests of 2-8 tokens over 1000-30000 in pages of 16, 1876 columns against 8192: score 36 and
 * 57 us, select 13 and 52. The other calls take the same time.
 */
#ifndef SPEC_SPARSE_H
#define SPEC_SPARSE_H

#include "spec_cache.h"

#ifdef __cplusplus
extern "C" {
#endif

#define SPEC_CACHE_BAD_SELECTION 0x1000u /* attend_selected: a column past the request's pages, or
                                            one that is not above the one before it; the row's
                                            outputs are not meaningful */

/* flags of spec_cache_weigh, test only: waits run out after some 0.1 ms, and one that the call needs
 * is never signalled, so that it ends with SPEC_STATUS_TIMEOUT */
#define SPEC_CACHE_TEST_WAIT_TIMEOUT 0x1u

typedef struct {
  int B;                     /* requests, >= 0 */
  int width;                 /* columns of block_table, >= 1 */
  long long table_stride;
  int max_q;                 /* most new tokens of one request that the caller expects, >= 1:
                                speed only */
  int kv_heads, dim, page_size;
  long long num_pages;
  int dtype;                 /* SPEC_CACHE_BF16 or SPEC_CACHE_F16: pages and bounds */
  const void* k_pages;       /* as in spec_cache_attend_args */
  long long kp_page, kp_token, kp_head;
  const int* block_table;    /* [B x width] */
  const int* kv_lens;        /* [B] */
  const int* cu_q;           /* [B+1], or NULL: all pages of every request */
  void* bounds;              /* [num_pages, kv_heads, 2, dim] in/out; strides in elements, dim's
                                is 1: the least (0) and the largest (1) of every channel */
  long long b_page, b_head, b_side;
} spec_cache_bounds_args;

/*
 * spec_cache_bounds — the channels' extremes over the held tokens (before kv_lens[r]) of every
 * page that holds one of a request's new tokens, or of all its pages. They are found from the
 * keys alone, whatever the bounds held before: tokens that a spec_cache_step dropped do not
 * count any more. Other pages keep their bounds. NaN goes into both. Pages of several requests
 * may be shared where they are held in full by each. A page number outside the pool sets
 * SPEC_CACHE_BAD_PAGE and is left out.
 */
int spec_cache_bounds(const spec_cache_bounds_args* a, void* stream, unsigned* device_status);

typedef struct {
  int B, width;
  long long table_stride;
  int num_tokens;            /* T: rows of q and scores */
  int max_q;                 /* as in spec_cache_bounds_args */
  int heads, kv_heads, dim, page_size;
  long long num_pages;
  int dtype;                 /* of q and bounds */
  const void* q;             /* [T, heads, dim]; strides in elements, dim's is 1 */
  long long q_token, q_head;
  const void* bounds;        /* [num_pages, kv_heads, 2, dim], finite */
  long long b_page, b_head, b_side;
  const int* block_table;
  const int* kv_lens;
  const int* cu_q;
  float* scores;             /* [T, kv_heads, width] out; columns adjacent */
  long long s_token, s_head;
} spec_cache_score_args;

/*
 * spec_cache_score — with lo and hi the bounds of column c, for each token and kv head
 *   scores[c] = sum over the G query heads of the kv head and the channels of
 *               max(q lo, q hi),
 * which no sum over the heads of q . k exceeds for a key k of the page; -inf for columns that
 * the token does not see. In fp32. Computed as P . hi + N . lo with P and N the sums over the
 * heads of q's positive and negative parts, so lo <= hi is taken for granted.
 */
int spec_cache_score(const spec_cache_score_args* a, void* stream, unsigned* device_status);

typedef struct {
  int B, num_tokens, kv_heads, page_size;
  int width;                 /* columns of scores */
  const float* scores;       /* [T, kv_heads, width]; columns adjacent */
  long long s_token, s_head;
  const int* kv_lens;
  const int* cu_q;
  int count;                 /* columns to select, >= 1 */
  int first, recent;         /* of them always: the first visible ones, and the last visible
                                ones up to the token's own; first + recent <= count */
  int* selected;             /* [T, kv_heads, count] out, contiguous: ascending columns, -1
                                past the last */
} spec_cache_select_args;

/*
 * spec_cache_select — for each token and kv head min(count, visible) columns: the first `first`
 * and the last `recent` visible ones, and of the others those of the highest scores (NaN counts
 * as +inf, -0 as 0; of equal ones the lowest columns). scores of columns that the token does not
 * see are not read.
 */
int spec_cache_select(const spec_cache_select_args* a, void* stream, unsigned* device_status);

typedef struct {
  int B, width;
  long long table_stride;
  int num_tokens;            /* T: rows of q, selected, out and lse */
  int heads, kv_heads, dim, page_size;
  long long num_pages;
  int dtype;
  const void* q;
  long long q_token, q_head;
  const void* k_pages;
  long long kp_page, kp_token, kp_head;
  const void* v_pages;
  long long vp_page, vp_token, vp_head;
  const int* block_table;
  const int* kv_lens;
  const int* cu_q;
  int count;                 /* columns of selected, >= 1 */
  const int* selected;       /* [T, kv_heads, count], contiguous: ascending columns, negative
                                past the last, as spec_cache_select leaves them */
  void* out;                 /* [T, heads, dim] out */
  long long out_token, out_head;
  float* lse;                /* [T, heads] out, or NULL */
  float scale;
} spec_cache_attend_selected_args;

/*
 * spec_cache_attend_selected — spec_cache_attend where token t and the query heads of kv head h
 * see the tokens up to t's own in the columns selected[t][h] alone. A row that sees nothing gives
 * out = 0 and lse = -inf. Scores, softmax statistics and sums are fp32; the softmax weights meet
 * the values with an error of 2^-15 (bf16) or 2^-21 (fp16) of themselves. Slots that no row sees do
 * not reach the outputs, whatever they hold; pages in no list are not read. A value that some row
 * sees and that is not finite may make other rows of its request and kv head NaN in its channel, also
 * rows whose lists do not have its page (they share a product, where its weight is 0). A key that is
 * not finite reaches only the rows that see it.
 */
int spec_cache_attend_selected(const spec_cache_attend_selected_args* a, void* stream,
                               unsigned* device_status);

typedef struct {
  int B, width;
  long long table_stride;
  int num_tokens;            /* T: rows of q and lse */
  int max_q;
  int heads, kv_heads, dim, page_size;
  long long num_pages;
  int dtype;
  const void* q;
  long long q_token, q_head;
  const void* k_pages;
  long long kp_page, kp_token, kp_head;
  const int* block_table;
  const int* kv_lens;
  const int* cu_q;
  const float* lse;          /* [T, heads], as spec_cache_attend gave it without a window */
  float* weights;            /* [num_pages, kv_heads, page_size] in/out, tokens adjacent */
  long long w_page, w_head;  /* elements */
  float scale, decay;        /* decay: finite */
  unsigned flags;            /* 0, or SPEC_CACHE_TEST_WAIT_TIMEOUT */
} spec_cache_weigh_args;

/*
 * spec_cache_weigh — for every held token j of each request with new tokens, and each kv head,
 *   w_j = (j is no new token ? decay * w_j : 0) + sum e^(scale q . k_j - lse)
 * over the new tokens at j or after and the head's query heads. New tokens' slots are written
 * whatever they held, and so are all with decay = 0. A row whose lse is -inf gives nothing (where
 * its scores are finite): what drafts gave stays in the sums when they are rejected, so a caller
 * who does not want that calls after the verification, with -inf in the rejected rows' lse.
 * Products and sums are fp32. Requests must not share pages (either's weights may be lost). A call
 * that sets SPEC_STATUS_TIMEOUT has updated some of the weights and others not.
 */
int spec_cache_weigh(const spec_cache_weigh_args* a, void* stream, unsigned* device_status);

typedef struct {
  int B, width;
  long long table_stride;
  int kv_heads, dim, page_size;
  int num_pages;             /* of the pool = entries of free_pages */
  int dtype;
  void* k_pages;             /* in/out; strides as in spec_cache_append_args */
  long long kp_page, kp_token, kp_head;
  void* v_pages;
  long long vp_page, vp_token, vp_head;
  float* weights;            /* in/out, as in spec_cache_weigh_args */
  long long w_page, w_head;
  const int* block_table;    /* [B x width]; stays as it is */
  const int* lens;           /* [B] tokens held */
  const int* budget;         /* [B] tokens to keep, >= 0 */
  int first, recent;         /* tokens that are always kept, >= 0 */
  int* free_pages;           /* [num_pages] in/out: a stack, top at free_count */
  const int* free_count;     /* [1] */
  int* lens_out;             /* [B] out */
  int* free_count_out;       /* [1] out */
  void* workspace;           /* spec_cache_evict_workspace bytes, 256-byte aligned; one call at
                                a time */
  size_t workspace_bytes;
} spec_cache_evict_args;

long long spec_cache_evict_workspace(const spec_cache_evict_args* a);

/*
 * spec_cache_evict — request r keeps lens_out = min(lens, max(budget, first + recent)) tokens.
 * Where that is fewer than it has, every kv head keeps the first `first` and the last `recent`
 * tokens, and of the others those of the highest weights (NaN counts as +inf, -0 as 0; of equal
 * ones the lowest positions), and the kept tokens' keys, values and weights move down to
 * positions 0 .. lens_out - 1 in their old order. Slots past those stay as they were. Pages past
 * ceil(lens_out / page_size) are pushed on the stack in order of requests and columns; table
 * entries stay. A kept token's position within its request changes, and differs from head to
 * head: the caller counts positions for rotary embeddings by itself, page bounds have to be found
 * anew, and no window fits any more.
 * A spec_cache_step that drops rejected drafts drops a request's last slots, whatever stands there,
 * and drafts, which few queries have looked at, are the first to go here. So where drafts await that
 * drop, `recent` has to be at least the most new tokens that a request has had in the round; or
 * the drop comes first, by a spec_cache_step with new_lens = 0. With less, older tokens are dropped
 * in the drafts' place and rejected drafts stay, and no status bit tells of it.
 * If a length or budget cannot be, or the stack would not hold the pages, SPEC_CACHE_BAD_LENGTHS
 * is set and nothing is changed (lens_out = lens, free_count_out = free_count). A page number
 * outside the pool sets SPEC_CACHE_BAD_PAGE; the request's tokens are not meaningful then. One that
 * would be given back stays off the stack and does not count in free_count_out (entries of
 * free_pages from there on are not meaningful then).
 * Requests must not share pages.
 */
int spec_cache_evict(const spec_cache_evict_args* a, void* stream, unsigned* device_status);

#ifdef __cplusplus
}
#endif

#endif /* SPEC_SPARSE_H */
