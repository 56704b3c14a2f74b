/*
 * spec_cache.h — C ABI of the paged key/value cache of a verification round.
 *
 * Draft-then-verify decoding runs the target model once over each request's
 * last kept token and its drafts, verifies (spec_verify.h), and drops what was
 * rejected. Three calls keep the cache that this pass reads:
 *
 *   spec_cache_step    after a verification: drop the rejected tokens, return
 *                      their pages, take pages for the next tokens, and write
 *                      the block table, the positions and the cache slots;
 *   spec_cache_append  write the new tokens' keys and values to their slots;
 *   spec_cache_attend  attention of the new tokens over the pages.
 *
 * The cache is a pool of num_pages pages of page_size tokens each. Request r
 * holds the pages block_table[r][0 .. ceil(len_r / page_size)); its token at
 * position p lives in slot block_table[r][p / page_size] * page_size +
 * p % page_size. Pages that no request holds are the first free_count entries
 * of the stack free_pages.
 *
 * Conventions (as in spec_verify.h):
 *  - array arguments are DEVICE pointers; the caller owns them;
 *  - calls are asynchronous on the given stream, allocate nothing, and never
 *    synchronise the host, so they can be captured into a CUDA graph;
 *  - argument errors are found on the host before anything is enqueued;
 *    errors in device data (lengths, slots, page numbers) set bits of
 *    *device_status (OR-ed in: clear it first), or with NULL of a word that the
 *    library has on each device (spec_cache_status reads it), and lead to no
 *    access out of bounds;
 *  - returns SPEC_OK or a SPEC_ERR_* code of spec_verify.h:
 *    SPEC_ERR_INVALID_ARG (null pointer, size, alignment),
 *    SPEC_ERR_UNSUPPORTED (a form the call does not have, or a device that is
 *    not sm_103), SPEC_ERR_CAPACITY (workspace too small), SPEC_ERR_CUDA.
 */
#ifndef SPEC_CACHE_H
#define SPEC_CACHE_H

#include <stddef.h>
#include <stdint.h>

#include "spec_verify.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Device status bits; they do not overlap SPEC_STATUS_*, and a wait that gave
 * up sets SPEC_STATUS_TIMEOUT (the call's outputs are not meaningful then). */
#define SPEC_CACHE_NO_PAGES 0x100u    /* step: too few free pages; nothing was changed */
#define SPEC_CACHE_BAD_LENGTHS 0x200u /* step: lengths or counts that cannot be; nothing was
                                         changed. attend: a request whose offsets or length
                                         cannot be; its rows see nothing. Or a call of more than
                                         2^30 steps (128 keys against some rows) for each
                                         multiprocessor, about ten minutes of work: all its
                                         rows see nothing */
#define SPEC_CACHE_BAD_SLOT 0x400u    /* append: a slot past the pool; it was skipped */
#define SPEC_CACHE_BAD_PAGE 0x800u    /* attend: a page number outside the pool; the
                                         request's outputs are not meaningful */

typedef enum { SPEC_CACHE_BF16 = 1, SPEC_CACHE_F16 = 2 } spec_cache_dtype;

typedef struct {
  int B;                   /* requests, >= 0 */
  int width;               /* columns of block_table, >= 1 */
  long long table_stride;  /* entries between rows of block_table, >= width */
  int page_size;           /* tokens per page, >= 1 */
  int num_pages;           /* pages of the pool = entries of free_pages, >= 1 */
  int num_tokens;          /* entries of positions and slots: the most new tokens */
  const int* held_lens;    /* [B] tokens whose pages each request holds */
  const int* new_lens;     /* [B] tokens to make room for, >= 0 */
  const int* cu_num_draft; /* [B+1] offsets of the drafts just verified (as in
                              spec_verify_batch), or NULL: nothing is dropped */
  const int* num_accepted; /* [B] accepted drafts (spec_verify_batch), or NULL */
  int* block_table;        /* [B x width] in/out */
  int* free_pages;         /* [num_pages] in/out: a stack, top at free_count */
  const int* free_count;   /* [1] free pages before the call */
  int* lens;               /* [B] out: tokens after the call */
  int* cu_new;             /* [B+1] out: offsets of the new tokens */
  int* positions;          /* [num_tokens] out: position of each new token, or NULL */
  long long* slots;        /* [num_tokens] out: slot of each new token */
  int* free_count_out;     /* [1] out: free pages after the call */
} spec_cache_step_args;

/*
 * spec_cache_step — the cache's bookkeeping between two rounds, in one kernel.
 * With kept_r = held_r - (gamma_r - accepted_r) and lens_r = kept_r + new_r
 * (held includes the drafts just verified), request r goes from
 * ceil(held_r / page_size) to ceil(lens_r / page_size) pages. Pages given up
 * are pushed on the stack in order of request and position, then the pages
 * taken are popped off its top in the same order, so the result does not
 * depend on scheduling. Table entries past a request's pages keep their old
 * values. New token t of request r (t = cu_new[r] .. cu_new[r+1] - 1) has
 * position kept_r + t - cu_new[r]; positions and slots past the last new
 * token are -1.
 * All or nothing: if pages run short, or a length is negative or past width
 * pages, or the new tokens exceed num_tokens, a status bit is set, tables and
 * stack stay as they are, lens = held_lens, cu_new = 0, positions = slots =
 * -1 and free_count_out = free_count.
 * What the call writes (the outputs, block_table, free_pages) overlaps no other
 * argument: SPEC_ERR_INVALID_ARG. It leaves its inputs but for the pages' owners
 * as they are, so it may be repeated with the same inputs and gives the same
 * result.
 */
int spec_cache_step(const spec_cache_step_args* a, void* stream, unsigned* device_status);

typedef struct {
  long long num_tokens;      /* T, >= 0 */
  int kv_heads, dim;         /* >= 1 */
  int page_size;             /* >= 1 */
  long long num_pages;       /* >= 1 */
  int dtype;                 /* SPEC_CACHE_BF16 or SPEC_CACHE_F16, of all four arrays */
  const void* k;             /* [T, kv_heads, dim]; strides in elements, dim's is 1 */
  long long k_token, k_head;
  const void* v;
  long long v_token, v_head;
  const long long* slots;    /* [T]; negative: the token is skipped */
  void* k_pages;             /* [num_pages, page_size, kv_heads, dim] by strides in */
  long long kp_page, kp_token, kp_head; /* elements, dim's is 1: tokens or heads outside */
  void* v_pages;
  long long vp_page, vp_token, vp_head;
} spec_cache_append_args;

/* spec_cache_append — copy each token's keys and values to its slot. Two
 * tokens with one slot leave either's values. Any alignment; 16-byte aligned
 * addresses and strides take 16-byte accesses. */
int spec_cache_append(const spec_cache_append_args* a, void* stream, unsigned* device_status);

typedef struct {
  int B;                     /* requests, >= 0 */
  int num_tokens;            /* T: rows of q, out and lse */
  int max_q;                 /* most new tokens of one request that the caller expects,
                                >= 1: speed only, larger requests are computed too */
  int heads, kv_heads, dim;  /* heads = G * kv_heads, G <= 128; dim a multiple of 8, <= 128 */
  int page_size;             /* a power of two, >= 8 */
  int width;                 /* columns of block_table, >= 1 */
  long long num_pages;       /* >= 1 */
  int dtype;                 /* SPEC_CACHE_BF16 or SPEC_CACHE_F16: q, pages and out */
  const void* q;             /* [T, heads, dim]; strides in elements, dim's is 1 */
  long long q_token, q_head;
  const void* k_pages;       /* as in spec_cache_append_args */
  long long kp_page, kp_token, kp_head;
  const void* v_pages;
  long long vp_page, vp_token, vp_head;
  const int* block_table;    /* [B x width] */
  long long table_stride;
  const int* kv_lens;        /* [B] tokens of each request, the new ones among them; at most
                                width pages and 2^31 - 2^16 */
  const int* cu_q;           /* [B+1] offsets of the new tokens in q: 0 .. <= T */
  void* out;                 /* [T, heads, dim] out */
  long long out_token, out_head;
  float* lse;                /* [T, heads] out: ln of the sum of exp(score), or NULL */
  float scale;               /* of the scores; 1 / sqrt(dim) as a rule. scale / ln 2 is finite */
  int window;                /* tokens that a row sees, itself among them; 0: all */
  int sinks;                 /* first tokens that a window leaves visible, >= 0 */
  void* workspace;           /* spec_cache_attend_workspace bytes, 256-byte aligned; its
                                contents do not matter; one call at a time */
  size_t workspace_bytes;
} spec_cache_attend_args;

/* spec_cache_attend_workspace — bytes of workspace that the call wants, by
 * the sizes of *a (its pointers are not looked at), or a negative SPEC_ERR_*. */
long long spec_cache_attend_workspace(const spec_cache_attend_args* a);

/*
 * spec_cache_attend — attention of each request's new tokens over its pages.
 * New token i of request r with n_r new tokens stands at position
 * p = kv_lens[r] - n_r + i and sees the tokens j <= p of its request, with a
 * window only those with p - j < window or j < sinks; query head h reads the
 * keys and values of head h / G:
 *   out = sum_j softmax_j(scale q . k_j) v_j,   lse = ln sum_j e^(scale q . k_j).
 * A token that sees nothing (p < 0), and the rows that belong to no request (past
 * cu_q[B], before cu_q[0]), give out = 0 and lse = -inf. Scores, softmax
 * statistics and sums are fp32; the softmax weights are rounded to the cache's
 * type before they meet the values. out, lse and workspace overlap nothing else.
 * Whatever the memory of slots that no row of a request sees holds, NaN and
 * infinities too, does not reach the outputs (a value that some row sees and that
 * is not finite may make other rows of its request not finite). Pages that lie
 * wholly outside every row's window are not read and may have been given to others.
 * The result is the same to the bit in every call with the same arguments on the
 * same kind of GPU.
 * Addresses and strides (of more than one element) of q, pages and out:
 * multiples of 16 bytes (SPEC_ERR_INVALID_ARG).
 */
int spec_cache_attend(const spec_cache_attend_args* a, void* stream, unsigned* device_status);

/*
 * spec_cache_status — wait for the current device's work, read the status bits of
 * the calls that had device_status = NULL on it, and clear them. Returns SPEC_OK,
 * or SPEC_ERR_DEVICE_STATUS where a bit is set.
 */
int spec_cache_status(unsigned* bits);

#ifdef __cplusplus
}
#endif

#endif /* SPEC_CACHE_H */
