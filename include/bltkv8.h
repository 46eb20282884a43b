/*
 * bltkv8.h -- C ABI of the 8-bit paged KV cache: storing, attention over it, and attention over
 * selected pages of it (sm_100a).  Part of libbltdec.so; the decoder engine of bltdec.h uses the same
 * calls in a handle with BLT_FLAG_KV8_INT8 or BLT_FLAG_KV8_E4M3.
 *
 * Cache.  Keys and values are 8-bit codes in pages of page_tokens positions; a page table gives each
 * sequence's pages.  Every 16 positions of one head (a "block") share one exponent byte e, one for
 * keys and one for values:
 *     value = code * 2^(e - 127),    code: int8 in -127..127, or e4m3 (largest magnitude 448).
 * e is the least value >= 16 with amax <= top * 2^(e - 127) (amax: the block's largest magnitude,
 * top: 127 or 448); codes are rounded to nearest even.  The scale is a power of two, so values are
 * exact in bf16.  A value is off by at most half a step: 2^(e - 128) for int8 (at most amax / 127),
 * 2^-4 of itself (or 2^(e - 137) where e4m3 is subnormal) for e4m3.  In a block with magnitudes near
 * fp32's largest a code's value can lie beyond it: it reads back as infinity and counts as fp32's
 * largest in a summary and, if it was a number, when the block is quantised again.
 *
 * Conventions common to every call
 *   - The cache and its buffers belong to the caller; nothing is kept between calls, allocated, or
 *     waited for.  Every call queues kernels on `stream` (a cudaStream_t; NULL is the legacy default
 *     stream) and may be captured into a CUDA graph.  Calls need no workspace, so calls that read the
 *     same cache may overlap; a call that writes it (append) must not overlap another on its pages.
 *   - Descriptors (the structs below) are read during the call only.  Pointers inside are device
 *     pointers; what they point to is read by the queued work, at the time it runs.
 *   - Return value: BLT_OK, BLT_ERR_INVALID_ARG or BLT_ERR_CUDA (see bltdec.h);
 *     blt_kv8_last_error() gives this thread's last message.  Nothing is queued on an error.
 *   - Errors found on the device (a page number outside the pool, offsets or positions out of range)
 *     are skipped over and reported as BLT_ERR_DEVICE in *status, if that is given; the call's other
 *     work is done.  So is a wait inside a kernel that ran out (about a second; none should): the
 *     rows and heads concerned are then not written.
 *   - Calls run on the device that holds the cache's keys, whichever is current; every other pointer
 *     has to be one that this device may use, and `stream` one of its streams.
 *   - Rows of a call: sequence s owns rows row_offsets[s] .. row_offsets[s + 1] - 1 (at most max_rows).
 *     Rows outside every sequence are left as they were.
 */
#ifndef BLTKV8_H
#define BLTKV8_H

#include <stdint.h>

#include "bltdec.h" /* return codes */

#ifdef __cplusplus
extern "C" {
#endif

#define BLT_KV8_INT8 0
#define BLT_KV8_E4M3 1

#define BLT_T_F32 0
#define BLT_T_BF16 1
#define BLT_T_F16 2

typedef struct {
  int32_t format;       /* BLT_KV8_* */
  int32_t n_heads;      /* key/value heads */
  int32_t head_dim;     /* 32, 64, 96 or 128 */
  int32_t page_tokens;  /* multiple of 16, at most 256 */
  int32_t n_pages;      /* pages in the pool */
  int32_t batch;        /* sequences: rows of page_table, at most 65535 */
  int32_t max_pages;    /* page_table [batch][max_pages] (max_pages * page_tokens < 2^30) */
  int32_t reserved;     /* 0 */
  uint8_t *k, *v;       /* codes: page p, head h, position t, channel c at p * page_stride + (h * page_tokens + t) * head_dim + c */
  uint8_t *k_exp, *v_exp; /* exponents: p * exp_stride + h * (page_tokens / 16) + t / 16 */
  int64_t page_stride;  /* bytes between pages of k and of v: a multiple of 16; 0: dense.  k and v 16-byte aligned */
  int64_t exp_stride;   /* bytes between pages of k_exp and of v_exp; 0: dense */
  /* Summaries for blt_kv8_select, all NULL or none: per page and head the least and greatest value of each key
   * channel over the positions held, k_min / k_max = round(value / 2^(k_sexp - 127)), k_sexp as an int8 block's e. */
  int8_t *k_min, *k_max; /* p * sum_stride + h * head_dim + c; 8-byte aligned */
  uint8_t *k_sexp;       /* p * sexp_stride + h */
  int64_t sum_stride;    /* bytes: a multiple of 8; 0: dense */
  int64_t sexp_stride;   /* 0: dense */
  const int32_t *page_table; /* entries outside 0 .. n_pages - 1: no page */
  int32_t *status;           /* device word for BLT_ERR_DEVICE, or NULL */
} blt_kv8_cache;

/* Rows of keys and values: row r, head h, channel c at k + r * row_stride + h * head_stride + c (elements). */
typedef struct {
  void *k, *v;
  int32_t dtype;  /* BLT_T_* */
  int32_t n_rows; /* rows in k and v */
  int32_t max_rows; /* most rows of one sequence */
  int32_t reserved;
  int64_t row_stride, head_stride;
  const int32_t *row_offsets; /* [batch + 1] */
  const int32_t *start;       /* [batch] position of each sequence's first row */
} blt_kv8_rows;

/* Store rows at positions start[s], start[s] + 1, ...  Positions before start[s] are kept, positions
 * behind the last new row are dropped (their codes stay, unread).  A block that holds kept rows is
 * quantised again from their stored values and the new rows together, so a kept row can lose low
 * bits when the block's exponent grows: it is then off by at most one step of the largest exponent
 * the block has had.  NaN is stored as 0, infinities as the largest code (amax ignores both).
 * Summaries, if the cache has them, are brought up to date for every page that takes a row.
 * No two sequences of a call may store into the same page.  Errors: INVALID_ARG, CUDA. */
int blt_kv8_append(const blt_kv8_cache *c, const blt_kv8_rows *rows, void *stream);

/* The values at positions start[s] ..., written to rows (exact in BF16 and F32; rounded in F16).
 * Rows whose page is missing become 0.  Rows and heads must not share elements. */
int blt_kv8_read(const blt_kv8_cache *c, const blt_kv8_rows *rows, void *stream);

typedef struct {
  const void *q; /* row r, head h, channel c at r * q_row_stride + h * q_head_stride + c (elements) */
  void *out;     /* the same with its own strides; same dtype; must not overlap q, nor a row or head another */
  float *lse;    /* [n_rows][n_q_heads] log-sum-exp (natural, of the scaled scores), or NULL */
  int32_t dtype; /* BLT_T_* of q and out */
  int32_t n_q_heads; /* a multiple of n_heads; query head h reads head h / (n_q_heads / n_heads) */
  int32_t n_rows, max_rows;
  int32_t max_keys; /* expected largest row_limit: chooses the launch shape, and with it the order of the sums */
  float scale;      /* finite */
  int64_t q_row_stride, q_head_stride, out_row_stride, out_head_stride;
  const int32_t *row_offsets; /* [batch + 1] */
  const int32_t *row_limit;   /* [n_rows] row r attends positions 0 .. row_limit[r] - 1 of its sequence */
  /* Selected pages, or NULL for all: row r, head h attends only the positions < row_limit[r] in pages
   * (indices into its sequence's page_table row) sel_pages[(r * n_heads + h) * n_select ..], the first
   * sel_count[r * n_heads + h] of them, in increasing order; an entry that is negative, at least
   * max_pages or not greater than the one before it is ignored. */
  const int32_t *sel_pages, *sel_count;
  int32_t n_select;
  int32_t flags; /* 0, or BLT_KV8_TEST_STALL */
} blt_kv8_attention;

#define BLT_KV8_TEST_STALL 1 /* test only: in a call of many rows, the keys for the first sequence's last tile of 128
                                queries and head 0 never come; waits run out within about 10 ms */

/* out = softmax(scale q K^T) V over each row's visible keys; a row that sees no key gets out 0 and
 * lse -inf.  Sums, maxima and products accumulate in fp32; fp32 q is used to 22 bits, and weights
 * enter the value product with 22 (F32, F16) or 11 (BF16) bits.  Cut are channels of q 2^32 below the
 * row's largest, and weights times their block's value scale 2^32 below the largest value scale among
 * the blocks that the row sees; keys and values that a row does not see take nothing from it.  The
 * tensor cores cut sums to fp32 where they do not round them, so an output over n keys can be off by
 * n / 4 + 64 steps of 2^-23 of its sum of magnitudes; for F32 and many rows they are cut over 512 keys
 * at a time and rounded in between.  Scores have to lie in fp32's range.
 * Positions below row_limit have to be stored.  The same call gives the same bits; the order of the
 * sums, and with it the last bits, depends on max_rows, max_keys, batch and the limits of the rows
 * that share a tile.  n_rows = 0 or max_rows = 0: nothing is done.
 * Errors: INVALID_ARG, CUDA. */
int blt_kv8_attend(const blt_kv8_cache *c, const blt_kv8_attention *a, void *stream);

typedef struct {
  const void *q;
  int32_t dtype, n_q_heads, n_rows, max_rows, max_keys;
  int32_t n_select; /* pages to choose, 1 .. max_pages or more */
  int32_t n_sink, n_local; /* the first and the last visible pages, always chosen: n_sink + n_local <= n_select */
  int64_t q_row_stride, q_head_stride;
  const int32_t *row_offsets, *row_limit;
  int32_t *sel_pages, *sel_count; /* as in blt_kv8_attention, unused entries -1 */
} blt_kv8_selection;

/* Choose pages for each row and key/value head by an estimate of the largest q.k: with the row's query
 * head g in 8 bits (qi_c = round(q_c / 2^(eq - 127)), eq as an int8 block's e over the head's channels),
 *     score(page) = max over g of 2^(eq + k_sexp - 254) * sum_c max(qi_c k_min_c, qi_c k_max_c),
 * the sum in whole numbers (a score beyond fp32's range counts as its end, one below it as 0).  Of
 * the ceil(row_limit / page_tokens) visible pages the first n_sink and the last n_local are chosen,
 * then those with the highest scores (equal scores: the lower page first) until n_select are; all of
 * them if there are no more.  q and the summaries are rounded to nearest, so a page's largest q.k can
 * exceed its score: by half a step of q times the sum of the page's largest magnitudes, and half a step
 * of k_sexp times the sum of |q|.  NaN in q counts as 0, infinities as the largest code.  Needs
 * summaries.  Errors: INVALID_ARG (max_pages above 49152), CUDA. */
int blt_kv8_select(const blt_kv8_cache *c, const blt_kv8_selection *s, void *stream);

/* Message of this thread's last failed blt_kv8_* call ("" if none). */
const char *blt_kv8_last_error(void);

#ifdef __cplusplus
}
#endif
#endif /* BLTKV8_H */
