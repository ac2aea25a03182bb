/*
 * mhc_attention.h -- C ABI of attention over a paged key-value cache.
 *
 * The attention sublayer between two mHC boundaries (mhc_boundary.h), for
 * serving: its projections are products of mhc_sublayer.h, its output is a
 * partial of the next boundary.
 *
 *   append  rotates the queries and keys of new tokens by their positions and
 *           writes keys and values into the cache
 *   attend  attention of each sequence's newest tokens over its cache: one
 *           token of each (decode), or any number (prompts, chunks of them,
 *           proposed tokens), causal, with an optional window and first
 *           positions that stay visible
 *
 * The cache: `pages` pages of page_size positions, for the keys
 * [pages][kv_heads][page_size][head_dim] and the same for the values; a page
 * is dense, pages lie *_page_stride elements apart.  BF16, or with
 * MHC_ATTENTION_FP8 E4M3 values with one positive FP32 scale for each position
 * and head, [pages][kv_heads][page_size] (dense); a value stands for value *
 * scale, and append takes the scale as amax / 448 of the row's largest
 * magnitude, floored at 2^-100, in the steps of mhc_sublayer.h.  A row of the
 * page table names a sequence's pages in order: position p is at offset p %
 * page_size of page table[p / page_size].  Pages may be shared by sequences
 * (a common prefix).
 *
 * Conventions: as in mhc_boundary.h (device pointers, caller-owned buffers,
 * every argument checked before the first launch, nothing aborts or traps).
 * A token's heads are contiguous; a *_stride is the distance of two tokens (or
 * of two rows of the page table) in elements.  BF16 and 8-bit rows and
 * the scales start on 16-byte boundaries.  Calls without tokens succeed and launch nothing.  What
 * lies in device memory is checked by the kernels: a page, slot, length or
 * start that is out of range is never followed, what it stands for is taken
 * as not there, and mhc_attention_check_errors reports it.  A handle owns
 * scratch that attend uses: its attend calls (and graphs that hold them) run
 * one after another, on one stream or on streams that the caller orders.
 */
#ifndef MHC_ATTENTION_H
#define MHC_ATTENTION_H

#include "mhc_boundary.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Config flags. */
enum {
  /* The cache is 8-bit with scales (else BF16). */
  MHC_ATTENTION_FP8 = 1u << 0,
  /* A rotation takes neighbouring elements (2i, 2i + 1) of a head, not (i, i +
   * rotary_dim / 2). */
  MHC_ATTENTION_INTERLEAVED = 1u << 1
};

/* Construction arguments.  heads is a multiple of kv_heads, at most 128 times
 * it; query head h reads key and value head h / (heads / kv_heads).  head_dim:
 * 64 or 128.  page_size: 16, 32, 64 or 128.  rotary_dim: the first elements of
 * a head that append rotates, a multiple of 16 up to head_dim, or 0 for none;
 * pair i of position p by the angle p * f(i), with f(i) = frequencies[i]
 * (rotary_dim / 2 values between -2^40 and 2^40 in host memory, read by create) or,
 * where that is NULL, theta^(-2i / rotary_dim), a double either way.  An angle's
 * whole turns are dropped exactly: f(i) / 2 pi is held in 64 bits behind the
 * point, and off by 2^-64 turns a position. */
typedef struct {
  int32_t heads, kv_heads, head_dim, page_size;
  int32_t rotary_dim;
  uint32_t flags;            /* MHC_ATTENTION_* */
  double theta;
  const double *frequencies;
} mhc_attention_config_t;

/* Token t goes to its slot, page * page_size + offset; slot -1 is a padding
 * token, which is not written to the cache.  No slot is given twice in a call
 * (which token it keeps would be open).  q_out (NULL: none) takes the rotated
 * queries of all tokens, padding too; it may be q itself.  q and q_out go
 * together; k and v are always given.  Strides are multiples of 8. */
typedef struct {
  int32_t tokens;
  int32_t pages;
  const void *q;             /* [tokens][heads][head_dim] bf16 or NULL */
  int64_t q_stride;
  const void *k;             /* [tokens][kv_heads][head_dim] bf16 */
  int64_t k_stride;
  const void *v;
  int64_t v_stride;
  const int32_t *positions;  /* [tokens] */
  const int32_t *slots;      /* [tokens] */
  void *q_out;               /* [tokens][heads][head_dim] bf16 or NULL */
  int64_t q_out_stride;
  void *k_cache;
  int64_t k_page_stride;
  void *v_cache;
  int64_t v_page_stride;
  float *k_scales;           /* MHC_ATTENTION_FP8 only */
  float *v_scales;
} mhc_attention_append_args_t;

/* Sequence s has lengths[s] positions in the cache, its newest tokens' among
 * them (append comes first), and the queries q_starts[s] .. q_starts[s + 1] - 1;
 * without q_starts one query, s (tokens = sequences).  Query i of n stands at
 * position p = lengths[s] - n + i and sees the positions j <= p with, where window
 * > 0, j > p - window or j < sinks.  A query's row of output is
 *   sum over j of exp(x_j) v_j / sum over j of exp(x_j),  x_j = scale * q k_j,
 * and lse the logarithm of the lower sum (natural); a row that sees nothing, or
 * whose scores are all minus infinity, has zeros and minus infinity.  Positions that a query does not see may hold
 * anything.  Rows of output from q_starts[sequences] on are left as they are.
 * A sequence with a start that is out of range (0 .. tokens) or whose two starts
 * decrease, and every sequence behind it, has no queries: their rows are left as
 * they are.
 * The softmax and all sums are held in FP32.  Sums of finite values are finite,
 * whatever their size, and values from 2^-90 on have all their bits (over an 8-bit
 * cache, in calls with q_starts or more than 16 heads for each kv head: values from
 * 2^-70 to 2^110).  In calls with q_starts or with more than 16 heads for each kv
 * head the weights are rounded to BF16, and over an 8-bit cache queries are off by
 * at most 2^-17 of their head's largest element (0 for elements from 2^-9 of it
 * on); in the others weights keep 16 bits over a BF16 cache, and over an 8-bit one
 * FP16's 11 (fewer below 2^-21 of the largest, where they are off by 2^-32 of it),
 * and queries are off by at most 2^-25 of their head's largest element.
 * output and lse overlap no input. */
typedef struct {
  int32_t tokens, sequences;
  int32_t pages;
  int32_t table_width;       /* pages that a row of the table has room for */
  const void *q;             /* [tokens][heads][head_dim] bf16 */
  int64_t q_stride;
  const int32_t *q_starts;   /* [sequences + 1], not decreasing, or NULL */
  const int32_t *lengths;    /* [sequences], at most table_width * page_size */
  const int32_t *page_table; /* [sequences][table_width] */
  int64_t table_stride;
  const void *k_cache;
  int64_t k_page_stride;
  const void *v_cache;
  int64_t v_page_stride;
  const float *k_scales;     /* MHC_ATTENTION_FP8 only */
  const float *v_scales;
  float scale;               /* positive */
  int32_t window, sinks;     /* window 0: every position up to the query's */
  void *output;              /* [tokens][heads][head_dim] bf16 */
  int64_t output_stride;
  float *lse;                /* [tokens][heads] or NULL */
} mhc_attention_attend_args_t;

typedef struct mhc_attention mhc_attention_t; /* opaque, library-owned */

mhc_status_t mhc_attention_create(const mhc_attention_config_t *config, int device, mhc_attention_t **out);
mhc_status_t mhc_attention_append(mhc_attention_t *a, const mhc_attention_append_args_t *args, mhc_stream_t stream);
mhc_status_t mhc_attention_attend(mhc_attention_t *a, const mhc_attention_attend_args_t *args, mhc_stream_t stream);
/* Synchronises the device and reports what kernels of earlier calls met:
 * MHC_ERR_TIMEOUT if one gave up a bounded wait (its outputs are not valid),
 * MHC_ERR_INVALID_ARG if a page, slot, length or start was out of range.  The
 * report is then cleared and the scratch made ready for the next call. */
mhc_status_t mhc_attention_check_errors(mhc_attention_t *a);
mhc_status_t mhc_attention_destroy(mhc_attention_t *a);
/* Message of the last failing call on `a` (NULL: of the last failing create). */
const char *mhc_attention_last_error(const mhc_attention_t *a);

#ifdef __cplusplus
}
#endif

#endif
