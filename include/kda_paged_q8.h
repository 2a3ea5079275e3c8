/*
 * kda_paged_q8.h -- C ABI of the paged cache in 8 bits of the MI355X (gfx950) KDA library.
 *
 * The attention side of a serving step (kda_paged.h) over a cache of half the bytes:
 *
 *   kda_kv_append_q8        a step's new key and value rows into the cache
 *   kda_kv_read_q8          cached rows of requests read back
 *   kda_paged_attention_q8  attention of the step's new tokens over it
 *
 * The cache.  K and V are pools [num_pages, Hkv, page_size, head_dim] of one-byte codes,
 * each with scales [num_pages, Hkv, page_size / block] fp32 (dense): one for `block`
 * consecutive positions of a page and head, block a divisor of page_size (from 1, a scale
 * per token, to page_size, one per page).  A code c of a block with scale s stands for s * c:
 *
 *   KDA_E4M3  c is the e4m3 number (448 at most, no infinities; 0x7f and 0xff are NaN)
 *   KDA_INT8  c is the signed number, -127 .. 127
 *
 * Scales are powers of two, 2^-126 at least: a division by one is exact, so that the code is the only
 * rounding, and every value of the cache (4 or 7 significant bits) is a bf16 number (but for e4m3's below
 * 2^-133, at scales below 2^-124).  All three
 * read a scale by its exponent: one that is no power of two (from elsewhere, as the largest magnitude
 * over 448) counts as the next power of two below, and an append that adds rows to its block
 * leaves a power of two there.
 *
 * All three address rows alike: request i owns rows [cu_seqlens[i], cu_seqlens[i+1]),
 * its newest positions: row x is at position p = seq_lens[i] - (rows of i) + (x - first row of i),
 * which lies on page block_table[i][p / page_size] at offset p % page_size.  A table entry
 * outside [0, num_pages) is no page.  Lengths and offsets stay below 2^31.
 *
 * Status codes, dtypes, error text (kda_last_error) and the conventions on ownership,
 * host-side checks, streams and reentrancy are those of kda.h: nothing is allocated,
 * nothing is queued or written on an error, work is queued on `stream`, and values in
 * device memory are the caller's contract.  Whatever they hold, no kernel reads or writes
 * outside the buffers described by the arguments.  Outputs share no memory with inputs or one another.
 */
#ifndef KDA_PAGED_Q8_H_
#define KDA_PAGED_Q8_H_

#include "kda_paged.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum kda_code {
  KDA_E4M3 = 0,
  KDA_INT8 = 1
} kda_code;

/*
 * kda_kv_append_q8_args -- rows [T, Hkv, head_dim] of K and V to their places in the cache;
 * a row without a page or with a position below 0 is skipped, as are rows behind the last request.
 *
 * For every block of the cache and head that the call's rows fall into, with `need` the least power of
 * two (2^-126 at least) such that the rows' finite magnitudes are at most need * 448 (need *
 * 127 for int8):
 *
 *   the block's first position is among the rows:  scale = need
 *   otherwise:  scale = max(scale, need), and where that is more, the codes at the
 *               block's earlier positions are rounded to it (a scale there that is no finite
 *               number counts for nothing: scale = need)
 *
 * and the rows' codes are their values over the scale, rounded to nearest, ties to even.
 * NaN and infinities have no part in `need`: e4m3 holds NaN for them, int8 0 for NaN and
 * +-127 for +-infinity.  Positions of the block behind the rows are left as they are.  Rows enter a
 * block in order: one that is written again (a rejected draft) keeps the block's scale.
 * Magnitudes stay below 2^127.  A page that receives rows is listed once in the table.
 *
 * Errors: KDA_ERR_ARG (NULL, bad struct, misaligned), KDA_ERR_DTYPE (dtype, code), KDA_ERR_SHAPE,
 * KDA_ERR_UNSUPPORTED (head_dim other than 64 or 128, num_pages * page_size or max_pages *
 * page_size above 2^30, (T / block + 2 n) * Hkv not below 2^24).
 */
typedef struct kda_kv_append_q8_args {
  size_t struct_size;          /* = sizeof(kda_kv_append_q8_args) */
  const void *k, *v;           /* (device) [T, Hkv, head_dim] dtype */
  void *k_cache, *v_cache;     /* (device) [num_pages, Hkv, page_size, head_dim] codes */
  float *k_scale, *v_scale;    /* (device) [num_pages, Hkv, page_size / block] */
  const int32_t *block_table;  /* (device) [n, max_pages] */
  const int32_t *cu_seqlens;   /* (device) [n + 1], 0, non-decreasing, <= T */
  const int32_t *seq_lens;     /* (device) [n] cached positions, the new ones included */
  int64_t total_tokens;        /* T >= 0 */
  int64_t k_stride, v_stride;  /* elements between tokens, 0 = Hkv * head_dim; a
                                  multiple of 16 bytes, at most 2^24 */
  int64_t k_page_stride, v_page_stride;  /* bytes between pages, 0 = dense; a multiple of 16 */
  int64_t table_stride;        /* entries between rows, 0 = max_pages */
  int32_t dtype, code;         /* kda_dtype, kda_code */
  int32_t n, hkv, head_dim, page_size, block, num_pages, max_pages;
  void *stream;                /* hipStream_t or NULL */
} kda_kv_append_q8_args;

kda_status kda_kv_append_q8(const kda_kv_append_q8_args *a);

/*
 * kda_kv_read_q8_args -- the values of the requests' rows, rounded to dtype; zeros for a
 * row without a page or with a position below 0.  Rows of k_out and v_out behind the last request are
 * left as they are.  cu_seqlens of the running sums of seq_lens reads whole contexts.
 *
 * Errors: as kda_kv_append_q8, with T / 4 + n not below 2^24 in place of the blocks.
 */
typedef struct kda_kv_read_q8_args {
  size_t struct_size;          /* = sizeof(kda_kv_read_q8_args) */
  const void *k_cache, *v_cache;
  const float *k_scale, *v_scale;
  const int32_t *block_table;
  const int32_t *cu_seqlens;
  const int32_t *seq_lens;
  void *k_out, *v_out;         /* (device) [T, Hkv, head_dim] dtype, dense */
  int64_t total_tokens;
  int64_t k_page_stride, v_page_stride;
  int64_t table_stride;
  int32_t dtype, code;
  int32_t n, hkv, head_dim, page_size, block, num_pages, max_pages;
  void *stream;
} kda_kv_read_q8_args;

kda_status kda_kv_read_q8(const kda_kv_read_q8_args *a);

/*
 * kda_paged_attention_q8_args -- kda_paged_attention over the values that the cache
 * stands for: the same rows, masks, splits, workspace and guarantees, with q and out in
 * bf16 or fp16 (a check in fp32 reads the cache back and attends over that).
 *
 * The values' magnitudes stay below 2^99 (rows in fp16: 65520).  In fp16 the values are rounded to
 * fp16 first, which changes only those below its normal numbers.  Scores, sums and softmax statistics
 * are fp32.  Probabilities are rounded to q's type, or, in a call whose requests have up to 32 rows per kv
 * head (by max_new_len), to bf16 after the product with V's scale: as a pair of bf16 (16 bits) up to 16
 * rows and in fp16.  What a hidden position's codes and its
 * block's scale hold does not reach a row that does not see it.
 *
 * Errors: as kda_paged_attention, and KDA_ERR_DTYPE for fp32 or an unknown code.
 */
typedef struct kda_paged_attention_q8_args {
  size_t struct_size;          /* = sizeof(kda_paged_attention_q8_args) */
  const void *q;               /* (device) [T, Hq, head_dim] dtype */
  const void *k_cache, *v_cache;  /* (device) [num_pages, Hkv, page_size, head_dim] codes */
  const float *k_scale, *v_scale; /* (device) [num_pages, Hkv, page_size / block] */
  const int32_t *block_table;  /* (device) [n, max_pages] */
  const int32_t *cu_seqlens;   /* (device) [n + 1], 0, non-decreasing, <= T */
  const int32_t *seq_lens;     /* (device) [n] cached keys, the new ones included */
  void *out;                   /* (device) [T, Hq, head_dim] dtype */
  float *lse;                  /* (device) [T, Hq] or NULL */
  void *workspace;             /* (device) >= kda_paged_attention_q8_workspace_size() */
  size_t workspace_bytes;
  int64_t total_tokens;        /* T: rows of q and out */
  int64_t q_stride;            /* elements between tokens, 0 = Hq * head_dim; a
                                  multiple of 16 bytes, at most 2^24 */
  int64_t k_page_stride, v_page_stride;  /* bytes between pages, 0 = dense; a multiple of 16 */
  int64_t table_stride;        /* entries between rows, 0 = max_pages */
  int32_t dtype, code;         /* kda_dtype (bf16 or fp16), kda_code */
  int32_t n, hq, hkv;          /* hq % hkv == 0 */
  int32_t head_dim, page_size, block, num_pages, max_pages;
  int32_t window, sinks, max_new_len, splits;  /* as kda_paged_attention's */
  float scale;
  void *stream;                /* hipStream_t or NULL */
} kda_paged_attention_q8_args;

/* As kda_paged_attention_workspace_size; KDA_PAGED_ATTENTION_WORKSPACE_MAX bytes serve every call. */
kda_status kda_paged_attention_q8_workspace_size(const kda_paged_attention_q8_args *a, size_t *bytes);
kda_status kda_paged_attention_q8(const kda_paged_attention_q8_args *a);

#ifdef __cplusplus
}
#endif
#endif /* KDA_PAGED_Q8_H_ */
