/*
 * kda_paged.h -- C ABI of the paged attention operators of the MI355X (gfx950)
 * KDA library.
 *
 * A hybrid model interleaves KDA layers with softmax attention layers, and a
 * step of its serving loop runs both over one ragged batch: the KDA layers over
 * the paged state pool (kda.h), the attention layers over a paged cache of keys
 * and values.  These entry points are the attention side:
 *
 *   kda_page_tables     block tables and slot maps of a step, from the requests'
 *                       lengths; its cu_seqlens also drives kda_chunk_fwd
 *   kda_kv_append       the step's new key and value rows into the cache
 *   kda_paged_attention attention of each request's new tokens over its pages,
 *                       causal, full or with a sliding window and first tokens
 *                       that stay visible; one new token per request is decode
 *
 * The cache.  K and V are pools [num_pages, Hkv, page_size, head_dim]; position t
 * of a request lives in page block_table[request][t / page_size], at offset
 * t % page_size.  A slot is page * page_size + offset.  Any page size >= 1 is
 * served.  A table entry outside [0, num_pages) is no page: its positions hold
 * no key.
 *
 * Status codes, dtypes, error text (kda_last_error) and the conventions on
 * ownership, host-side checks, streams and reentrancy are those of kda.h:
 * nothing is allocated, nothing is queued or written on an error, work is
 * queued on `stream`, and values in device memory are the caller's contract.
 * Whatever they hold, no kernel reads or writes outside the buffers described
 * by the arguments.
 */
#ifndef KDA_PAGED_H_
#define KDA_PAGED_H_

#include "kda.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * kda_page_tables_args -- a step's tables.  With c = max(context_lens[i], 0),
 * t = max(new_lens[i], 0) and P = page_size, request i has ceil(c / P) pages,
 * listed in its row of block_table, and needs ceil((c + t) / P); the missing
 * ones are taken from the front of free_pages, in request order, and written
 * into the row (in place; all other entries are left as they are).  Then
 *
 *   cu_seqlens[i]  = new tokens of the requests before i
 *   seq_lens[i]    = c + t
 *   positions[x]   = the position of new token x in its request
 *   slot_mapping[x] = its slot, -1 where it has no page
 *   pages_taken[0] = pages needed in all
 *
 * Entries of positions and slot_mapping behind the last new token are -1.  New tokens
 * past max_tokens have no entry in either; the other outputs, and the pages entered in
 * block_table, are the whole step's all the same.  When
 * free_pages runs out (pages_taken[0] > num_free), the tokens left over get
 * slot -1 and their table entries -1.  A position past the table's width has no
 * page.  Pages given out are distinct as long as those in free_pages are.  Sums
 * and lengths stay below 2^31.  No output may share memory with an input: the
 * seq_lens of one step serve the next as context_lens, but that step then needs
 * a seq_lens of its own (a call with shared memory is refused).
 *
 * Errors: KDA_ERR_ARG (NULL, bad struct, shared memory), KDA_ERR_SHAPE,
 * KDA_ERR_UNSUPPORTED (num_pages * page_size, max_pages * page_size or max_tokens
 * above 2^30).
 */
typedef struct kda_page_tables_args {
  size_t struct_size;          /* = sizeof(kda_page_tables_args) */
  const int32_t *context_lens; /* (device) [n] tokens already cached */
  const int32_t *new_lens;     /* (device) [n] tokens of this step */
  const int32_t *free_pages;   /* (device) [num_free] */
  int32_t *block_table;        /* (device) [n, max_pages], in place */
  int64_t table_stride;        /* entries between rows, 0 = max_pages */
  int32_t n, num_free, max_pages;
  int32_t page_size;           /* >= 1 */
  int32_t num_pages;           /* pages of the cache */
  int64_t max_tokens;          /* room in slot_mapping and positions */
  int64_t *slot_mapping;       /* (device) [max_tokens] */
  int32_t *positions;          /* (device) [max_tokens] or NULL */
  int32_t *cu_seqlens;         /* (device) [n + 1] */
  int32_t *seq_lens;           /* (device) [n] */
  int32_t *pages_taken;        /* (device) [1] */
  void *stream;                /* hipStream_t or NULL */
} kda_page_tables_args;

kda_status kda_page_tables(const kda_page_tables_args *a);

/*
 * kda_kv_append_args -- rows [T, Hkv, head_dim] of K and V copied to their cache
 * slots; a slot outside [0, num_pages * page_size) skips its token.  Slots are
 * distinct (of two equal ones, either token's bytes may land), and no slot is a
 * row that the call reads.
 *
 * Errors: KDA_ERR_ARG (NULL, bad struct, misaligned), KDA_ERR_DTYPE,
 * KDA_ERR_SHAPE, KDA_ERR_UNSUPPORTED (head_dim other than 64 or 128, num_pages *
 * page_size above 2^30, K or V of 2^35 bytes and more).
 */
typedef struct kda_kv_append_args {
  size_t struct_size;          /* = sizeof(kda_kv_append_args) */
  const void *k, *v;           /* (device) [T, Hkv, head_dim] dtype */
  void *k_cache, *v_cache;     /* (device) [num_pages, Hkv, page_size, head_dim] */
  const int64_t *slot_mapping; /* (device) [T] */
  int64_t total_tokens;        /* T >= 0 */
  int64_t k_stride, v_stride;  /* elements between tokens, 0 = Hkv * head_dim; a
                                  multiple of 16 bytes, at most 2^24 */
  int64_t k_page_stride, v_page_stride;  /* elements between pages, 0 = dense; a
                                  multiple of 16 bytes (K and V may share pages) */
  int32_t dtype;               /* kda_dtype */
  int32_t hkv, head_dim, page_size, num_pages;
  void *stream;                /* hipStream_t or NULL */
} kda_kv_append_args;

kda_status kda_kv_append(const kda_kv_append_args *a);

/*
 * kda_paged_attention_args -- attention over the cache.
 *
 * Request i owns rows [cu_seqlens[i], cu_seqlens[i+1]) of q and out, its newest
 * tokens: row x sits at position p = seq_lens[i] - (rows of i) + (x - first row
 * of i), and its own key is already in the cache.  Query head h reads kv head
 * h / (Hq / Hkv).  A row sees the keys at positions j <= p with
 *
 *   window == 0, or p - j < window, or j < sinks
 *
 * (the window counts the row's own key; sinks are the first tokens of the
 * request), that lie on a page of the table, and
 *
 *   out[x][h] = sum_j softmax_j(scale q[x][h] . k_j) v_j
 *   lse[x][h] = log sum_j exp(scale q[x][h] . k_j)
 *
 * Scores, softmax statistics and sums are held in fp32; for 16-bit types the
 * probabilities are rounded to the input type for their product with V, and out
 * is rounded once.  A row that sees no key (a position below 0, no page) gets
 * zeros and lse = -inf, as does one whose scores are all -inf.  Scaled scores stay
 * below 2.35e38 (fp32's largest over log2(e)), values below 2^119 over the number of
 * keys (they are summed with weights of up to 2^8 before the division).  What lies at
 * positions that a row does not see does not reach it, be it infinite or NaN.
 * Rows of out and lse behind the last request are left as they are.  A length
 * beyond the table's width reads the table's positions only.
 *
 * Long key ranges are cut into splits that run in parallel and are joined in a
 * fixed order, so equal calls give equal bits; the count is chosen from sizes
 * alone unless `splits` sets it.  The partial results lie in the workspace,
 * which one call uses at a time.
 *
 * Errors: KDA_ERR_ARG (NULL, bad struct, misaligned), KDA_ERR_DTYPE,
 * KDA_ERR_SHAPE, KDA_ERR_UNSUPPORTED (head_dim other than 64 or 128, T * Hq above
 * 2^25, n * Hkv near 2^24, max_pages * page_size above 2^30), KDA_ERR_WORKSPACE.
 */
typedef struct kda_paged_attention_args {
  size_t struct_size;          /* = sizeof(kda_paged_attention_args) */
  const void *q;               /* (device) [T, Hq, head_dim] dtype */
  const void *k_cache, *v_cache;  /* (device) [num_pages, Hkv, page_size, head_dim] */
  const int32_t *block_table;  /* (device) [n, max_pages] */
  const int32_t *cu_seqlens;   /* (device) [n + 1], 0, non-decreasing, <= T */
  const int32_t *seq_lens;     /* (device) [n] cached keys, the new ones included */
  void *out;                   /* (device) [T, Hq, head_dim] dtype */
  float *lse;                  /* (device) [T, Hq] or NULL */
  void *workspace;             /* (device) >= kda_paged_attention_workspace_size() */
  size_t workspace_bytes;
  int64_t total_tokens;        /* T: rows of q and out */
  int64_t q_stride;            /* elements between tokens, 0 = Hq * head_dim; a
                                  multiple of 16 bytes, at most 2^24 */
  int64_t k_page_stride, v_page_stride;  /* as kda_kv_append's */
  int64_t table_stride;        /* entries between rows, 0 = max_pages */
  int32_t dtype;               /* kda_dtype */
  int32_t n, hq, hkv;          /* hq % hkv == 0 */
  int32_t head_dim, page_size, num_pages, max_pages;
  int32_t window, sinks;       /* >= 0; window 0 = every earlier key */
  int32_t max_new_len;         /* planning hint: the longest request's new tokens,
                                  0 = unknown; results do not depend on it, but
                                  for the order of sums */
  int32_t splits;              /* 0 = auto, else at most that many (1..64) */
  float scale;                 /* > 0 and below 2.35e38 (head_dim^-0.5 is the usual value) */
  void *stream;                /* hipStream_t or NULL */
} kda_paged_attention_args;

/* Workspace bytes of the call (0 is possible).  Reads only sizes, window, sinks,
 * max_new_len and splits.
 *
 * The need follows the plan of these very sizes: with splits = 0 fewer tokens or requests
 * may be cut into more pieces and need more bytes, so a workspace asked for one shape is
 * not one for smaller shapes.  KDA_PAGED_ATTENTION_WORKSPACE_MAX bytes serve every call.
 * The pieces follow the table's width (max_pages), which is all that the host knows of the
 * lengths: a step whose requests are short asks for less over the columns that they use
 * (a smaller max_pages with the same table_stride), and one with splits = 1 for nothing. */
#define KDA_PAGED_ATTENTION_WORKSPACE_MAX (((size_t)1 << 30) + ((size_t)1 << 25))
kda_status kda_paged_attention_workspace_size(const kda_paged_attention_args *a, size_t *bytes);
kda_status kda_paged_attention(const kda_paged_attention_args *a);

#ifdef __cplusplus
}
#endif
#endif /* KDA_PAGED_H_ */
