/*
 * kda_rotary.h -- C ABI of the rotary positions of the MI355X (gfx950) KDA library.
 *
 * The softmax attention layers between KDA layers may turn their query and key rows to
 * their positions before the keys enter the paged cache (kda_paged.h, kda_paged_q8.h);
 * kda_page_tables gives the positions of a step's tokens.
 *
 * Status codes, dtypes, error text (kda_last_error) and the conventions on ownership,
 * host-side checks, streams and reentrancy are those of kda.h: nothing is allocated,
 * nothing is queued or written on an error, work is queued on `stream`, and values in
 * device memory are the caller's contract.
 */
#ifndef KDA_ROTARY_H_
#define KDA_ROTARY_H_

#include "kda.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * kda_rotary_args -- rows of q and, where k is not NULL, of k, turned to their positions.
 * Pair i of a head's first 2 * pairs channels is (x, y) = channels (i, i + pairs), or
 * (2 i, 2 i + 1) with interleaved != 0.  With the angle a = positions[t] * frequencies[i],
 *
 *   x' = scale (x cos a - y sin a)      y' = scale (x sin a + y cos a)
 *
 * and -a in place of a with inverse != 0: the transpose, which takes the gradient of
 * the result to that of the rows.  The other channels pass unchanged.  Rows at a negative
 * position are left as they are (not written): those behind a step's last token.
 *
 * Angles are reduced to a part of a turn in fp64 (off by less than 2^-20 turns at position 2^31),
 * sines, cosines and products are fp32, and a result is rounded once to the rows' type.
 * Outputs are the inputs themselves (the same address and stride) or share no memory with
 * them or with one another.
 *
 * Errors: KDA_ERR_ARG (NULL, bad struct, misaligned, shared memory), KDA_ERR_DTYPE, KDA_ERR_SHAPE,
 * KDA_ERR_UNSUPPORTED (head_dim not a multiple of 8 or above 512, rows that need more than
 * 2^31 - 1 pieces of 16 bytes, more than 2^26 - 4 tokens).
 */
typedef struct kda_rotary_args {
  size_t struct_size;          /* = sizeof(kda_rotary_args) */
  const void *q, *k;           /* (device) [T, Hq, head_dim], [T, Hk, head_dim] dtype; k may be NULL */
  void *q_out, *k_out;         /* (device) the same shapes */
  const int32_t *positions;    /* (device) [T] */
  const double *frequencies;   /* (device) [pairs] radians per position */
  int64_t total_tokens;        /* T >= 0 */
  int64_t q_stride, k_stride;  /* elements between tokens, 0 = dense; multiples of 16 bytes,
                                  at most 2^24 */
  int64_t q_out_stride, k_out_stride;  /* the same of the outputs */
  int32_t dtype;               /* kda_dtype */
  int32_t hq, hk;              /* hk is ignored where k is NULL */
  int32_t head_dim;
  int32_t pairs;               /* 1 .. head_dim / 2 */
  int32_t interleaved, inverse;
  float scale;                 /* finite; the attention factor of a stretched context, usually 1 */
  void *stream;                /* hipStream_t or NULL */
} kda_rotary_args;

kda_status kda_rotary(const kda_rotary_args *a);

#ifdef __cplusplus
}
#endif
#endif /* KDA_ROTARY_H_ */
