/*
 * lk_sample.h -- the next token drawn from the logits, beside lk_argmax of lk.h.
 *
 * The conventions of lk.h hold (device pointers owned by the caller, nothing
 * allocated, asynchronous on the given stream, arguments checked before
 * anything is launched; cfg's pdl field is used).  The source pages have no
 * counterpart; the entry point is the library's own.
 */
#ifndef LK_SAMPLE_H
#define LK_SAMPLE_H

#include "lk.h"

#ifdef __cplusplus
extern "C" {
#endif

#define LK_SAMPLE_MAX_N (1 << 21) /* logits of a row */

/*
 * One token for each of M rows of logits l (f32 [M][N], 4-byte aligned, 0 <= M <=
 * LK_MAX_BATCH, 1 <= N <= LK_SAMPLE_MAX_N), from the given random numbers.  Settings are f32 / int32
 * [M] device arrays, one of each row; NULL turns one off for all.  Of a row:
 *   e_i = exp((l_i - max l) / temperature).  Temperature not above 0 (or NaN): the
 *         first of the largest logits, probability 1, nothing drawn.
 *   Tokens are ordered by l, the largest first (equal values: the lower index).
 *   top_k > 0    the first top_k of the order stay
 *   top_p < 1    of these the shortest beginning whose sum of e reaches top_p
 *                times theirs, at least one token
 *   min_p > 0    of these the ones with e_i >= min(min_p, 1)
 *   idx          the lowest index i such that the sum of e over the tokens that
 *                stay, from the lowest index up to i, exceeds u times their sum
 *                (u >= 1: as the largest number below 1)
 *   prob         optional f32 [M]: e_idx over that sum, to 2^-22 relatively
 * A logit of NaN counts as -inf (never drawn), +inf as the largest f32; a row
 * without any other gets idx -1, prob 0.  A difference of logits past f32's range is an
 * infinite one.  The e are formed to 2^-29 relatively; those below 2^-48.5 count
 * as 0, all of them together less than N 2^-48.5; sums are within 2^-28 but for
 * these: the token differs from the exact one only where u or top_p lies within 2^-27 (N
 * above 2^18: 2^-26) of a border between tokens, or min_p within 2^-29 of a
 * token's e, relatively.  The same call gives the same bits; the same row among others
 * (M, or another alignment of its logits) the same token but for such borders.
 *   u    f32 [M], >= 0 (below 0 or NaN: 0);  idx int32 [M]
 * What is written must not overlap what is read (LK_ERR_ARG).
 */
lk_status lk_sample(const float* logits, int M, int N, const float* temperature, const int32_t* top_k,
                    const float* top_p, const float* min_p, const float* u, int32_t* idx, float* prob,
                    const lk_launch_cfg* cfg, cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* LK_SAMPLE_H */
