/*
 * lk_moe.h -- the feed-forward step of a mixture-of-experts decoder's token:
 * each row's experts chosen from its router logits, and the products with the
 * chosen experts' Q8_0 matrices, in place of the gate/up and down projections
 * of lk.h.
 *
 * The conventions of lk.h hold: device pointers owned by the caller, nothing
 * allocated, asynchronous on the given stream, arguments checked before
 * anything is launched, cfg as everywhere (these calls use its pdl field; the
 * products also path: 2 the kernel for single rows, 3 the tensor-core kernel, LK_INT8ACT
 * and LK_TWOPASS only, 0 the library's choice, the same bits from both).
 * Make the first call on a device before any stream capture there (it looks up
 * addresses and sets kernel attributes).  Device-side waits are bounded (option
 * "wait_us"); one that runs out ends its kernel and sets bit 256 of the error
 * word (lk_device_error), the results being then undefined.
 *
 * The pages the other entry points cite have no counterpart of these; they
 * are the library's own.
 *
 * Rows and pairs.  A call works on M rows (tokens), 0 <= M <= LK_MAX_BATCH, with
 * k experts each, 1 <= k <= LK_MOE_MAX_K; ids int32 [M][k] (device) are their
 * numbers.  Pair t*k + j is expert ids[t][j] with row t.  A number outside
 * [0, E) is no expert: such a pair costs nothing and counts as absent (a row of
 * padding has k of them).  The same expert twice in a row is two pairs.
 *
 * Experts.  Matrix n of a stack [E][rows][K] is a Q8_0 matrix as everywhere
 * (levels int8, f16 scales [E][rows][K/32]), 16-byte aligned both.  rows and K
 * are multiples of 128, E <= LK_MOE_MAX_E, K <= LK_MOE_MAX_LEN, E * rows < 2^31, k * rows < 2^29.
 *
 * What a call writes must not overlap what it reads or anything else it writes
 * (LK_ERR_ARG).
 */
#ifndef LK_MOE_H
#define LK_MOE_H

#include "lk.h"

#ifdef __cplusplus
extern "C" {
#endif

#define LK_MOE_MAX_E 1024  /* experts */
#define LK_MOE_MAX_K 32    /* experts of a row */
#define LK_MOE_MAX_GROUPS 32
#define LK_MOE_MAX_LEN (1 << 30) /* values of a matrix's row */

typedef enum { LK_SCORE_SOFTMAX = 0, LK_SCORE_SIGMOID = 1 } lk_score;

/*
 * The experts of each row, by its router logits l (f32 [M][E], 4-byte aligned).
 *   s = softmax(l) over the row, or 1 / (1 + exp(-l))
 *   c = s + bias (f32 [E]) if there is one, which then decides the choice but
 *       is no part of the weights; without it the choice goes by l itself
 *   The E experts are n_group groups of neighbours (n_group divides E); a
 *   group's value is the sum of its group_sum (1 or 2) largest c (without a bias:
 *   of s; group_sum 1: its largest l); the top_group groups of the largest
 *   values stay (equal values: the lower number), the others' experts are out.
 *   ids: the k experts of the largest c, the largest first (equal values: the
 *   lower number); weights: scale * s, with renorm nonzero over the sum of the k.
 * Choices are those of s, c and the groups' sums in f64: where f32 does not
 * decide, f64 does.  Weights are f32, within 2^-15 of their values relatively (2^-126 below
 * f32's normal range); with renorm they are 0 where no sigmoid of the k is in
 * that of f64 (logits below -708).
 * An expert whose logit is NaN or -inf, or whose bias is not finite, is out; a
 * logit of +inf counts as the largest f32.  Where fewer than k are left, the rest
 * are -1 with weight 0.
 *   ids int32 [M][k], weights f32 [M][k]
 * 1 <= E <= LK_MOE_MAX_E, 1 <= k <= min(E, LK_MOE_MAX_K), scale finite.
 */
lk_status lk_moe_route(const float* logits, const float* bias, int M, int E, lk_score score, int n_group,
                       int top_group, int group_sum, int k, int renorm, float scale, int32_t* ids, float* weights,
                       const lk_launch_cfg* cfg, cudaStream_t stream);

/*
 * The gate and up products of every pair and their SwiGLU: with e = ids[t][j],
 *   h[t*k + j] = swiglu(Wg_e x_t, Wu_e x_t),
 * each product as lk_gemv_q8 forms it in this mode (the same bits in the
 * quantized modes; LK_DEQUANT within 1e-5 of sum |w x|, its f32 sums over
 * 4096 values at most added without loss), the SwiGLU as lk_swiglu_quant.  An absent pair's rows are
 * left as they are.
 *   wg, wsg / wu, wsu   stacks [E][F][K]
 *   x, xq, xl, xs       the M rows by mode, as lk_gemv_q8's, 16-byte aligned
 *   h    f32 [M*k][F], 16-byte aligned: always written
 *   hq, hl, hs   optional together (hq NULL: none; LK_INT8ACT, LK_TWOPASS): h's
 *        words and scales as lk_quantize_act's, [M*k][F], [M*k][F], [M*k][F/32],
 *        16-byte aligned
 *   cnt  with hq: int32 [M*k*F/32] zeroed by the caller before the first call;
 *        every completed call leaves it zeroed (after LK_ERR_DEVICE_TIMEOUT zero it
 *        again).  Calls that may run at the same time need separate ones
 * LK_ERR_SHAPE where the row of x does not fit in shared memory (K up to 32768
 * always does): LK_DEQUANT, and with path 2 (the library's choice is path 3 then).
 */
lk_status lk_moe_glu_q8(const int8_t* wg, const uint16_t* wsg, const int8_t* wu, const uint16_t* wsu, int E, int F,
                        int K, lk_mode mode, const float* x, const int8_t* xq, const int8_t* xl, const float* xs, int M,
                        const int32_t* ids, int k, float* h, int8_t* hq, int8_t* hl, float* hs, int* cnt,
                        const lk_launch_cfg* cfg, cudaStream_t stream);

/*
 * The down products of every pair, summed with the routing weights:
 *   y[t] = sum over j of weights[t][j] * (Wd_e h[t*k + j]),  e = ids[t][j],
 * each product as lk_gemv_q8 forms it in this mode, the sum over the present
 * pairs as f32 fused multiply-adds in ascending j from 0 (a row without any: 0).
 *   wd, wsd   stack [E][N][F]
 *   h, hq, hl, hs   the M*k pairs' rows by mode, as lk_moe_glu_q8 writes them,
 *             16-byte aligned
 *   weights   f32 [M][k];  y  f32 [M][N], 16-byte aligned
 * LK_ERR_SHAPE where a row's k activations do not fit in shared memory (k * F up to
 * 32768 always do): LK_DEQUANT, and with path 2 (the library's choice is path 3 then).
 */
lk_status lk_moe_down_q8(const int8_t* wd, const uint16_t* wsd, int E, int N, int F, lk_mode mode, const float* h,
                         const int8_t* hq, const int8_t* hl, const float* hs, int M, const int32_t* ids,
                         const float* weights, int k, float* y, const lk_launch_cfg* cfg, cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* LK_MOE_H */
