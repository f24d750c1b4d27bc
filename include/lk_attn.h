/*
 * lk_attn.h -- the attention step of a decode token, between the q|k|v
 * projection and the o projection of lk.h: new keys and values appended to a
 * paged cache with their rotation, and the attention that reads the cache,
 * per sequence or over a prefix that a batch shares.
 *
 * The conventions of lk.h hold: device pointers owned by the caller, nothing
 * allocated, asynchronous on the given stream, arguments checked before
 * anything is launched, cfg as everywhere (these calls use its pdl field).
 * Make the first call on a device before any stream capture there (it looks up
 * addresses and sets kernel attributes).  Device-side waits are bounded (option
 * "wait_us"); one that runs out ends its kernel and sets a bit of the error word
 * (lk_device_error): 64 in the streaming kernel, 128 in the tile kernel (which
 * is which: lk_attn_launches), the results being then undefined.
 *
 * The pages the other entry points cite have no counterpart of these; they
 * are the library's own.
 *
 * Rows.  A call works on B sequences of R new tokens each: M = B*R rows,
 * 0 <= M <= LK_MAX_BATCH, row b*R + r being token r of sequence b.  lens[b]
 * (int32, device) is the number of keys that sequence b has in the cache
 * with its R new ones.  B == 0 or R == 0 launches nothing, LK_OK.
 *
 * The cache.  k and v are pages of `page` tokens:
 *     [n_pages][n_kv][page][head_dim]
 * of f16, bf16 or int8 levels (n_pages * n_kv * page < 2^31); LK_KV_Q8 holds
 * one f16 scale per 32 values of a token's head in ks, vs
 * [n_pages][n_kv][page][head_dim/32] (NULL for the other types), the value
 * being scale * level.  k, v, ks and vs are 16-byte aligned; head_dim is 64 or
 * 128; page a power of two, 16 .. 1024.  Token j of
 * sequence b lies in page table[b*table_w + j/page] (int32, device), slot
 * j % page.  The table is B rows of table_w page numbers; a sequence has room
 * for table_w * page tokens.  A page number outside [0, n_pages) is never
 * followed: its tokens count as absent.  Sequences may share pages, except
 * those that an append writes.  Stored values below lens[b] must be finite,
 * scales finite and not negative; what lies behind them may be anything.  An
 * infinite value below lens[b] (what an append rounds past 65504 to f16) makes
 * results infinite or NaN, on its head and in the sequences that hold it only.
 */
#ifndef LK_ATTN_H
#define LK_ATTN_H

#include "lk.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { LK_KV_F16 = 0, LK_KV_BF16 = 1, LK_KV_Q8 = 2 } lk_kv_type;

/* A cache (the struct itself is HOST memory, read during the call only). */
typedef struct {
  void* k;
  void* v;
  uint16_t* ks;   /* LK_KV_Q8 only: f16 scales */
  uint16_t* vs;
  int type;       /* lk_kv_type */
  int n_kv;       /* key/value heads, >= 1 */
  int head_dim;
  int page;
  int n_pages;    /* >= 1 */
  int reserved;
} lk_kv_cache;

/*
 * Append the new tokens' keys and values, rotated, and rotate their queries.
 * Row b*R + r has position p = lens[b] - R + r in its sequence.  Per head of
 * q and k:
 *   with a gain (optional, f32 [head_dim]): x[i] = RN(x[i] * gain[i] /
 *     sqrt(mean(x^2) + eps)), formed in f64 and rounded to f32 once;
 *   rotation of the first `rot` values by row p0 + p of the tables cosines,
 *     sines (f32 [n_pos][rot/2]): pair (a, b) -> (RN(RN(a c) - RN(b s)),
 *     RN(RN(b c) + RN(a s))); the pairs are values (i, i + rot/2), or the
 *     neighbours (2i, 2i + 1) if `paired` is nonzero.
 * Then k and v are stored at token p: rounded to nearest to f16 / bf16, or
 * (LK_KV_Q8) per 32 values with a = max|v|: scale = RN16(min(RN(a/127),
 * 65504)), level = rn(v / scale) clamped to +-127, 0 where the scale is 0.
 *   q, k, v  f32 rows, row t at q + t*ld and so on (the column ranges of one
 *            fused projection output, or separate matrices of the same pitch);
 *            n_q, n_kv, n_kv heads of head_dim values.  16-byte aligned, ld a
 *            multiple of 4
 *   qr       f32 [M][n_q*head_dim], 16-byte aligned: the rotated queries; must
 *            not overlap q, k or v (LK_ERR_ARG)
 *   rot      0 (no rotation; the tables are not read), 64 or 128, at most head_dim
 *   p0       >= 0: added to a token's position for the tables (the length of
 *            a prefix that the sequences share)
 * A row is left out, nothing of it written (qr and cache), if p < 0
 * (a padding sequence has lens[b] <= 0), if p0 + p >= n_pos (rot > 0), or if
 * token p has no page (a full sequence: what attention then makes of the old qr
 * means nothing).  n_q is a positive multiple of n_kv, at most 4096.
 */
lk_status lk_kv_append(const lk_kv_cache* cache, const float* q, const float* k, const float* v, long ld, int n_q,
                       const int32_t* table, int table_w, const int32_t* lens, int B, int R, int p0,
                       const float* cosines, const float* sines, int n_pos, int rot, int paired,
                       const float* q_gain, const float* k_gain, float eps, float* qr, const lk_launch_cfg* cfg,
                       cudaStream_t stream);

/*
 * Attention of the M rows over their sequences' cached keys.  Query head h
 * reads key/value head h / (n_q / n_kv).  Row b*R + r sees the first
 * n = min(lens[b] - R + 1 + r, table_w * page) tokens of sequence b (itself
 * and what came before it), absent tokens excepted:
 *   out = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale * q.k_j - max)
 * and zeros where it sees none.  Sums and statistics are f32.  Keys and values
 * enter as stored (Q8 under many rows: as two f16 terms, to 2^-22), queries and
 * weights as two 16-bit terms of the cache's type (Q8: f16).  With W = sum_j p_j
 * |v_j| / sum_j p_j and A the largest scale * sum_i |q_i k_ji| of the row (f16, Q8:
 * with no |q_i| taken below 2^-17 of the row's largest, the terms end there), out is
 * within (2^-15 + c A) W of the exact value, c = 2^-17 (f16, Q8) or 2^-14 (bf16),
 * plus (2^-27 + N 2^-32) max|v| over its N tokens; on the whole far nearer (about
 * 2^-20 of its norm; 2^-18 where a bf16 cache goes through the tile kernel).
 * The result does not depend on timing: the same call gives the same bits.  The
 * same row may differ in its last bits between calls of other B, R, lens or
 * table_w (the keys are split between blocks by all of them).
 *   q     f32 [M][n_q*head_dim], 16-byte aligned, finite.  A head of a row that
 *         is not comes out as NaN if it sees a token, zeros if it sees none, and
 *         changes no other result (quantized words of NaN are unspecified)
 *   mode, out, hq, hl, hs   the result for the next projection, as
 *         lk_swiglu_quant gives it: out f32 [M][n_q*head_dim] (required under
 *         LK_DEQUANT, else optional; may be q), under LK_INT8ACT / LK_TWOPASS
 *         its words and scales as lk_quantize_act's
 *   ws    ws_bytes >= lk_attn_workspace_bytes(...), 16-byte aligned; its
 *         content needs no preparation and means nothing after the call.
 *         Calls that may run at the same time need separate ones
 *   What is written (out, hq, hl, hs, ws) must not overlap each other or
 *         anything that is read, but for out == q (LK_ERR_ARG)
 *   scale finite (1/sqrt(head_dim) as a rule)
 * Rows behind the last sequence are not touched.  LK_ERR_SHAPE also where the
 * key units of all items together, n_kv * B * ceil(R * n_q/n_kv / 8) * ceil(table_w *
 * page / 32) (and the prefix's), pass 2^31.
 */
lk_status lk_attn(const lk_kv_cache* cache, const float* q, int n_q, const int32_t* table, int table_w,
                  const int32_t* lens, int B, int R, float scale, lk_mode mode, float* out, int8_t* hq, int8_t* hl,
                  float* hs, void* ws, size_t ws_bytes, const lk_launch_cfg* cfg, cudaStream_t stream);

/*
 * lk_attn for a batch whose sequences continue one prefix of `prefix_len`
 * tokens, held once in the cache in the pages prefix_table lists (int32,
 * device, prefix_w of them; prefix_len <= prefix_w * page).  table and lens
 * describe each sequence's own tokens, which follow the prefix.  Row b*R + r
 * sees the whole prefix and the first lens[b] - R + 1 + r own tokens (none if
 * that is not positive); a sequence with lens[b] < 0 is padding and gets
 * zeros.  The prefix's keys and values are read for all rows together (a short
 * one by each sequence, where that is faster).
 * The other arguments are lk_attn's; prefix_len 0 is lk_attn (prefix_table
 * may then be NULL).
 */
lk_status lk_attn_shared(const lk_kv_cache* cache, const float* q, int n_q, const int32_t* prefix_table,
                         int prefix_w, int prefix_len, const int32_t* table, int table_w, const int32_t* lens, int B,
                         int R, float scale, lk_mode mode, float* out, int8_t* hq, int8_t* hl, float* hs, void* ws,
                         size_t ws_bytes, const lk_launch_cfg* cfg, cudaStream_t stream);

/* Bytes of the workspace of lk_attn (shared 0) or lk_attn_shared (shared 1);
 * 0 for arguments those calls refuse. */
size_t lk_attn_workspace_bytes(int n_q, int n_kv, int head_dim, int B, int R, int shared);

/* Kernels that such a call launches (lk_attn: prefix_len 0): the streaming
 * kernel (up to 8 query rows on each read of the keys) and / or the tile kernel
 * (tcgen05, up to 256; chosen by rows, type and prefix length), and the join of
 * their partial results; few sequences with little room (table_w * page tokens)
 * take the streaming kernel in clusters, which join their own.  0 for arguments
 * the calls refuse and for no rows. */
int lk_attn_launches(int type, int n_q, int n_kv, int head_dim, int B, int R, int prefix_len, int room);

#ifdef __cplusplus
}
#endif

#endif /* LK_ATTN_H */
