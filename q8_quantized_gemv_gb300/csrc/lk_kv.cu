// New keys and values into a paged cache, with the per-head norm and the
// rotation of q and k on the way (include/lk_attn.h, lk_kv_append).
//
// A warp takes one head of one row: lane l holds the values l + 32 c, so a
// rotation pair (i, i + rot/2) is in one lane (rot/2 is a multiple of 32), a
// neighbour pair in lanes l and l ^ 1, and a Q8 group of 32 values is one
// value per lane.  Every operation is rounded as the header writes it, so
// the results are bit-fixed.  A few KB a row: the call is bound by its launch
// and one chain of dependent loads (lens -> table, beside the row itself): 2.1 us
// for one row of 32 + 8 + 8 heads of 128, 3.4 us for 64 rows to Q8, 5.5 with the
// norm (3 MB, 0.4 us of memory time; f64 for every head made it 16.6): of its 2560
// normed heads some 7 have a value so near a rounding boundary that the f64 form
// decides (378 f64 instructions counted), and the call waits for that one's chain of
// a sum, a root and quotients, some 2.5 us.  One row's 40 mostly have none.
#include <cuda_bf16.h>

#include "lk_attn.cuh"

using namespace lk;
using namespace lkh;

namespace {

struct AppendArgs {
  const float* q;
  const float* k;
  const float* v;
  long ld;
  int n_q, n_kv, page_log2, n_pages;
  void* ck;
  void* cv;
  __half* cks;
  __half* cvs;
  const int* table;
  int table_w;
  const int* lens;
  int R, p0;
  const float* cosines;
  const float* sines;
  int n_pos, rot, paired;
  const float* q_gain;
  const float* k_gain;
  float eps;
  float* qr;
  long heads;  // rows * (n_q + 2 n_kv)
};

template <int TYPE, int D>
__device__ __forceinline__ void store_head(void* base, __half* scales, long row, const float (&x)[D / 32], int lane) {
#pragma unroll
  for (int c = 0; c < D / 32; ++c) {
    const long i = row * D + 32 * c + lane;
    if constexpr (TYPE == LK_KV_F16) ((__half*)base)[i] = __float2half_rn(x[c]);
    if constexpr (TYPE == LK_KV_BF16) ((__nv_bfloat16*)base)[i] = __float2bfloat16_rn(x[c]);
    if constexpr (TYPE == LK_KV_Q8) {
      const __half s = __float2half_rn(fminf(div127(warp_absmax(x[c])), 65504.0f));
      const float f = __half2float(s);
      const int z = f > 0.0f ? __float2int_rn(fminf(fmaxf(__fdiv_rn(x[c], f), -127.0f), 127.0f)) : 0;
      ((int8_t*)base)[i] = (int8_t)z;
      if (lane == 0) scales[row * (D / 32) + c] = s;
    }
  }
}

// ---- the per-head norm ----------------------------------------------------------------
// x[i] = RN32(x[i] g[i] / sqrt(mean(x^2) + eps)) with everything inside in f64.
template <int C>
__device__ __forceinline__ void norm_f64(float (&x)[C], const float (&g)[C], float eps) {
  double ss = 0.0;
#pragma unroll
  for (int c = 0; c < C; ++c) ss = __fma_rn((double)x[c], (double)x[c], ss);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(FULL, ss, o);
  const double den = __dsqrt_rn(ss / (32 * C) + (double)eps);
#pragma unroll
  for (int c = 0; c < C; ++c) x[c] = __double2float_rn(__ddiv_rn((double)x[c] * (double)g[c], den));
}

// The same values from pairs of f32 (unevaluated sums hi + lo, T. J. Dekker,
// Numer. Math. 18, 1971), about 2^-44 accurate: the f64 pipe issues a warp's
// instruction in 16 cycles and the 45 of a head took 14 of the 17 us of 64
// rows.  Returns whether the lane's results are certainly the f64 form's: no
// value within 2^-40 of a rounding boundary, and magnitudes far from the
// ends of the range, where the pairs' low parts would vanish.
__device__ __forceinline__ void two_sum(float a, float b, float& s, float& e) {
  s = __fadd_rn(a, b);
  const float t = __fsub_rn(s, a);
  e = __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t));
}
__device__ __forceinline__ void two_prod(float a, float b, float& p, float& e) {
  p = __fmul_rn(a, b);
  e = __fmaf_rn(a, b, -p);
}
template <int C>
__device__ __forceinline__ bool norm_pairs(const float (&x)[C], const float (&g)[C], float eps, float (&out)[C]) {
  float h = 0.0f, l = 0.0f;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    float p, e, s, f;
    two_prod(x[c], x[c], p, e);
    two_sum(h, p, s, f);
    l = __fadd_rn(l, __fadd_rn(e, f));
    h = s;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float ho = __shfl_xor_sync(FULL, h, o), lo = __shfl_xor_sync(FULL, l, o);
    float s, f;
    two_sum(h, ho, s, f);
    l = __fadd_rn(__fadd_rn(l, lo), f);
    h = s;
  }
  // mean (a power of two) plus eps, brought to hi + lo with |lo| <= ulp(hi) / 2
  float m, f, r;
  two_sum(h * (1.0f / (32 * C)), eps, m, f);
  f = __fadd_rn(f, l * (1.0f / (32 * C)));
  two_sum(m, f, h, l);
  // 1 / sqrt(h + l) = y + z: one Newton step from y, its residual 1 - (h + l) y^2 in pairs
  const float y = rsqrtf(h);
  float a, b, c0, d;
  two_prod(y, y, a, b);
  two_prod(h, a, c0, d);
  d = __fadd_rn(d, __fmaf_rn(h, b, __fmul_rn(l, a)));
  r = __fsub_rn(__fsub_rn(1.0f, c0), d);
  const float z = __fmul_rn(y, __fmaf_rn(__fmul_rn(0.375f, r), r, __fmul_rn(0.5f, r)));
  bool sure = h > 0x1p-60f && h < 0x1p60f;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    float p, e, q, w, t, u;
    two_prod(x[c], g[c], p, e);
    two_prod(p, y, q, w);
    w = __fadd_rn(w, __fmaf_rn(p, z, __fmul_rn(e, y)));
    two_sum(q, w, t, u);  // t = RN(q + w), u what that left
    // half the distance to t's neighbour below and above (they differ at a power of two)
    const float at = fabsf(t), up = __fmul_rn(0.5f, __fsub_rn(__uint_as_float(__float_as_uint(at) + 1), at)),
                dn = __fmul_rn(0.5f, __fsub_rn(at, __uint_as_float(__float_as_uint(at) - 1)));
    const float au = fabsf(u), near = __fmul_rn(at, 0x1p-40f);
    const bool fine = at > 0x1p-60f && at < 0x1p60f && fabsf(p) > 0x1p-60f && fabsf(__fsub_rn(au, up)) > near &&
                      fabsf(__fsub_rn(au, dn)) > near;
    sure = sure && (fine || x[c] == 0.0f);
    out[c] = x[c] == 0.0f ? p : t;  // a zero keeps its sign
  }
  return sure;
}

template <int TYPE, int D>
__global__ void __launch_bounds__(256) kv_append_kernel(const AppendArgs a) {
  constexpr int C = D / 32;
  asm volatile("griddepcontrol.launch_dependents;" :::);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const long w = (long)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (w >= a.heads) return;  // whole warps
  const int lane = threadIdx.x & 31, per = a.n_q + 2 * a.n_kv;
  const int t = (int)(w / per), h = (int)(w - (long)t * per);
  const bool is_q = h < a.n_q, is_v = h >= a.n_q + a.n_kv;
  const int hh = is_q ? h : is_v ? h - a.n_q - a.n_kv : h - a.n_q;
  const float* src = (is_q ? a.q : is_v ? a.v : a.k) + t * a.ld + (long)hh * D;
  // the row itself, beside the chain lens -> table (all in bounds whether or not
  // the row is left out)
  float x[C];
#pragma unroll
  for (int c = 0; c < C; ++c) x[c] = __ldcg(src + 32 * c + lane);
  const int b = t / a.R, r = t - b * a.R;
  const int len = __ldcg(a.lens + b);
  const int p = len - a.R + r;
  if (len <= 0 || p < 0 || (p >> a.page_log2) >= a.table_w) return;
  if (a.rot && p >= a.n_pos - a.p0) return;
  const int pid = __ldcg(a.table + (long)b * a.table_w + (p >> a.page_log2));
  if ((unsigned)pid >= (unsigned)a.n_pages) return;
  // (gains and tables too may be a launch before's: no loads by the read-only path)
  if (!is_v) {
    const float* gain = is_q ? a.q_gain : a.k_gain;
    if (gain) {
      float gv[C];
#pragma unroll
      for (int c = 0; c < C; ++c) gv[c] = __ldcg(gain + 32 * c + lane);
      float y[C];
      if (__all_sync(FULL, norm_pairs<C>(x, gv, a.eps, y))) {
#pragma unroll
        for (int c = 0; c < C; ++c) x[c] = y[c];
      } else {
        norm_f64<C>(x, gv, a.eps);
      }
    }
    if (a.rot) {
      const long at = (long)(a.p0 + p) * (a.rot >> 1);
      if (a.paired) {
#pragma unroll
        for (int c = 0; c < C; ++c) {
          if (32 * c >= a.rot) continue;
          const int i = (32 * c + lane) >> 1;
          const float cs = __ldcg(a.cosines + at + i), sn = __ldcg(a.sines + at + i);
          const float o = __shfl_xor_sync(FULL, x[c], 1);
          const float u = __fmul_rn(x[c], cs), z = __fmul_rn(o, sn);
          x[c] = (lane & 1) ? __fadd_rn(u, z) : __fsub_rn(u, z);
        }
      } else {
        const int hc = a.rot >> 6;  // registers between the values of a pair
#pragma unroll
        for (int c = 0; c < C / 2; ++c) {
          if (c >= hc) continue;
          const float cs = __ldcg(a.cosines + at + 32 * c + lane), sn = __ldcg(a.sines + at + 32 * c + lane);
          // partner register c + hc: hc is 1 (rot 64) or 2 (rot 128)
          const float y = C == 4 && hc == 2 ? x[(c + 2) % C] : x[(c + 1) % C];
          const float u = __fsub_rn(__fmul_rn(x[c], cs), __fmul_rn(y, sn));
          const float z = __fadd_rn(__fmul_rn(y, cs), __fmul_rn(x[c], sn));
          x[c] = u;
          if (C == 4 && hc == 2) x[(c + 2) % C] = z;
          else x[(c + 1) % C] = z;
        }
      }
    }
  }
  if (is_q) {
    float* dst = a.qr + ((long)t * a.n_q + hh) * D;
#pragma unroll
    for (int c = 0; c < C; ++c) dst[32 * c + lane] = x[c];
    return;
  }
  const long row = (((long)pid * a.n_kv + hh) << a.page_log2) + (p & ((1 << a.page_log2) - 1));
  if (is_v) store_head<TYPE, D>(a.cv, a.cvs, row, x, lane);
  else store_head<TYPE, D>(a.ck, a.cks, row, x, lane);
}

// rows x span floats at pitch ld from p, against n dense floats from q
bool rows_overlap(const float* p, long ld, int rows, long span, const float* q, long n) {
  const float* end = p + (rows - 1) * ld + span;
  return p < q + n && q < end;
}

template <int TYPE>
lk_status launch_append(const AppendArgs& a, int D, int pdl, cudaStream_t stream) {
  const dim3 grid((unsigned)((a.heads + 7) / 8)), block(256);
  static std::atomic<int> done[2][kMaxDevices];
  const auto f = D == 128 ? kv_append_kernel<TYPE, 128> : kv_append_kernel<TYPE, 64>;
  if (!lkattn::prepare_kernel(f, done[D == 128], 0)) return LK_ERR_CUDA;
  return lkattn::launch(f, grid, block, 0, pdl, stream, a) == cudaSuccess ? LK_OK : LK_ERR_CUDA;
}

}  // namespace

extern "C" lk_status lk_kv_append(const lk_kv_cache* cache, const float* q, const float* k, const float* v, long ld,
                                  int n_q, const int32_t* table, int table_w, const int32_t* lens, int B, int R,
                                  int p0, const float* cosines, const float* sines, int n_pos, int rot, int paired,
                                  const float* q_gain, const float* k_gain, float eps, float* qr,
                                  const lk_launch_cfg* cfg, cudaStream_t stream) {
  if (check_launch_cfg(cfg)) return LK_ERR_ARG;
  lk_status st = lkattn::check_cache(cache, n_q);
  if (st) return st;
  if ((st = lkattn::check_rows(cache, table, table_w, lens, B, R))) return st;
  const int D = cache->head_dim;
  if ((rot != 0 && rot != 64 && rot != 128) || rot > D || p0 < 0 || n_pos < 0) return LK_ERR_SHAPE;
  const long M = (long)B * R;
  if (M == 0) return LK_OK;
  if (!q || !k || !v || !qr || (rot && n_pos && (!cosines || !sines))) return LK_ERR_ARG;
  if (ld < (long)n_q * D || ld < (long)cache->n_kv * D) return LK_ERR_SHAPE;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(qr, 16) || ld % 4) return LK_ERR_ALIGN;
  if ((cosines && !aligned(cosines, 4)) || (sines && !aligned(sines, 4)) || (q_gain && !aligned(q_gain, 4)) ||
      (k_gain && !aligned(k_gain, 4)))
    return LK_ERR_ALIGN;
  const long nq = M * n_q * D;
  if (rows_overlap(q, ld, (int)M, (long)n_q * D, qr, nq) || rows_overlap(k, ld, (int)M, (long)cache->n_kv * D, qr, nq) ||
      rows_overlap(v, ld, (int)M, (long)cache->n_kv * D, qr, nq))
    return LK_ERR_ARG;
  AppendArgs a;
  a.q = q;
  a.k = k;
  a.v = v;
  a.ld = ld;
  a.n_q = n_q;
  a.n_kv = cache->n_kv;
  a.page_log2 = lkattn::log2_of(cache->page);
  a.n_pages = cache->n_pages;
  a.ck = cache->k;
  a.cv = cache->v;
  a.cks = (__half*)cache->ks;
  a.cvs = (__half*)cache->vs;
  a.table = table;
  a.table_w = table_w;
  a.lens = lens;
  a.R = R;
  a.p0 = p0;
  a.cosines = cosines;
  a.sines = sines;
  a.n_pos = n_pos;
  a.rot = rot;
  a.paired = paired;
  a.q_gain = q_gain;
  a.k_gain = k_gain;
  a.eps = eps;
  a.qr = qr;
  a.heads = M * (n_q + 2 * cache->n_kv);
  const int pdl = cfg_pdl(cfg);
  if (cache->type == LK_KV_F16) return launch_append<LK_KV_F16>(a, D, pdl, stream);
  if (cache->type == LK_KV_BF16) return launch_append<LK_KV_BF16>(a, D, pdl, stream);
  return launch_append<LK_KV_Q8>(a, D, pdl, stream);
}
