// The next token from the logits (include/lk_sample.h): lk_sample.
//
// Weights.  e = exp((l - max) / T) as a whole number of 2^-39: the argument
// (l - max) log2(e) / T as an unevaluated sum of two floats, its nearest
// multiple of 1/256 taken out (k / 256), 2^(frac(k / 256)) from a table of 256
// and the remaining factor, 1 + q with |q| < 2^-9.5, from a cubic in f32 (a
// table-driven exponential after P. T. P. Tang, ACM TOMS 15(2), 1989): relative
// error below 2^-32 where the weight is above 2^-8, else the last place.  Whole
// numbers add to the same sum in any order, so nothing here depends on how a
// row is split, and the largest weight is exactly 2^39.
//
// The order of tokens (the largest logit first, equal ones by index) is that of
// the 64-bit keys (complement of the logit's order-preserving bits, index);
// what top_k and top_p keep is all keys up to a border.
#include <float.h>
#include <math.h>

#include "lk_device.cuh"
#include "lk_sample.h"
#include "lk_spans.h"

using namespace lk;
using namespace lkh;

namespace {

typedef unsigned long long u64;

constexpr int ONE = 39;                         // a weight of 1 is 2^39
constexpr double ONE_F = (double)(1ull << ONE);

// ---- the weights -------------------------------------------------------------------

// 2^(j/256) 2^ONE, rounded: exp's series in f64 on the host
constexpr u64 exp2_entry(int j) {
  const double x = 0.69314718055994530942 * j / 256;
  double sum = 1, term = 1;
  for (int n = 1; n < 24; ++n) {
    term = term * x / n;
    sum += term;
  }
  return (u64)(sum * ONE_F + 0.5);
}
struct Exp2Table {
  u64 v[256];
  constexpr Exp2Table() : v() {
    for (int j = 0; j < 256; ++j) v[j] = exp2_entry(j);
  }
};
__device__ const Exp2Table kExp2 = Exp2Table();

// log2(e) / T as two floats
struct Slope {
  float hi, lo;
};
__device__ __forceinline__ Slope slope_of(float T) {
  const double c = fmin(1.4426950408889634074 / (double)T, 1e37);
  Slope s;
  s.hi = (float)c;
  s.lo = (float)(c - (double)s.hi);
  return s;
}

// e = (mant 2^-n) 2^-ONE, mant in [2^ONE, 2^(ONE+1)); n 63 for what is nothing
__device__ __forceinline__ u64 weight_parts(float l, float m, const Slope& c, const u64* table, int& n) {
  // l - m = d + r exactly (D. E. Knuth's two-sum)
  const float d = __fsub_rn(l, m), bb = __fsub_rn(d, l);
  const float r = __fadd_rn(__fsub_rn(l, __fsub_rn(d, bb)), __fsub_rn(-m, bb));
  const float t = __fmul_rn(d, c.hi);
  if (!(t >= -62.0f)) {
    n = 63;
    return 0;
  }
  const float te = __fmaf_rn(d, c.hi, -t) + __fmaf_rn(d, c.lo, __fmul_rn(r, c.hi));
  const float kf = rintf(__fmul_rn(t, 256.0f));
  const int k = (int)kf;
  const float f = __fadd_rn(__fmaf_rn(kf, -0.00390625f, t), te);  // |f| <= 1/512
  const float q = __fmul_rn(f, fmaf(f, fmaf(f, 0.055504109f, 0.24022651f), 0.69314718f));
  const u64 w = table[k & 255];
  n = -(k >> 8);
  return w + (long long)__float2int_rn(__fmul_rn((float)w, q));  // |w q| < 2^30.5
}
__device__ __forceinline__ u64 weight_of(float l, float m, const Slope& c, const u64* table) {
  int n;
  const u64 w = weight_parts(l, m, c, table, n);
  return n > ONE + 1 ? 0ull : n > 0 ? (w + (1ull << (n - 1))) >> n : w;
}

// ---- rows --------------------------------------------------------------------------

__device__ __forceinline__ float clean(float x) {
  if (!(x >= -INFINITY)) return -INFINITY;  // NaN
  return fminf(x, FLT_MAX);
}
__device__ __forceinline__ unsigned down_bits(float v) {  // the larger v, the smaller
  const unsigned u = __float_as_uint(v == 0.0f ? 0.0f : v);
  return (u & 0x80000000u) ? u : ~(u | 0x80000000u);
}
__device__ __forceinline__ u64 key_of(float l, unsigned i) { return ((u64)down_bits(l) << 32) | i; }

struct SampleArgs {
  const float* logits;
  int N;
  const float* T;
  const int* top_k;
  const float* top_p;
  const float* min_p;
  const float* u;
  int* idx;
  float* prob;
};

constexpr int THREADS = 1024;

__device__ __forceinline__ u64 warp_sum(u64 v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(FULL, v, o);
  return v;
}
// Sum over the block, in every thread.
__device__ u64 block_sum(u64 v, u64* sh) {
  v = warp_sum(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
  __syncthreads();
  return warp_sum(sh[threadIdx.x & 31]);
}
__device__ u64 block_min(u64 v, u64* sh) {
  v = ~warp_max_u64(~v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = v;
  __syncthreads();
  return ~warp_max_u64(~sh[threadIdx.x & 31]);
}

__global__ void __launch_bounds__(THREADS) sample_kernel(const SampleArgs a) {
  __shared__ u64 sh[32];
  __shared__ u64 table[256];
  asm volatile("griddepcontrol.launch_dependents;" :::);
  for (int i = threadIdx.x; i < 256; i += THREADS) table[i] = kExp2.v[i];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const long row = blockIdx.x;
  const float* x = a.logits + row * a.N;
  const int N = a.N;
  u64 first = ~0ull;
  for (int i = threadIdx.x; i < N; i += THREADS) {
    const u64 k = key_of(clean(__ldcg(x + i)), i);
    first = k < first ? k : first;
  }
  first = block_min(first, sh);
  const int imax = (int)(first & 0xFFFFFFFFu);
  const float m = clean(__ldcg(x + imax)), T = a.T ? __ldcg(a.T + row) : 1.0f;
  if (m == -INFINITY || !(T > 0.0f)) {
    if (threadIdx.x == 0) {
      a.idx[row] = m == -INFINITY ? -1 : imax;
      if (a.prob) a.prob[row] = m == -INFINITY ? 0.0f : 1.0f;
    }
    return;
  }
  const Slope c = slope_of(T);
  // the smallest border whose keys up to it count (weigh) at least `want`
  auto border = [&](bool weigh, u64 want, u64 hi) {
    u64 lo = first;
    while (lo < hi) {
      const u64 mid = lo + (hi - lo) / 2;
      u64 s = 0;
      for (int i = threadIdx.x; i < N; i += THREADS) {
        const float l = clean(__ldcg(x + i));
        if (key_of(l, i) <= mid) s += weigh ? weight_of(l, m, c, table) : 1;
      }
      s = block_sum(s, sh);
      if (s >= want) hi = mid;
      else lo = mid + 1;
    }
    return lo;
  };
  u64 last = ~0ull;
  const int tk = a.top_k ? __ldcg(a.top_k + row) : 0;
  if (tk > 0 && tk < N) last = border(false, tk, last);
  const float mp0 = a.min_p ? __ldcg(a.min_p + row) : 0.0f, mp = mp0 > 0.0f ? fminf(mp0, 1.0f) : 0.0f;
  auto sum_kept = [&](u64 least) {
    u64 s = 0;
    for (int i = threadIdx.x; i < N; i += THREADS) {
      const float l = clean(__ldcg(x + i));
      if (key_of(l, i) > last) continue;
      const u64 w = weight_of(l, m, c, table);
      if (w >= least) s += w;
    }
    return block_sum(s, sh);
  };
  const float tp = a.top_p ? __ldcg(a.top_p + row) : 1.0f;
  if (tp < 1.0f) {
    const double want = ceil((double)tp * (double)sum_kept(0));
    last = border(true, want >= 1.0 ? (u64)want : 1ull, last);
  }
  const u64 least = mp > 0.0f ? (u64)ceil((double)mp * ONE_F) : 0ull;
  const u64 total = sum_kept(least);
  float u = __ldcg(a.u + row);
  u = u > 0.0f ? u : 0.0f;
  u64 goal = u < 1.0f ? (u64)((double)u * (double)total) : total - 1;
  if (goal >= total) goal = total - 1;
  // the first index whose running sum exceeds the goal
  u64 before = 0;
  for (int i0 = 0; i0 < N; i0 += THREADS) {
    const int i = i0 + threadIdx.x;
    u64 w = 0;
    float l = 0.f;
    if (i < N) {
      l = clean(__ldcg(x + i));
      if (key_of(l, i) <= last) w = weight_of(l, m, c, table);
      if (w < least) w = 0;
    }
    const u64 all = block_sum(w, sh);
    if (before + all <= goal) {
      before += all;
      continue;
    }
    // inclusive sums over the block's threads
    u64 s = w;
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const u64 y = __shfl_up_sync(FULL, s, o);
      if (lane >= o) s += y;
    }
    __syncthreads();
    if (lane == 31) sh[threadIdx.x >> 5] = s;
    __syncthreads();
    for (int v = 0; v < (int)(threadIdx.x >> 5); ++v) s += sh[v];
    if (before + s > goal && before + s - w <= goal) {
      a.idx[row] = i;
      if (a.prob) {
        int n;
        const u64 p = weight_parts(l, m, c, table, n);
        a.prob[row] = (float)(scalbn((double)p, -n) / (double)total);
      }
    }
    break;
  }
}

}  // namespace

extern "C" lk_status lk_sample(const float* logits, int M, int N, const float* temperature, const int32_t* top_k,
                               const float* top_p, const float* min_p, const float* u, int32_t* idx, float* prob,
                               const lk_launch_cfg* cfg, cudaStream_t stream) {
  if (check_launch_cfg(cfg)) return LK_ERR_ARG;
  if (M < 0 || M > LK_MAX_BATCH || N < 1 || N > LK_SAMPLE_MAX_N) return LK_ERR_SHAPE;
  if (M == 0) return LK_OK;
  if (!logits || !u || !idx) return LK_ERR_ARG;
  const void* const all[] = {logits, temperature, top_k, top_p, min_p, u, idx, prob};
  for (const void* p : all)
    if (!aligned(p, 4)) return LK_ERR_ALIGN;
  const size_t r = (size_t)M * 4;
  const Span spans[] = {{idx, r},   {prob, r},  {logits, (size_t)M * N * 4}, {temperature, r},
                        {top_k, r}, {top_p, r}, {min_p, r},                  {u, r}};
  if (spans_clash(spans, 2, 8)) return LK_ERR_ARG;
  const SampleArgs a = {logits, N, temperature, top_k, top_p, min_p, u, idx, prob};
  launch_pdl(sample_kernel, dim3(M), dim3(THREADS), stream, cfg_pdl(cfg), a);
  return launch_status();
}
