// Routing to experts (include/lk_moe.h): lk_moe_route.
//
// A warp works on a row, its lanes hold the experts lane + 32 v.  The k largest
// are taken one by one: each lane keeps its own largest, one warp maximum of
// the values' order-preserving bits and one minimum of the holders' numbers
// give the next, and its lane drops it.  What this costs is latency (a launch,
// one read, k + 1 rounds of two warp reductions); there are no bytes to speak of.
//
// Which experts are taken is decided in f32 where f32 can.  With u = 2^-24, of a softmax (e =
// exp(-x), x = max - l) each e is within e (x + 4) u <= 4 u (the argument's rounding, exp to two
// places), and a rounding of s takes u more: two scores are 10 u of the largest off each
// other.  The sum is off by (V + 4) u of itself for its additions, V in a lane and 5 between them,
// and by 8 u for its terms (the most that up to 1023 terms e (x + 4) beside a 1 come to), its
// reciprocal by u: all scores by the same factor, so a difference of two by (V + 13) u of
// the largest at most.  A sigmoid is within 2^-21.  So values further apart than (V + 24) u of
// the largest score (2^-20), and 2^-22 of themselves, for the rounding of s + bias, are in the
// right order; groups' sums of two twice that, of the largest of what they are sums of.  Where
// two neighbours of the order taken are nearer (one row in some hundreds), f64 decides, whose exp is slow on this GPU's narrow
// f64 pipe: for sigmoids of the experts in question alone, one a lane; with a
// softmax, whose sum takes all of them, or where it is about groups, of the whole row (some
// 8 us for 256 experts).  Without a bias the order is the logits' own, and exact.
#include <float.h>
#include <math.h>

#include "lk_device.cuh"
#include "lk_moe.h"
#include "lk_spans.h"

using namespace lk;
using namespace lkh;

namespace {

struct RouteArgs {
  const float* logits;
  const float* bias;
  int E, n_group, top_group, group_sum, k;
  int gs;          // experts of a group
  unsigned g_inv;  // ceil(2^20 / gs): i / gs = i * g_inv >> 20 for i < 1024
  int sigmoid, renorm;
  float scale;
  int* ids;
  float* weights;
};

// ---- the two precisions ------------------------------------------------------------

__device__ __forceinline__ unsigned ordered(float v) {
  const unsigned u = __float_as_uint(v == 0.0f ? 0.0f : v);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float unordered(unsigned u) {
  return __uint_as_float((u & 0x80000000u) ? (u & 0x7FFFFFFFu) : ~u);
}
__device__ __forceinline__ float warp_max(float v) { return unordered(__reduce_max_sync(FULL, ordered(v))); }
__device__ __forceinline__ double warp_max(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmax(v, __shfl_xor_sync(FULL, v, o));
  return v;
}
__device__ __forceinline__ float exp_of(float x) { return expf(x); }
__device__ __forceinline__ double exp_of(double x) { return exp(x); }

enum { SURE, ALL };  // what f32 leaves open: nothing, or the whole row

// One row in precision T: the chosen experts and their weights in lanes < k.
template <typename T, int V>
__device__ __forceinline__ int route_row(const RouteArgs& a, const float (&l)[V], const float (&b)[V], int lane,
                                          T* vals, int& id, float& weight) {
  constexpr bool F32 = sizeof(T) == 4;
  const T none = (T)-INFINITY;
  const bool by_logit = a.bias == nullptr;
  T p[V], c[V];
  T m = none, pmax = (T)1;
#pragma unroll
  for (int v = 0; v < V; ++v) m = l[v] > m ? (T)l[v] : m;
  m = warp_max(m);
  if (m == none) m = (T)0;  // no expert at all
  if (!a.sigmoid) {
    T sum = (T)0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      p[v] = l[v] > -INFINITY ? exp_of((T)l[v] - m) : (T)0;
      sum += p[v];
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(FULL, sum, o);
    pmax = sum > (T)0 ? (T)1 / sum : (T)1;
#pragma unroll
    for (int v = 0; v < V; ++v) p[v] *= pmax;
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) p[v] = l[v] > -INFINITY ? (T)1 / ((T)1 + exp_of(-(T)l[v])) : (T)0;
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const bool there = l[v] > -INFINITY && b[v] - b[v] == 0.0f;
    c[v] = !there ? none : by_logit ? (T)l[v] : p[v] + (T)b[v];
  }
  const T slack = F32 ? (a.sigmoid ? (T)0x1p-20f : (T)((V + 24) * 0x1p-24f) * pmax) : (T)0;
  const T part = F32 ? (T)0x1p-22f : (T)0;
  bool sure = true;

  if (a.n_group > 1) {
    const bool sums = a.group_sum == 2, of_scores = by_logit && sums;
    __syncwarp();
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int i = lane + 32 * v;
      if (i < a.E) vals[i] = of_scores && c[v] > none ? p[v] : c[v];
    }
    __syncwarp();
    T t1 = none, t2 = none;
    if (lane < a.n_group)
      for (int i = lane * a.gs; i < (lane + 1) * a.gs; ++i) {
        const T x = vals[i];
        t2 = x > t1 ? t1 : x > t2 ? x : t2;
        t1 = x > t1 ? x : t1;
      }
    const bool two = sums && t2 > none;
    const T val = two ? t1 + t2 : t1;
    int rank = 0;
    for (int g = 0; g < a.n_group; ++g) {
      const T w = __shfl_sync(FULL, val, g);
      rank += w > val || (w == val && g < lane);
    }
    const unsigned stay = __ballot_sync(FULL, lane < a.n_group && val > none && rank < a.top_group);
    if (F32 && !(by_logit && !sums)) {
      // the largest of what the sums are of: the two may cancel
      const float size = val > none ? fabsf((float)t1) + (two ? fabsf((float)t2) : 0.f) : 0.f;
      const float most = __uint_as_float(__reduce_max_sync(FULL, __float_as_uint(size)));
      for (int g = 0; g < a.n_group; ++g) {
        const T w = __shfl_sync(FULL, val, g);
        if (lane < a.n_group && val > none && w > none && (((stay >> g) ^ (stay >> lane)) & 1u))
          sure = sure && fabsf((float)(w - val)) > 2.0f * (float)slack + 2.0f * (float)part * most;
      }
      if (!__all_sync(FULL, sure)) return ALL;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const unsigned i = lane + 32 * v;
      if (!((stay >> ((i * a.g_inv) >> 20)) & 1u)) c[v] = none;
    }
  }

  T best = none, pb = (T)0, prev = none;
  float lb = 0.f, bb = 0.f, lmine = 0.f;
  T pmine = (T)0;
  int vb = 0;
  id = -1;
  auto own_best = [&] {
    best = none;
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (c[v] > best) {
        best = c[v];
        vb = v;
        pb = p[v];
        lb = l[v];
        bb = b[v];
      }
  };
  own_best();
  const int rounds = a.k + (F32 && !by_logit ? 1 : 0);  // one more: the gap behind the last
  float logit = 0.f, shift = 0.f;                       // of the lane's candidate
  int cand = -1;
  T last = none;  // the k-th value
  for (int j = 0; j < 33; ++j) {
    const T top = warp_max(best);
    if (top == none) break;
    if (j >= rounds) {
      // the order is open: all that may be among the k, in lanes of their own
      if (sure || last - top > slack + part * (T)fabsf((float)last)) break;
      if (j == 32) return ALL;
    }
    const unsigned i = __reduce_min_sync(FULL, best == top ? (unsigned)(lane + 32 * vb) : 0xFFFFFFFFu);
    const int owner = (int)(i & 31u);
    if (F32 && !by_logit && j > 0) sure = sure && prev - top > slack + part * (T)fabsf((float)prev);
    if (F32 && j == 32 && !sure) return ALL;  // (no lane for it)
    prev = top;
    if (j == a.k - 1) last = top;
    const T pt = __shfl_sync(FULL, pb, owner);
    const float lt = __shfl_sync(FULL, lb, owner), bt = __shfl_sync(FULL, bb, owner);
    if (lane == j) {
      cand = (int)i;
      logit = lt;
      shift = bt;
    }
    if (lane == j && j < a.k) {
      id = (int)i;
      pmine = pt;
      lmine = lt;
    }
    if (lane == owner) {
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (v == vb) c[v] = none;
      own_best();
    }
  }

  if (F32 && !sure) {
    if (!a.sigmoid) return ALL;
    // the candidates by their values in f64 (equal ones: the lower number)
    const double d = cand >= 0 ? 1.0 / (1.0 + exp(-(double)logit)) + (double)shift : -INFINITY;
    int rank = 0;
    for (int j = 0; j < 32; ++j) {
      const double o = __shfl_sync(FULL, d, j);
      const int n = __shfl_sync(FULL, cand, j);
      rank += o > d || (o == d && n >= 0 && n < cand);
    }
    // lane j takes the candidate of rank j
    int from = 0;
    for (int j = 0; j < 32; ++j) {
      const int r = __shfl_sync(FULL, rank, j), n = __shfl_sync(FULL, cand, j);
      if (n >= 0 && r == lane) from = j;
    }
    const float lt = __shfl_sync(FULL, logit, from);
    const int n = __shfl_sync(FULL, cand, from);
    id = id >= 0 ? n : -1;
    lmine = lt;
    pmine = (T)1 / ((T)1 + exp_of(-(T)lt));
  }

  T w = id >= 0 ? pmine : (T)0;
  bool low = F32 && id >= 0 && w < (T)0x1p-126f;
  if (a.renorm) {
    // from the chosen logits alone: the row's largest may be in no chosen group; below -40 a
    // sigmoid is exp(l) to 2^-57, and f64 may not hold the smaller ones (none from -708 on)
    const T lm = !F32 || !a.sigmoid ? warp_max(id >= 0 ? (T)lmine : none) : (T)0;
    if (!a.sigmoid || lm < (T)-40) w = id >= 0 && (!a.sigmoid || lm >= (T)-708) ? exp_of((T)lmine - lm) : (T)0;
    low = F32 && id >= 0 && w < (T)0x1p-126f;
    T sum = w;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(FULL, sum, o);
    w = sum > (T)0 ? w / sum : (T)0;
  }
  // Scores below f32's range whose weights need not be, for their sum or for the scale: f64 has them.
  // (exp(-88) is below 2^-126; masked experts that fill up a row are far below)
  if (F32 && __any_sync(FULL, low)) {
    const float most = warp_max(id >= 0 ? lmine : -INFINITY), from = a.sigmoid ? fminf(most, 0.f) : most;
    if (__any_sync(FULL, low && lmine - from > -88.0f - fmaxf(logf(fabsf(a.scale)), 0.f))) return ALL;
  }
  weight = (float)(w * (T)a.scale);
  return SURE;
}

template <int V>
__device__ __noinline__ void route_row_f64(const RouteArgs& a, const float (&l)[V], const float (&b)[V], int lane,
                                           double* vals, int& id, float& weight) {
  route_row<double, V>(a, l, b, lane, vals, id, weight);
}

template <int V>
__global__ void __launch_bounds__(32) route_kernel(const RouteArgs a) {
  __shared__ double vals[32 * V];
  const int lane = threadIdx.x;
  const long row = blockIdx.x;
  asm volatile("griddepcontrol.launch_dependents;" :::);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  float l[V], b[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int i = lane + 32 * v;
    float x = i < a.E ? __ldcg(a.logits + row * a.E + i) : -INFINITY;
    b[v] = a.bias && i < a.E ? __ldcg(a.bias + i) : 0.0f;
    if (!(x >= -INFINITY)) x = -INFINITY;  // NaN
    l[v] = fminf(x, FLT_MAX);
  }
  int id;
  float w;
  if (route_row<float, V>(a, l, b, lane, (float*)vals, id, w) != SURE) route_row_f64<V>(a, l, b, lane, vals, id, w);
  if (lane < a.k) {
    a.ids[row * a.k + lane] = id;
    a.weights[row * a.k + lane] = w;
  }
}

lk_status launch_route(void (*f)(const RouteArgs), int M, int pdl, cudaStream_t stream, const RouteArgs& a) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(M);
  cfg.blockDim = dim3(32);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, f, a) == cudaSuccess ? LK_OK : LK_ERR_CUDA;
}

}  // namespace

extern "C" lk_status lk_moe_route(const float* logits, const float* bias, int M, int E, lk_score score, int n_group,
                                  int top_group, int group_sum, int k, int renorm, float scale, int32_t* ids,
                                  float* weights, const lk_launch_cfg* cfg, cudaStream_t stream) {
  if ((score != LK_SCORE_SOFTMAX && score != LK_SCORE_SIGMOID) || check_launch_cfg(cfg)) return LK_ERR_ARG;
  if (!(scale - scale == 0.0f)) return LK_ERR_ARG;  // not finite
  if (M < 0 || M > LK_MAX_BATCH || E < 1 || E > LK_MOE_MAX_E || k < 1 || k > E || k > LK_MOE_MAX_K) return LK_ERR_SHAPE;
  if (n_group < 1 || n_group > LK_MOE_MAX_GROUPS || E % n_group || top_group < 1 || top_group > n_group ||
      group_sum < 1 || group_sum > 2)
    return LK_ERR_SHAPE;
  if (M == 0) return LK_OK;
  if (!logits || !ids || !weights) return LK_ERR_ARG;
  if (!aligned(logits, 4) || !aligned(bias, 4) || !aligned(ids, 4) || !aligned(weights, 4)) return LK_ERR_ALIGN;
  const size_t out = (size_t)M * k * 4;
  const Span spans[] = {{ids, out}, {weights, out}, {logits, (size_t)M * E * 4}, {bias, (size_t)E * 4}};
  if (spans_clash(spans, 2, 4)) return LK_ERR_ARG;
  RouteArgs a;
  a.logits = logits;
  a.bias = bias;
  a.E = E;
  a.n_group = n_group;
  a.top_group = top_group;
  a.group_sum = group_sum;
  a.k = k;
  a.gs = E / n_group;
  a.g_inv = ((1u << 20) + a.gs - 1) / a.gs;
  a.sigmoid = score == LK_SCORE_SIGMOID;
  a.renorm = renorm != 0;
  a.scale = scale;
  a.ids = ids;
  a.weights = weights;
  const int pdl = cfg_pdl(cfg);
  // values a lane holds: the smallest of these that fit, fewer steps a round
  return E <= 128   ? launch_route(route_kernel<4>, M, pdl, stream, a)
         : E <= 256 ? launch_route(route_kernel<8>, M, pdl, stream, a)
                    : launch_route(route_kernel<32>, M, pdl, stream, a);
}
