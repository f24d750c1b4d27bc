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

#include <cooperative_groups.h>

#include "lk_device.cuh"
#include "lk_sample.h"
#include "lk_spans.h"

using namespace lk;
using namespace lkh;
namespace cg = cooperative_groups;

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

__device__ __forceinline__ float value_of(u64 key) {
  const unsigned d = (unsigned)(key >> 32);
  return __uint_as_float((d & 0x80000000u) ? d : ~(d | 0x80000000u));
}

struct SampleArgs {
  const float* logits;
  int N;
  int part;  // tokens of a warp's part of a row, a multiple of 32
  const float* T;
  const int* top_k;
  const float* top_p;
  const float* min_p;
  const float* u;
  int* idx;
  float* prob;
};

constexpr int NW = 16;             // warps of a block
constexpr int THREADS = 32 * NW;
constexpr int MAX_C = 8;           // blocks of a row at most
constexpr int NB = 2048;           // bins of the order
constexpr int CAP = 4096;          // tokens near the borders that are sorted
constexpr float REACH = 41.0f;     // log2 of the largest weight over the smallest that is not 0
constexpr float SLACK = 1e-4f;     // of the bins' estimated sums

struct Shared {
  u64 table[256];
  unsigned cnt[NB], pos[NB];       // this block's tokens in each bin, and their places in it
  union {
    struct {
      unsigned cnt[NB], pos[NB];   // the row's
    } all;
    u64 sorted[CAP];
  };
  u64 list[CAP];                   // keys near the borders: this block's
  u64 drawn[MAX_C * NW];           // sums of the parts, of what is kept for the draw
  u64 first[MAX_C];                // of each block: its first key,
  float low[MAX_C];                // its lowest logit,
  unsigned n_list[MAX_C];          // its tokens in list,
  u64 kept[MAX_C], mid[MAX_C];     // its sums before and between the windows
  u64 sums[2][MAX_C];
  u64 warp[NW];
  float fwarp[NW];
  unsigned listed;
  int mark[4];                     // the bins of the borders
  float est[2];
  u64 last;
  u64 goal;
  int at;
};

__device__ __forceinline__ u64 warp_sum(u64 v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(FULL, v, o);
  return v;
}
// Sum over the block, in every thread.
__device__ u64 block_sum(u64 v, Shared& s) {
  v = warp_sum(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) s.warp[threadIdx.x >> 5] = v;
  __syncthreads();
  return warp_sum((threadIdx.x & 31) < NW ? s.warp[threadIdx.x & 31] : 0ull);
}
// Sum of the values of the threads before this one; `all` gets the block's.
__device__ u64 block_before(u64 v, u64& all, Shared& s) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  u64 inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const u64 y = __shfl_up_sync(FULL, inc, o);
    if (lane >= o) inc += y;
  }
  __syncthreads();
  if (lane == 31) s.warp[w] = inc;
  __syncthreads();
  const u64 tot = lane < NW ? s.warp[lane] : 0ull;
  all = warp_sum(tot);
  return warp_sum(lane < w ? tot : 0ull) + inc - v;
}
__device__ float block_before(float v, float& all, Shared& s) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  float inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const float y = __shfl_up_sync(FULL, inc, o);
    if (lane >= o) inc += y;
  }
  __syncthreads();
  if (lane == 31) s.fwarp[w] = inc;
  __syncthreads();
  float before = 0.f;
  all = 0.f;
  for (int i = 0; i < NW; ++i) {
    if (i < w) before += s.fwarp[i];
    all += s.fwarp[i];
  }
  return before + inc - v;
}

// Where a token lies in the order: 256 times its bin, plus its place there.
struct Bins {
  float m, c, scale;
  __device__ __forceinline__ float depth(float l) const { return __fmul_rn(__fsub_rn(m, l), c); }  // in log2
  // any monotone function of the logit serves; all of it is finite for depth < REACH
  __device__ __forceinline__ unsigned place(float depth) const {
    return min((unsigned)__float_as_int(__fadd_rn(__fmul_rn(depth, scale), 8388608.0f)) & 0x7FFFFFu, 256u * NB - 1u);
  }
};

// The tokens of this warp's part, eight loads in flight a lane: f(logit, index).
template <typename F>
__device__ __forceinline__ void each(const float* x, int lo, int hi, F f) {
  const int lane = threadIdx.x & 31;
  for (int i0 = lo + lane; i0 - lane < hi; i0 += 256) {
    float l[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) l[j] = i0 + 32 * j < hi ? __ldcg(x + i0 + 32 * j) : NAN;
#pragma unroll
    for (int j = 0; j < 8; ++j) f(clean(l[j]), i0 + 32 * j);
  }
}

__global__ void __launch_bounds__(THREADS) sample_kernel(const SampleArgs a) {
  extern __shared__ __align__(16) unsigned char smem[];
  Shared& s = *(Shared*)smem;
  cg::cluster_group cl = cg::this_cluster();
  const int C = (int)cl.num_blocks(), me = (int)cl.block_rank();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    s.listed = 0;
    asm volatile("griddepcontrol.launch_dependents;" :::);
  }
  for (int i = threadIdx.x; i < 256; i += THREADS) s.table[i] = kExp2.v[i];
  for (int i = threadIdx.x; i < NB; i += THREADS) s.cnt[i] = s.pos[i] = 0;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const long row = blockIdx.x / C;
  const int N = a.N;
  const float* x = a.logits + row * N;
  const int slot = me * NW + warp;
  const int lo = min(N, slot * a.part), hi = min(N, lo + a.part);

  // the first of the order, and the lowest logit
  {
    u64 first = ~0ull;
    float low = INFINITY;
    each(x, lo, hi, [&](float l, int i) {
      const u64 k = key_of(l, i);
      first = l > -INFINITY && k < first ? k : first;
      low = l > -INFINITY ? fminf(low, l) : low;
    });
    first = ~warp_max_u64(~first);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) low = fminf(low, __shfl_xor_sync(FULL, low, o));
    if (lane == 0) {
      s.warp[warp] = first;
      s.fwarp[warp] = low;
    }
    __syncthreads();
    if (warp == 0) {
      first = ~warp_max_u64(lane < NW ? ~s.warp[lane] : 0ull);
      low = lane < NW ? s.fwarp[lane] : INFINITY;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) low = fminf(low, __shfl_xor_sync(FULL, low, o));
      if (lane < C) {
        Shared* to = cl.map_shared_rank(&s, lane);
        to->first[me] = first;
        to->low[me] = low;
      }
    }
  }
  cl.sync();
  u64 first = ~0ull;
  float low = INFINITY;
  for (int c = 0; c < C; ++c) {
    first = s.first[c] < first ? s.first[c] : first;
    low = fminf(low, s.low[c]);
  }
  const float T = a.T ? __ldcg(a.T + row) : 1.0f;
  if (first == ~0ull || !(T > 0.0f)) {
    if (me == 0 && threadIdx.x == 0) {
      a.idx[row] = first == ~0ull ? -1 : (int)(first & 0xFFFFFFFFu);
      if (a.prob) a.prob[row] = first == ~0ull ? 0.0f : 1.0f;
    }
    return;
  }
  const float m = value_of(first);
  const Slope c = slope_of(T);
  const int tk = a.top_k ? __ldcg(a.top_k + row) : 0;
  const float tp = a.top_p ? __ldcg(a.top_p + row) : 1.0f;
  const float mp0 = a.min_p ? __ldcg(a.min_p + row) : 0.0f, mp = mp0 > 0.0f ? fminf(mp0, 1.0f) : 0.0f;
  const u64 least = mp > 0.0f ? (u64)ceil((double)mp * ONE_F) : 0ull;
  const bool by_k = tk > 0 && tk < N, by_p = tp < 1.0f;
  // what is kept is all keys up to `last`, with weights of `least` at least
  u64 last = ~0ull;
  bool summed = false;  // drawn[] has the parts' sums

  if (by_k || by_p) {
    // ---- the order in bins ----
    const float reach = fminf(REACH, __fmul_rn(__fsub_rn(m, low), c.hi));
    const Bins bins = {m, c.hi, fminf(256.0f * (NB - 1) / fmaxf(reach, 1e-30f), 1e30f)};
    each(x, lo, hi, [&](float l, int) {
      const float d = bins.depth(l);
      if (d < REACH) {
        const unsigned p = bins.place(d);
        atomicAdd(&s.cnt[p >> 8], 1u);
        atomicAdd(&s.pos[p >> 8], p & 255u);
      }
    });
    cl.sync();
    const int per = NB / C;
    for (int i = threadIdx.x; i < per; i += THREADS) {
      const int b = me * per + i;
      unsigned n = 0, p = 0;
      for (int q = 0; q < C; ++q) {
        const Shared* from = cl.map_shared_rank(&s, q);
        n += from->cnt[b];
        p += from->pos[b];
      }
      for (int q = 0; q < C; ++q) {
        Shared* to = cl.map_shared_rank(&s, q);
        to->all.cnt[b] = n;
        to->all.pos[b] = p;
      }
    }
    cl.sync();
    // ---- the windows: the bin of the top_k border, those of the top_p border ----
    // A bin's sum of weights is estimated from its tokens' mean place: within
    // (ln2 * width)^2 / 8 of it, width at most 41 / 2047, half a place's rounding and
    // the f32 sums: 1e-4 covers them with room.
    constexpr int PER = NB / THREADS;
    unsigned n[PER], nt = 0;
    float w[PER], wt = 0.f;
    const float step = reach / (NB - 1);
    for (int j = 0; j < PER; ++j) {
      const int b = threadIdx.x * PER + j;
      n[j] = s.all.cnt[b];
      w[j] = n[j] ? n[j] * exp2f(-step * (b + s.all.pos[b] / (256.0f * n[j]))) : 0.f;
      nt += n[j];
      wt += w[j];
    }
    float w_all;
    u64 n_all;
    u64 nb = block_before((u64)nt, n_all, s);
    float wb = block_before(wt, w_all, s);
    int* mark = s.mark;
    if (threadIdx.x == 0) {
      mark[0] = NB;      // bin of the top_k border, NB: past the last
      mark[1] = 0;       // tokens of it that stay
      mark[2] = NB;
      mark[3] = NB - 1;
      s.est[0] = w_all;
    }
    __syncthreads();
    if (by_k) {
      u64 nn = nb;
      float ww = wb;
      for (int j = 0; j < PER; ++j) {
        if (nn < (u64)tk && nn + n[j] >= (u64)tk) {
          mark[0] = threadIdx.x * PER + j;
          mark[1] = (int)((u64)tk - nn);
          // of its tokens the heaviest: no less than all at its far edge, no more than at its near one
          s.est[0] = ww;
          s.est[1] = (float)(tk - (int)nn) * exp2f(-step * (threadIdx.x * PER + j));
        }
        nn += n[j];
        ww += w[j];
      }
    }
    __syncthreads();
    const int bk = mark[0], nk = mark[1];
    if (by_p) {
      const float z_hi = (s.est[0] + (bk < NB ? s.est[1] : 0.f)) * (1.0f + SLACK);
      const float z_lo = (s.est[0] + (bk < NB ? s.est[1] * exp2f(-step) : 0.f)) * (1.0f - SLACK);
      float ww = wb;
      const float p = fmaxf(tp, 0.f);
      for (int j = 0; j < PER; ++j) {
        const int b = threadIdx.x * PER + j;
        const float upto = ww + w[j];
        // the border lies in no bin before the first that may reach it, in none
        // behind the first that must have reached it
        if (n[j] && upto * (1.0f + SLACK) >= p * z_lo) atomicMin(mark + 2, b);
        if (n[j] && upto * (1.0f - SLACK) >= p * z_hi) atomicMin(mark + 3, b);
        ww = upto;
      }
      __syncthreads();
    }
    const int p_hi = by_p ? min(mark[3], bk) : -1, p_lo = by_p ? min(mark[2], p_hi) : NB;
    const int safe = by_p ? min(p_lo, bk) : bk;  // bins before it stay whole
    __syncthreads();
    // ---- the sums beside the windows, the tokens in them ----
    u64 part = 0, kept = 0, mid = 0;
    each(x, lo, hi, [&](float l, int i) {
      const float d = bins.depth(l);
      const int b = d < REACH ? (int)(bins.place(d) >> 8) : NB;
      if (b > bk || b == NB) return;
      if (b < safe) {
        const u64 e = weight_of(l, m, c, s.table);
        kept += e;
        part += e >= least ? e : 0ull;
      } else if (b == bk || (b >= p_lo && b <= p_hi)) {
        const unsigned at = atomicAdd(&s.listed, 1u);
        if (at < CAP) s.list[at] = key_of(l, i);
      } else {
        mid += weight_of(l, m, c, s.table);
      }
    });
    part = warp_sum(part);
    if (lane == 0) cl.map_shared_rank(&s, 0)->drawn[slot] = part;
    kept = block_sum(kept, s);
    mid = block_sum(mid, s);
    if (threadIdx.x < C) {
      Shared* to = cl.map_shared_rank(&s, threadIdx.x);
      to->n_list[me] = s.listed;
      to->kept[me] = kept;
      to->mid[me] = mid;
    }
    cl.sync();
    unsigned listed = 0;
    for (int q = 0; q < C; ++q) listed += s.n_list[q];
    if (listed <= CAP) {
      summed = true;
      if (me == 0) {
        kept = mid = 0;
        unsigned done = 0;
        for (int q = 0; q < C; ++q) {
          kept += s.kept[q];
          mid += s.mid[q];
          const Shared* from = cl.map_shared_rank(&s, q);
          for (unsigned i = threadIdx.x; i < s.n_list[q]; i += THREADS) s.sorted[done + i] = from->list[i];
          done += s.n_list[q];
        }
        unsigned pad = 32;
        while (pad < listed) pad *= 2;
        for (unsigned i = listed + threadIdx.x; i < pad; i += THREADS) s.sorted[i] = ~0ull;
        __syncthreads();
        for (unsigned k = 2; k <= pad; k *= 2)
          for (unsigned j = k / 2; j > 0; j /= 2) {
            for (unsigned i = threadIdx.x; i < pad / 2; i += THREADS) {
              const unsigned p = 2 * i - (i & (j - 1)), q = p + j;
              const u64 y = s.sorted[p], z = s.sorted[q];
              if ((y > z) == !(p & k)) {
                s.sorted[p] = z;
                s.sorted[q] = y;
              }
            }
            __syncthreads();
          }
        // the border among them: of top_k the nk-th of its bin, of top_p the first whose sum reaches
        constexpr int EACH = CAP / THREADS;
        u64 e[EACH], sum = 0;
        unsigned before_k = 0;  // of the listed, those before the top_k bin
        for (int j = 0; j < EACH; ++j) {
          const unsigned i = threadIdx.x * EACH + j;
          e[j] = 0;
          if (i >= listed) continue;
          const float l = value_of(s.sorted[i]);
          e[j] = weight_of(l, m, c, s.table);
          before_k += (int)(bins.place(bins.depth(l)) >> 8) < bk;
        }
        const unsigned stay = by_k && bk < NB ? (unsigned)block_sum(before_k, s) + nk : listed;
        for (int j = 0; j < EACH; ++j) sum += threadIdx.x * EACH + j < stay ? e[j] : 0ull;
        u64 all;
        u64 run = block_before(sum, all, s);
        const u64 z = kept + mid + all;
        const double want = by_p ? ceil((double)tp * (double)z) : 0.0;
        const u64 goal = want >= 1.0 ? (u64)want : 1ull;
        if (threadIdx.x == 0) s.last = stay ? s.sorted[stay - 1] : 0ull;
        __syncthreads();
        if (by_p)
          for (int j = 0; j < EACH; ++j) {
            const unsigned i = threadIdx.x * EACH + j;
            if (i < stay && kept + run < goal && kept + run + e[j] >= goal) s.last = s.sorted[i];
            run += e[j];
          }
        __syncthreads();
        // all bins behind the top_k border's that the list does not show
        last = !by_p && !(by_k && bk < NB) ? ~0ull : s.last;
        for (int j = 0; j < EACH; ++j) {
          const unsigned i = threadIdx.x * EACH + j;
          if (i < listed && s.sorted[i] <= last && e[j] >= least)
            atomicAdd(&s.drawn[(unsigned)(s.sorted[i] & 0xFFFFFFFFu) / (unsigned)a.part], e[j]);
        }
        __syncthreads();
      }
    } else {
      // too many tokens near a border (equal ones, as a rule): by halving the keys
      int turn = 0;
      auto whole = [&](u64 v) {
        v = block_sum(v, s);
        if (threadIdx.x < C) cl.map_shared_rank(&s, threadIdx.x)->sums[turn][me] = v;
        cl.sync();
        u64 r = 0;
        for (int q = 0; q < C; ++q) r += s.sums[turn][q];
        turn ^= 1;
        return r;
      };
      auto upto = [&](u64 key, bool weigh) {
        u64 v = 0;
        each(x, lo, hi, [&](float l, int i) {
          if (l > -INFINITY && key_of(l, i) <= key) v += weigh ? weight_of(l, m, c, s.table) : 1ull;
        });
        return whole(v);
      };
      auto border = [&](bool weigh, u64 want, u64 top) {
        u64 bottom = first;
        while (bottom < top) {
          const u64 half = bottom + (top - bottom) / 2;
          if (upto(half, weigh) >= want) top = half;
          else bottom = half + 1;
        }
        return bottom;
      };
      const u64 end = key_of(low, (unsigned)N);
      last = end;
      if (by_k && upto(end, false) >= (u64)tk) last = border(false, tk, end);
      if (by_p) {
        const double want = ceil((double)tp * (double)upto(last, true));
        last = border(true, want >= 1.0 ? (u64)want : 1ull, last);
      }
    }
  }
  if (!summed) {
    u64 part = 0;
    each(x, lo, hi, [&](float l, int i) {
      const u64 e = key_of(l, i) <= last ? weight_of(l, m, c, s.table) : 0ull;
      part += e >= least ? e : 0ull;
    });
    part = warp_sum(part);
    if (lane == 0) cl.map_shared_rank(&s, 0)->drawn[slot] = part;
  }
  // (the last time that blocks look into one another)
  cl.sync();
  if (me != 0) return;

  // ---- the draw: the part in which the running sum passes the goal, then the token ----
  if (warp == 0) {
    constexpr int PER = MAX_C * NW / 32;
    u64 v[PER], sum = 0;
    for (int j = 0; j < PER; ++j) {
      const int i = lane * PER + j;
      v[j] = i < C * NW ? s.drawn[i] : 0ull;
      sum += v[j];
    }
    u64 inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const u64 y = __shfl_up_sync(FULL, inc, o);
      if (lane >= o) inc += y;
    }
    const u64 total = __shfl_sync(FULL, inc, 31);
    float u = __ldcg(a.u + row);
    u = u > 0.0f ? u : 0.0f;
    u64 goal = u < 1.0f ? (u64)((double)u * (double)total) : total;
    goal = goal < total ? goal : total - 1;
    u64 run = inc - sum;
    for (int j = 0; j < PER; ++j) {
      if (run <= goal && run + v[j] > goal) {
        s.at = lane * PER + j;
        s.goal = goal - run;
      }
      run += v[j];
    }
    if (lane == 0) s.kept[0] = total;
  }
  __syncthreads();
  const u64 goal = s.goal, total = s.kept[0];
  const int begin = s.at * a.part, end = min(N, begin + a.part);
  const int len = (end - begin + THREADS - 1) / THREADS;
  u64 sum = 0;
  auto weight_at = [&](int i, float& l) {
    l = clean(__ldcg(x + i));
    const u64 e = key_of(l, i) <= last ? weight_of(l, m, c, s.table) : 0ull;
    return e >= least ? e : 0ull;
  };
  const int b0 = begin + threadIdx.x * len, b1 = min(end, b0 + len);
  float l;
  for (int i = b0; i < b1; ++i) sum += weight_at(i, l);
  u64 all;
  u64 run = block_before(sum, all, s);
  if (run <= goal && run + sum > goal)
    for (int i = b0; i < b1; ++i) {
      const u64 e = weight_at(i, l);
      if (run + e > goal) {
        a.idx[row] = i;
        if (a.prob) {
          int n;
          const u64 p = weight_parts(l, m, c, s.table, n);
          a.prob[row] = (float)(scalbn((double)p, -n) / (double)total);
        }
        break;
      }
      run += e;
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
  const DeviceInfo* d = device_info(nullptr);
  int dev = 0;
  if (!d || cudaGetDevice(&dev) != cudaSuccess) return LK_ERR_CUDA;
  static std::atomic<int> done[kMaxDevices];
  if (!done[dev].load(std::memory_order_acquire)) {
    if (cudaFuncSetAttribute(sample_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(Shared)) !=
        cudaSuccess)
      return LK_ERR_CUDA;
    carveout_max_shared(sample_kernel);
    done[dev].store(1, std::memory_order_release);
  }
  // blocks of a row: as many as the SMs take at once, none with less than 2048 tokens
  int C = 1;
  while (C < MAX_C && M * C * 2 <= d->sm_count && N >= C * 4096) C *= 2;
  const int parts = C * NW;
  const SampleArgs a = {logits, N, ((N + parts - 1) / parts + 31) & ~31, temperature, top_k, top_p, min_p, u, idx, prob};
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3(M * C);
  lc.blockDim = dim3(THREADS);
  lc.dynamicSmemBytes = sizeof(Shared);
  lc.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = C;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = attr;
  lc.numAttrs = cfg_pdl(cfg) ? 2 : 1;
  return cudaLaunchKernelEx(&lc, sample_kernel, a) == cudaSuccess ? LK_OK : LK_ERR_CUDA;
}
