// The next token from the logits (include/lk_sample.h): lk_sample.
//
// Weights.  e = exp((l - max) / T): the nearest multiple of 1/64 of l log2(e) / T
// is taken out of it (one fused multiply-add leaves the rest, below 1/128, to 2^-32),
// 2^(frac) comes from a table of 64, and the remaining factor, 1 + q with
// |q| < 2^-6.5, from a quartic in f32 (a table-driven exponential after P. T. P. Tang, ACM
// TOMS 15(2), 1989): relative error below 2^-29.  Each lane has a copy of the table in its
// own banks.  Weights below 2^-REACH of the largest count as nothing, N of them for N 2^-48.5 of
// it.  Sums are whole numbers of 2^-42 (all of a row's fit in 64 bits), and those of a warp's
// part, in which the token is found, of 2^-48, so that no weight that counts is rounded to 0;
// a lane's sum over its part of a row is kept as three f32 sums, of the weights'
// multiples of two grids that make them exact and of the rests (whole numbers of 64 bits
// cost three times the instructions), then rounded to a whole number: what is summed over
// lanes and blocks does not depend on their order.
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

constexpr int ONE = 42;                         // a weight of 1 is 2^42,
constexpr int FINE = 48;                        // within a part 2^48

// ---- the weights -------------------------------------------------------------------

constexpr int TAB = 64;                         // entries of the table
constexpr float REACH = 48.5f;                  // 2^-REACH of the largest and below is nothing

// 2^(j/TAB): as a float, and what it is more than that, relatively (exp's series in f64 on
// the host, of which an f32 rest keeps enough)
constexpr double exp2_of(int j) {
  const double x = 0.69314718055994530942 * j / TAB;
  double sum = 1, term = 1;
  for (int n = 1; n < 24; ++n) {
    term = term * x / n;
    sum += term;
  }
  return sum;
}
struct Exp2Table {
  float hi[TAB], lo[TAB];
  constexpr Exp2Table() : hi(), lo() {
    for (int j = 0; j < TAB; ++j) {
      hi[j] = (float)exp2_of(j);
      lo[j] = (float)(exp2_of(j) / (double)hi[j] - 1.0);
    }
  }
};
__device__ const Exp2Table kExp2 = Exp2Table();

// The weights of a row.
struct Weights {
  float m;              // the largest logit
  float hi, lo;         // log2(e) / T as two floats
  float base;           // taken off the logits first, where they are so large that
                        // it is needed: exactly, for all within reach of m
  float hi_tab;         // hi * TAB
  int k_m;              // m's multiple of 1 / TAB
  float f_m;            // and its rest
  const float2* tab;    // this lane's copy of the table, entries 32 apart

  __device__ __forceinline__ float split(float x, int& k) const {
    const float big = __fmaf_rn(x, hi_tab, 12582912.0f);  // 1.5 * 2^23: a whole number in the low bits
    k = __float_as_int(big) - 0x4B400000;
    const float kf = __fsub_rn(big, 12582912.0f);
    return __fmaf_rn(x, lo, __fmaf_rn(x, hi, __fmul_rn(kf, -1.0f / TAB)));
  }
  __device__ __forceinline__ Weights(float max, float T, const float2* table) : m(max) {
    // (in f32: f64 divisions by all of a block's threads took microseconds)
    constexpr float L_HI = 1.44269502f, L_LO = 1.92596300e-8f;  // log2(e)
    const float t = fmaxf(T, 1e-34f);
    hi = __fdiv_rn(L_HI, t);
    lo = hi > 0.0f ? __fdiv_rn(__fadd_rn(__fmaf_rn(-hi, t, L_HI), L_LO), t) : 0.0f;
    hi_tab = hi * TAB;
    base = fabsf(m) * hi > 8192.0f ? m : 0.0f;
    tab = table + (threadIdx.x & 31);
    f_m = split(__fsub_rn(m, base), k_m);
  }
  // how far below the largest, in log2
  __device__ __forceinline__ float depth(float l) const { return __fmul_rn(__fsub_rn(m, l), hi); }
  // e = big (1 + small) for a depth below REACH (else anything)
  __device__ __forceinline__ float parts(float l, float& small) const {
    int k;
    const float f = __fsub_rn(split(__fsub_rn(l, base), k), f_m);
    k -= k_m;
    const float2 t = tab[(k & (TAB - 1)) * 32];
    small = fmaf(f, fmaf(f, fmaf(f, fmaf(f, 0.0096181291f, 0.055504109f), 0.24022651f), 0.69314718f), t.y);
    return __int_as_float(__float_as_int(t.x) + (k >> 6) * (1 << 23));
  }
  // as a whole number of 2^-BITS, rounded to nearest
  template <int BITS>
  __device__ __forceinline__ u64 of(float l) const {
    float small;
    const float big = parts(l, small);
    // in two steps: the integer of big (exact or nearest), and the rest
    const float scaled = __fmul_rn(big, (float)(1ull << BITS)), rest = __fmul_rn(scaled, small);
    const long long whole = __float2ll_rn(scaled);
    const float left = __fadd_rn(__fsub_rn(scaled, __ll2float_rn(whole)), rest);
    return depth(l) < REACH ? (u64)(whole + __float2ll_rn(left)) : 0ull;
  }
  // e >= min_p, the same answer wherever it is asked
  static __device__ __forceinline__ bool enough(float big, float small, float min_p) {
    return __fmaf_rn(big, small, __fsub_rn(big, min_p)) >= 0.0f;
  }
  __device__ __forceinline__ bool enough(float l, float min_p) const {
    float small;
    const float big = parts(l, small);
    return depth(l) < REACH && enough(big, small, min_p);
  }
};
static_assert(TAB == 64, "parts() shifts by this");

// A weight as a multiple of GRID / 2^23 = 2^-15, one of FINE_GRID / 2^23 = 2^-31 (2^-16 at most),
// and what it is more than these: 2^-32 at most, and 2^-25 of the weight.
constexpr float GRID = 256.0f, FINE_GRID = 0x1p-8f;
struct Split {
  float multiple, fine, rest;
  __device__ __forceinline__ Split(float big, float small) {
    const float r = __fmul_rn(big, small), hi = __fadd_rn(big, r), lo = __fsub_rn(r, __fsub_rn(hi, big));
    multiple = __fsub_rn(__fadd_rn(hi, 1.5f * GRID), 1.5f * GRID);
    const float more = __fsub_rn(hi, multiple);
    fine = __fsub_rn(__fadd_rn(more, 1.5f * FINE_GRID), 1.5f * FINE_GRID);
    rest = __fadd_rn(__fsub_rn(more, fine), lo);
  }
};
// A lane's sum of up to GRID of them: of both multiples exactly, and the rests of 256 weights
// come to 2^-24 at most, so what f32 loses of these is below 2^-41 (one grid only lost
// 2^-26 where all weights were alike and below 2^-16).
struct Sum {
  float high = 0.f, middle = 0.f, low = 0.f;
  u64 all = 0;
  __device__ __forceinline__ void add(const Split& v) {
    high = __fadd_rn(high, v.multiple);
    middle = __fadd_rn(middle, v.fine);
    low = __fadd_rn(low, v.rest);
  }
  __device__ __forceinline__ void flush() {
    constexpr float one = (float)(1ull << ONE);
    all += (u64)(__float2ll_rn(__fmul_rn(high, one)) + __float2ll_rn(__fmul_rn(middle, one)) +
                 __float2ll_rn(__fmul_rn(low, one)));
    high = middle = low = 0.f;
  }
};

// floor (ceil) of x * total, x from 0 to 1 (below 2^-40: as 2^-40's multiples)
__device__ __forceinline__ u64 share_down(float x, u64 total) {
  return __umul64hi(__float2ull_rz(__fmul_rn(x, 0x1p40f)) << 24, total);
}
__device__ __forceinline__ u64 share_up(float x, u64 total) {
  const u64 f = __float2ull_rz(__fmul_rn(x, 0x1p40f)) << 24;
  return __umul64hi(f, total) + (f * total != 0);
}

// ---- rows --------------------------------------------------------------------------

// (the maximum with a NaN is the other)
__device__ __forceinline__ float clean(float x) { return fminf(fmaxf(x, -INFINITY), FLT_MAX); }
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
  int C;     // blocks of a row
  int part;  // tokens of a warp's part of a row, a multiple of 128
  int held;  // of these, in shared memory
  const float* T;
  const int* top_k;
  const float* top_p;
  const float* min_p;
  const float* u;
  int* idx;
  float* prob;
};

constexpr int CAP = 4096;          // tokens near the borders that are sorted
constexpr int HELD = 32768;        // tokens of a block in shared memory at most

__device__ __forceinline__ u64 warp_sum(u64 v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(FULL, v, o);
  return v;
}

// A row's blocks, up to MAX_C (8 or 16) of NW warps each.  Few tokens go with few warps: most of
// what a block runs through is run through by all of its warps, whatever they have to do.
// (Loops over 16 blocks cost rows of fewer 2 %, so those have kernels of their own.)
template <int NW, int MAX_C>
struct Rows {
static constexpr int THREADS = 32 * NW;
static constexpr int NB = 64 * NW;                  // bins of the order
static constexpr int PLACES = 32768 / NB;           // places in a bin
static constexpr int POS_BITS = NW == 32 ? 18 : NW == 16 ? 19 : 20;  // a bin's word: the sum of its tokens' places, above it
                                                    // their number, below 2^(32 - POS_BITS)
// Of the bins' estimated sums.  A bin's sum of weights is estimated from its tokens' mean
// place: within (ln2 * width)^2 / 8 of it (width REACH / (NB - 1) at most: 3.4e-5, 1.4e-4 or 5.4e-4),
// half a place's rounding (5.2e-4) and the f32 sums.
static constexpr float SLACK = NW == 8 ? 1.3e-3f : 8e-4f;

struct alignas(16) Shared {
  float2 table[TAB * 32];
  unsigned bin[NB];                // this block's tokens in each bin, and their places in it
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
  unsigned n_list[MAX_C];          // its tokens in list, and in bins,
  unsigned n_bin[MAX_C];
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

// (the tokens held lie behind it, read and written by 16 bytes)
static_assert(sizeof(Shared) % 16 == 0 && sizeof(Shared) + HELD * 4 <= 227 * 1024, "shared memory");

// Sum over the block, in every thread.
static __device__ u64 block_sum(u64 v, Shared& s) {
  v = warp_sum(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) s.warp[threadIdx.x >> 5] = v;
  __syncthreads();
  return warp_sum((threadIdx.x & 31) < NW ? s.warp[threadIdx.x & 31] : 0ull);
}
// Sum of the values of the threads before this one; `all` gets the block's.
static __device__ u64 block_before(u64 v, u64& all, Shared& s) {
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
static __device__ float block_before(float v, float& all, Shared& s) {
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
  const float tot = lane < NW ? s.fwarp[lane] : 0.f;
  float before = lane < w ? tot : 0.f;
  all = tot;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    before += __shfl_xor_sync(FULL, before, o);
    all += __shfl_xor_sync(FULL, all, o);
  }
  return before + inc - v;
}

// Sum of the values of the threads behind this one.
static __device__ float block_after(float v, Shared& s) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  float inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const float y = __shfl_down_sync(FULL, inc, o);
    if (lane + o < 32) inc += y;
  }
  __syncthreads();
  if (lane == 0) s.fwarp[w] = inc;
  __syncthreads();
  float after = lane > w && lane < NW ? s.fwarp[lane] : 0.f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) after += __shfl_xor_sync(FULL, after, o);
  return after + __shfl_down_sync(FULL, inc, 1) * (lane < 31);
}

// Where a token lies in the order: PLACES times its bin, plus its place there.
struct Bins {
  float scale;
  // any monotone function of the depth serves; it is finite below REACH
  __device__ __forceinline__ unsigned place(float depth) const {
    return min((unsigned)__float_as_int(__fadd_rn(__fmul_rn(depth, scale), 8388608.0f)) & 0x7FFFFFu, (unsigned)PLACES * NB - 1u);
  }
};

// A warp's part of a row: tokens [lo, hi), of which the first `held` are in its
// shared memory once they have been read.  Rows need not begin at 16 bytes: the
// part's first `skew` places (below 4) lie before it and are no tokens.
struct Part {
  const float* x;
  float* mem;
  int lo, hi, held;
  __device__ __forceinline__ float4 load(int i) const {
    float4 v;
    if (i >= 0 && i + 3 < hi) {
      v = __ldcg((const float4*)(x + i));
    } else {
      v.x = i >= 0 && i < hi ? __ldcg(x + i) : NAN;
      v.y = i + 1 >= 0 && i + 1 < hi ? __ldcg(x + i + 1) : NAN;
      v.z = i + 2 >= 0 && i + 2 < hi ? __ldcg(x + i + 2) : NAN;
      v.w = i + 3 < hi ? __ldcg(x + i + 3) : NAN;
    }
    return make_float4(clean(v.x), clean(v.y), clean(v.z), clean(v.w));
  }
  // f(logit, index) of every token, and of some places that are none with -inf:
  // from global memory, eight loads in flight a lane, to shared memory.
  template <typename F>
  __device__ __forceinline__ void first(F f) const {
    const int lane = threadIdx.x & 31;
    constexpr int U = 8;
    for (int i0 = lo + 4 * lane; i0 - 4 * lane < hi; i0 += 128 * U) {
      float4 v[U];
#pragma unroll
      for (int j = 0; j < U; ++j) v[j] = load(i0 + 128 * j);
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const int i = i0 + 128 * j;
        if (i - 4 * lane >= hi) break;  // (the whole warp)
        if (i - lo < held) *(float4*)(mem + (i - lo)) = v[j];
        f(v[j].x, i);
        f(v[j].y, i + 1);
        f(v[j].z, i + 2);
        f(v[j].w, i + 3);
      }
    }
  }
  // The same again, where the tokens are now: f(four logits, the first one's index).
  // The loop is rolled (f is some hundred instructions: fetching more code takes longer
  // than the work), with the next two loads in flight.
  template <typename F>
  __device__ __forceinline__ void again(F f) const {
    const int lane = threadIdx.x & 31;
    auto get = [&](int i) -> float4 {
      if (i - lo < held) return *(const float4*)(mem + (i - lo));
      return load(i);
    };
    int i = lo + 4 * lane;
    float4 v = get(i), next = get(i + 128);
#pragma unroll 1
    for (; i - 4 * lane < hi; i += 128) {
      const float4 later = get(i + 256);
      const float l[4] = {v.x, v.y, v.z, v.w};
      f(l, i);
      v = next;
      next = later;
    }
  }
};

static __device__ __forceinline__ void run(const SampleArgs& a, unsigned char* smem) {
  Shared& s = *(Shared*)smem;
  cg::cluster_group cl = cg::this_cluster();
  const int C = (int)cl.num_blocks(), me = (int)cl.block_rank();
  // all threads of the row's blocks
  auto meet = [&] {
    if (C == 1) __syncthreads();
    else cl.sync();
  };
  // A block's shared memory may be written by another once it has begun, which its arrival here
  // tells; the wait lies behind the row's read, which hides it (nothing is handed over: relaxed).
  if (C > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" :::);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    s.listed = 0;
    asm volatile("griddepcontrol.launch_dependents;" :::);
  }
  // (the table's entries are under way while the row is read)
  constexpr int ENTRIES = TAB / NW;  // of a warp
  float2 entry[ENTRIES];
#pragma unroll
  for (int j = 0; j < ENTRIES; ++j) entry[j] = make_float2(kExp2.hi[j * NW + warp], kExp2.lo[j * NW + warp]);
  for (int i = threadIdx.x; i < NB; i += THREADS) s.bin[i] = 0;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const long row = blockIdx.x / C;
  const int N = a.N;
  const float* x = a.logits + row * N;
  const int slot = me * NW + warp;
  // parts begin at 16 bytes: the first at up to three places before the row
  const int skew = (int)(((uintptr_t)x >> 2) & 3);
  Part mine;
  mine.x = x;
  mine.lo = min(N, slot * a.part - skew);
  mine.hi = min(N, (slot + 1) * a.part - skew);
  mine.held = a.held;
  mine.mem = (float*)(smem + sizeof(Shared)) + (size_t)warp * a.held;

  // the first of the order, and the lowest logit
  float top = -INFINITY;  // this lane's largest
  {
    u64 first = ~0ull;
    float low = INFINITY;
    int at = 0;
    mine.first([&](float l, int i) {
      if (l > top) {  // (indices ascend in a lane)
        top = l;
        at = i;
      }
      low = l > -INFINITY ? fminf(low, l) : low;
    });
    if (top > -INFINITY) first = key_of(top, at);
#pragma unroll
    for (int j = 0; j < ENTRIES; ++j) s.table[THREADS * j + threadIdx.x] = entry[j];
    first = ~warp_max_u64(~first);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) low = fminf(low, __shfl_xor_sync(FULL, low, o));
    if (lane == 0) {
      s.warp[warp] = first;
      s.fwarp[warp] = low;
    }
    __syncthreads();
    if (C > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
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
  meet();
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
  const Weights w = Weights(value_of(first), T, s.table);
  const int tk = a.top_k ? __ldcg(a.top_k + row) : 0;
  const float tp = a.top_p ? __ldcg(a.top_p + row) : 1.0f;
  const float mp0 = a.min_p ? __ldcg(a.min_p + row) : 0.0f, mp = mp0 > 0.0f ? fminf(mp0, 1.0f) : 0.0f;
  const bool by_k = tk > 0 && tk < N, by_p = tp < 1.0f;
  // what is kept is all keys up to `last`, with weights of mp at least
  u64 last = ~0ull;
  bool summed = false;  // drawn[] has the parts' sums

  // this lane's sum of the weights (number) of the keys up to one, of those of min_p at least
  auto sum_up_to = [&](u64 key, bool weigh, float min_p) {
    Sum sum;
    u64 number = 0;
    int turns = 0;
    mine.again([&](const float (&l)[4], int i) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float small;
        const float big = w.parts(l[q], small);
        const bool in = l[q] > -INFINITY && key_of(l[q], i + q) <= key;
        number += in;
        if (in && w.depth(l[q]) < REACH && Weights::enough(big, small, min_p)) sum.add(Split(big, small));
      }
      if (++turns == (int)GRID / 4) {
        turns = 0;
        sum.flush();
      }
    });
    sum.flush();
    return weigh ? sum.all : number;
  };
  // this lane's sum of all weights of min_p at least, where no border is (without its keys: 64 rows of
  // 151936 37.6 -> 34.6 us)
  auto sum_all = [&](float min_p) {
    Sum sum;
    int turns = 0;
    mine.again([&](const float (&l)[4], int) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float small;
        const float big = w.parts(l[q], small);
        if (w.depth(l[q]) < REACH && (min_p == 0.0f || Weights::enough(big, small, min_p))) sum.add(Split(big, small));
      }
      if (++turns == (int)GRID / 4) {
        turns = 0;
        sum.flush();
      }
    });
    sum.flush();
    return sum.all;
  };

  if (by_k || by_p) {
    // ---- the order in bins ----
    const float reach = fminf(REACH, w.depth(low));
    const Bins bins = {fminf((float)PLACES * (NB - 1) / fmaxf(reach, 1e-30f), 1e30f)};
    unsigned binned = 0;
    auto count = [&](float l) {
      const float d = w.depth(l);
      const unsigned p = bins.place(d);
      if (d < REACH) {
        atomicAdd(&s.bin[p / PLACES], (1u << POS_BITS) + p % PLACES);
        ++binned;
      }
    };
    // Few of many: the lanes' largest alone are counted.  The bin in which theirs
    // reach top_k is not before the true one, and with eight lanes to each there are
    // hardly more tokens up to it than top_k: all of them are listed.
    bool few = by_k && tk <= C * THREADS / 8 && tk <= CAP / 4;
    // the row's bins, in every block
    auto merge = [&] {
      if (!few) {
        binned = (unsigned)block_sum(binned, s);
        if (threadIdx.x < C) cl.map_shared_rank(&s, threadIdx.x)->n_bin[me] = binned;
      }
      meet();
      const int per = NB / C;
      for (int i = threadIdx.x; i < per; i += THREADS) {
        const int b = me * per + i;
        unsigned v[MAX_C], n = 0, p = 0;
#pragma unroll
        for (int q = 0; q < MAX_C; ++q) v[q] = q < C ? cl.map_shared_rank(&s, q)->bin[b] : 0u;
#pragma unroll
        for (int q = 0; q < MAX_C; ++q) {
          n += v[q] >> POS_BITS;
          p += v[q] & ((1u << POS_BITS) - 1u);
        }
#pragma unroll
        for (int q = 0; q < MAX_C; ++q)
          if (q < C) {
            Shared* to = cl.map_shared_rank(&s, q);
            to->all.cnt[b] = n;
            to->all.pos[b] = p;
          }
      }
      meet();
    };
    constexpr int PER = NB / THREADS;
    const int b0 = threadIdx.x * PER;
    int* mark = s.mark;
    unsigned n[PER];
    u64 n_all, n_before;
    // the bin in which the count reaches top_k, and how many of it stay
    auto find_k = [&] {
      unsigned nt = 0;
      for (int j = 0; j < PER; ++j) nt += n[j] = s.all.cnt[b0 + j];
      n_before = block_before((u64)nt, n_all, s);
      if (threadIdx.x == 0) {
        mark[0] = NB;  // past the last
        mark[1] = 0;
        mark[2] = NB;
        mark[3] = NB - 1;
      }
      __syncthreads();
      if (by_k) {
        u64 nn = n_before;
        for (int j = 0; j < PER; ++j) {
          if (nn < (u64)tk && nn + n[j] >= (u64)tk) {
            mark[0] = b0 + j;
            mark[1] = (int)((u64)tk - nn);
          }
          nn += n[j];
        }
      }
      __syncthreads();
    };
    // bins by their first places, as place() has them before it takes the whole number out
    auto from = [&](int b) { return 8388608.0f + (float)(PLACES * b); };
    int bk = NB, nk = 0, p_lo = NB, p_hi = -1, safe = 0;
    bool full = false, ends_before = false, unsure = false;
    if (few) {
      if (top > -INFINITY) count(top);
      merge();
      find_k();
      bk = mark[0];
      nk = tk;
      p_lo = 0;
      p_hi = bk;
      if (bk == NB) {  // too few lanes have any within reach
        few = false;
        for (int i = threadIdx.x; i < NB; i += THREADS) s.bin[i] = 0;
        meet();
      }
    }
    if (!few) {
      binned = 0;
      mine.again([&](const float (&l)[4], int) {
#pragma unroll
        for (int q = 0; q < 4; ++q) count(l[q]);
      });
      merge();
      find_k();
      bk = mark[0];
      nk = mark[1];
      p_lo = NB;
      p_hi = -1;
      // a bin of more tokens than its word counts loses some: the row is done by halving then
      unsigned expected = 0;
      for (int q = 0; q < C; ++q) expected += s.n_bin[q];
      full = n_all != expected;
      if (by_p) {
        // ---- the bins of the top_p border ----
        float v[PER], sum = 0.f;
        const float step = reach / (NB - 1);
        for (int j = 0; j < PER; ++j) {
          v[j] = n[j] ? n[j] * exp2f(-step * (b0 + j + s.all.pos[b0 + j] / ((float)PLACES * n[j]))) : 0.f;
          sum += v[j];
        }
        float all;
        const float before = block_before(sum, all, s);
        float after = block_after(sum, s);
        if (threadIdx.x == 0) {
          s.est[0] = all;
          s.est[1] = 0.f;
        }
        __syncthreads();
        if (bk >= b0 && bk < b0 + PER) {
          float x = before;
          for (int j = 0; j < bk - b0; ++j) x += v[j];
          s.est[0] = x;
          // of its tokens the heaviest: no less than all at its far edge, no more than at its near one
          s.est[1] = (float)nk * exp2f(-step * bk);
        }
        __syncthreads();
        const float z_hi = (s.est[0] + s.est[1]) * (1.0f + SLACK);
        const float z_lo = (s.est[0] + s.est[1] * exp2f(-step)) * (1.0f - SLACK);
        const float p = fmaxf(tp, 0.f), rest = 1.0f - p;
        // The border lies in no bin before the first that may reach it, in none behind
        // the first that must have.  With no top_k the sums from the end say it too, and
        // nearer where top_p is close to 1.
        float upto = before, left = after + sum;
        for (int j = 0; j < PER; ++j) {
          upto += v[j];
          left = j + 1 < PER ? left - v[j] : after;
          bool may = upto * (1.0f + SLACK) >= p * z_lo, must = upto * (1.0f - SLACK) >= p * z_hi;
          if (bk == NB) {
            // (a difference of f32 sums is off by 2^-23 of what is taken from)
            const float blur = j + 1 < PER ? 0x1p-22f * (after + sum) : 0.f;
            may = may && left * (1.0f - SLACK) - blur <= rest * z_hi;
            must = must || left * (1.0f + SLACK) + blur <= rest * z_lo;
          }
          if (n[j] && may) atomicMin(mark + 2, b0 + j);
          if (n[j] && must) atomicMin(mark + 3, b0 + j);
        }
        __syncthreads();
        p_hi = min(mark[3], bk);
        p_lo = min(mark[2], p_hi);
      }
      safe = by_p ? min(p_lo, bk) : bk;  // bins before it stay whole
      // What min_p keeps is a beginning of the order too.  Where it ends in bins that stay whole under
      // top_k and top_p, it is what is kept, and their borders need not be found; where it ends behind
      // these bins, they stay whole under it as well (a sum of its own for it took registers: 64 rows of
      // 151936 with top_p 82 us against 77).  2^-12: log2f's error and the depth's, many times.
      if (mp > 0.0f && !full) {
        const float d = -log2f(mp);
        ends_before = __fadd_rn(__fmul_rn(d + 0x1p-12f, bins.scale), 8388608.0f) < from(safe) - 1.0f;
        unsure = !ends_before && __fadd_rn(__fmul_rn(d - 0x1p-12f, bins.scale), 8388608.0f) < from(safe);
      }
    }
    __syncthreads();
    // ---- the sums beside the windows, the tokens in them ----
    if (!ends_before) {
      u64 kept = 0, mid = 0;
      if (few) {
        // (a loop of its own, so short that fetching its code does not count)
        const float t_k1 = 8388608.0f + (float)(PLACES * (bk + 1));
        mine.again([&](const float (&l)[4], int i) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const float d = w.depth(l[q]);
            if (d < REACH && __fadd_rn(__fmul_rn(d, bins.scale), 8388608.0f) < t_k1) {
              const unsigned n = atomicAdd(&s.listed, 1u);
              if (n < CAP) s.list[n] = key_of(l[q], i + q);
            }
          }
        });
      } else if (!full) {
        Sum sum_kept, sum_mid;
        const float t_safe = from(safe), t_lo = from(p_lo), t_hi = from(p_hi + 1), t_k = from(bk), t_k1 = from(bk + 1);
        int turns = 0;
        mine.again([&](const float (&l)[4], int i) {
          // (without branches: the four tokens' chains of dependent steps interleave)
          float at[4];
          bool near[4], some = false, sums = false;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const float d = w.depth(l[q]);
            at[q] = d < REACH ? __fadd_rn(__fmul_rn(d, bins.scale), 8388608.0f) : INFINITY;
            near[q] = (at[q] >= t_lo && at[q] < t_hi) || (at[q] >= t_k && at[q] < t_k1);
            some = some || near[q];
            sums = sums || (at[q] < t_k && !near[q]);
          }
          if (__any_sync(FULL, sums)) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              float small;
              const float big = w.parts(l[q], small);
              const Split e(big, small);
              if (at[q] < t_safe) sum_kept.add(e);
              else if (at[q] < t_k && !near[q]) sum_mid.add(e);
            }
            if (++turns == (int)GRID / 4) {
              turns = 0;
              sum_kept.flush();
              sum_mid.flush();
            }
          }
          if (some)
#pragma unroll
            for (int q = 0; q < 4; ++q)
              if (near[q]) {
                const unsigned n = atomicAdd(&s.listed, 1u);
                if (n < CAP) s.list[n] = key_of(l[q], i + q);
              }
        });
        sum_kept.flush();
        sum_mid.flush();
        kept = sum_kept.all;
        mid = sum_mid.all;
      }
      const u64 part = warp_sum(kept);
      if (lane == 0) cl.map_shared_rank(&s, 0)->drawn[slot] = part;
      kept = block_sum(kept, s);
      mid = block_sum(mid, s);
      if (threadIdx.x < C) {
        Shared* to = cl.map_shared_rank(&s, threadIdx.x);
        to->n_list[me] = s.listed;
        to->kept[me] = kept;
        to->mid[me] = mid;
      }
      meet();
      unsigned listed = 0;
      for (int q = 0; q < C; ++q) listed += s.n_list[q];
      if (listed <= CAP && !full) {
        summed = !unsure;
        if (me == 0) {
          kept = mid = 0;
          for (int q = 0; q < C; ++q) {
            kept += s.kept[q];
            mid += s.mid[q];
          }
          for (unsigned i = threadIdx.x; i < listed; i += THREADS) {
            unsigned j = i;
            int q = 0;
            while (j >= s.n_list[q]) j -= s.n_list[q++];
            s.sorted[i] = cl.map_shared_rank(&s, q)->list[j];
          }
          __syncthreads();
          if (listed <= THREADS) {
            // a key a thread; neighbours below 32 meet by shuffles
            const unsigned i = threadIdx.x;
            unsigned pad = 32;
            while (pad < listed) pad *= 2;
            u64 v = i < listed ? s.sorted[i] : ~0ull;
#pragma unroll 1
            for (unsigned k = 2; k <= pad; k *= 2)
#pragma unroll 1
              for (unsigned j = k / 2; j > 0; j /= 2) {
                u64 o;
                if (j >= 32) {
                  __syncthreads();
                  s.sorted[i] = v;
                  __syncthreads();
                  o = s.sorted[i ^ j];
                } else {
                  o = __shfl_xor_sync(FULL, v, j);
                }
                v = (((i & j) == 0) == ((i & k) == 0)) == (o < v) ? o : v;
              }
            __syncthreads();
            s.sorted[i] = v;
          } else {
            unsigned pad = THREADS;
            while (pad < listed) pad *= 2;
            for (unsigned i = listed + threadIdx.x; i < pad; i += THREADS) s.sorted[i] = ~0ull;
            __syncthreads();
#pragma unroll 1
            for (unsigned k = 2; k <= pad; k *= 2)
#pragma unroll 1
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
          }
          __syncthreads();
          // the border among them: of top_k the nk-th of its bin, of top_p the first whose sum reaches
          u64* weight = s.list;  // of the sorted keys (the block's own list is in sorted[] now)
          const bool k_there = by_k && bk < NB;
#pragma unroll 1
          for (unsigned i = threadIdx.x; i < listed; i += THREADS)
            weight[i] = w.of<ONE>(value_of(s.sorted[i]));
          __syncthreads();
          if (warp == 0) {
            unsigned stay = listed;
            if (k_there) {
              unsigned before = 0;  // of the keys, those before the top_k bin
              if (!few)
                for (unsigned i = lane; i < listed; i += 32)
                  before += (int)(bins.place(w.depth(value_of(s.sorted[i]))) / PLACES) < bk;
              stay = __reduce_add_sync(FULL, before) + nk;
            }
            u64 key = stay ? s.sorted[stay - 1] : 0ull;
            if (by_p) {
              u64 z = 0;
#pragma unroll 1
              for (unsigned i = lane; i < stay; i += 32) z += weight[i];
              z = warp_sum(z) + kept + mid;
              const u64 want = share_up(fmaxf(tp, 0.f), z), goal = want ? want : 1ull;
              u64 run = kept;
#pragma unroll 1
              for (unsigned i0 = 0; i0 < stay; i0 += 32) {
                u64 inc = i0 + lane < stay ? weight[i0 + lane] : 0ull;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                  const u64 y = __shfl_up_sync(FULL, inc, o);
                  if (lane >= o) inc += y;
                }
                const unsigned there = __ballot_sync(FULL, run + inc >= goal);
                if (there) {
                  const unsigned i = i0 + __ffs(there) - 1;
                  key = s.sorted[i < stay ? i : stay - 1];
                  break;
                }
                run += __shfl_sync(FULL, inc, 31);
              }
            }
            // all keys where no border is in the bins
            if (lane == 0) s.last = !by_p && !k_there ? ~0ull : key;
          }
          __syncthreads();
          last = s.last;
          if (unsure) {
            if (threadIdx.x < C) cl.map_shared_rank(&s, threadIdx.x)->last = last;
          } else {
#pragma unroll 1
            for (unsigned i = threadIdx.x; i < listed; i += THREADS)
              if (s.sorted[i] <= last && (mp == 0.0f || w.enough(value_of(s.sorted[i]), mp)))
                atomicAdd(&s.drawn[((unsigned)(s.sorted[i] & 0xFFFFFFFFu) + skew) / (unsigned)a.part], weight[i]);
          }
          __syncthreads();
        }
        if (unsure) {  // (the sums of all blocks' tokens up to the border, below)
          meet();
          last = s.last;
        }
      } else {
        // too many tokens near a border (equal ones, as a rule): by halving the keys
        int turn = 0;
        auto whole = [&](u64 v) {
          v = block_sum(v, s);
          if (threadIdx.x < C) cl.map_shared_rank(&s, threadIdx.x)->sums[turn][me] = v;
          meet();
          u64 r = 0;
          for (int q = 0; q < C; ++q) r += s.sums[turn][q];
          turn ^= 1;
          return r;
        };
        auto upto = [&](u64 key, bool weigh) {
          return whole(sum_up_to(key, weigh, 0.0f));
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
          const u64 want = share_up(fmaxf(tp, 0.f), upto(last, true));
          last = border(true, want ? want : 1ull, last);
        }
      }
    }
  }
  if (!summed) {
    u64 part = last == ~0ull ? sum_all(mp) : sum_up_to(last, true, mp);
    part = warp_sum(part);
    if (lane == 0) cl.map_shared_rank(&s, 0)->drawn[slot] = part;
  }
  // (the last time that blocks look into one another)
  meet();
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
    u64 goal = u < 1.0f ? share_down(u, total) : total;
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
  const int begin = max(0, s.at * a.part - skew), end = min(N, (s.at + 1) * a.part - skew);
  // (The part's sum was rounded lane by lane: should the goal lie past what its tokens come
  // to here, the second turn takes the last of them.  A part with a sum has tokens that count.)
  u64 run = 0, want = goal << (FINE - ONE);
#pragma unroll 1
  for (int turn = 0; turn < 2; ++turn) {
    run = 0;
#pragma unroll 1
    for (int i0 = begin; i0 < end && run <= want; i0 += THREADS) {
      const int i = i0 + threadIdx.x;
      const float l = i < end ? clean(__ldcg(x + i)) : -INFINITY;
      u64 e = i < end && key_of(l, i) <= last && (mp == 0.0f || w.enough(l, mp)) ? w.of<FINE>(l) : 0ull;
      u64 all;
      const u64 r = run + block_before(e, all, s);
      if (r <= want && r + e > want) {
        a.idx[row] = i;
        if (a.prob) {
          float small;
          const float big = w.parts(l, small);
          a.prob[row] = __fdiv_rn(__fmul_rn(__fmaf_rn(big, small, big), (float)(1ull << ONE)), __ull2float_rn(total));
        }
      }
      run += all;
    }
    if (run > want) break;
    want = run - 1;
  }
}

};

template <int NW, int MAX_C>
__global__ void __launch_bounds__(32 * NW) sample_kernel(const SampleArgs a) {
  extern __shared__ __align__(128) unsigned char smem[];
  Rows<NW, MAX_C>::run(a, smem);
}

constexpr int LARGE = 32768, SMALL = 6144;  // tokens of a block above which it has 32 (16) warps
constexpr int MOST = 1 << 20;               // tokens of a block: more would pass 64 bits in a part's sum
static_assert(((unsigned long long)MOST / 32 + 128) <= (~0ull >> FINE), "a part's sum");

template <int NW, int MAX_C>
lk_status launch_rows(SampleArgs a, int M, int dev, int pdl, cudaStream_t stream) {
  typedef Rows<NW, MAX_C> R;
  cudaLaunchConfig_t lc = {};
  lc.blockDim = dim3(R::THREADS);
  lc.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = attr;
  lc.numAttrs = pdl ? 2 : 1;
  static std::atomic<int> done[kMaxDevices];
  if (!done[dev].load(std::memory_order_acquire)) {
    if (cudaFuncSetAttribute(sample_kernel<NW, MAX_C>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)(sizeof(typename R::Shared) + HELD * 4)) != cudaSuccess ||
        (MAX_C > 8 &&
         cudaFuncSetAttribute(sample_kernel<NW, MAX_C>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess))
      return LK_ERR_CUDA;
    carveout_max_shared(sample_kernel<NW, MAX_C>);
    done[dev].store(1, std::memory_order_release);
  }
  const int parts = a.C * NW;
  a.part = ((a.N + 3 + parts - 1) / parts + 127) & ~127;
  a.held = a.part < HELD / NW ? a.part : HELD / NW;
  lc.gridDim = dim3(M * a.C);
  lc.dynamicSmemBytes = sizeof(typename R::Shared) + (size_t)NW * a.held * 4;
  attr[0].val.clusterDim.x = a.C;
  return cudaLaunchKernelEx(&lc, sample_kernel<NW, MAX_C>, a) == cudaSuccess ? LK_OK : LK_ERR_CUDA;
}

// Clusters of 2, 4, 8 and 16 blocks that the device takes at once, 8 bits each (0: an error).
int clusters_at_once(int dev) {
  static std::atomic<int> known[kMaxDevices];
  int fits = known[dev].load(std::memory_order_acquire);
  if (fits) return fits;
  typedef Rows<32, 16> R;
  const size_t most = sizeof(typename R::Shared) + HELD * 4;
  if (cudaFuncSetAttribute(sample_kernel<32, 16>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most) != cudaSuccess ||
      cudaFuncSetAttribute(sample_kernel<32, 16>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
    return 0;
  cudaLaunchConfig_t lc = {};
  lc.blockDim = dim3(R::THREADS);
  lc.dynamicSmemBytes = most;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  lc.attrs = attr;
  lc.numAttrs = 1;
  for (int i = 0; i < 4; ++i) {
    int n = 0;
    attr[0].val.clusterDim.x = 2u << i;
    lc.gridDim = dim3(2u << i);
    if (cudaOccupancyMaxActiveClusters(&n, sample_kernel<32, 16>, &lc) != cudaSuccess) return 0;
    fits |= (n < 127 ? n : 127) << (8 * i);
  }
  known[dev].store(fits, std::memory_order_release);
  return fits;
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
  int dev = 0;
  if (!device_info(&dev)) return LK_ERR_CUDA;
  const int fits = clusters_at_once(dev);
  if (!fits) return LK_ERR_CUDA;
  // blocks of a row: as many as are on the SMs at once with all rows', none with less than 2048 tokens
  // (one row of 151936 in 16 blocks, not 8: top_p 31 -> 24 us, top_k 50 and top_p 17 -> 15)
  int C = 1;
  for (int i = 0; i < 4 && ((M <= ((fits >> (8 * i)) & 127) && N >= C * 4096) || N > C * MOST); ++i) C *= 2;
  const SampleArgs a = {logits, N, C, 0, 0, temperature, top_k, top_p, min_p, u, idx, prob};
  const int pdl = cfg_pdl(cfg), tokens = N / C;
  if (C == 16)
    return tokens > LARGE   ? launch_rows<32, 16>(a, M, dev, pdl, stream)
           : tokens > SMALL ? launch_rows<16, 16>(a, M, dev, pdl, stream)
                            : launch_rows<8, 16>(a, M, dev, pdl, stream);
  return tokens > LARGE   ? launch_rows<32, 8>(a, M, dev, pdl, stream)
         : tokens > SMALL ? launch_rows<16, 8>(a, M, dev, pdl, stream)
                          : launch_rows<8, 8>(a, M, dev, pdl, stream);
}
