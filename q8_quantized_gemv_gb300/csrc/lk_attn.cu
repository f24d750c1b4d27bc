// Attention over the paged cache (include/lk_attn.h): lk_attn,
// lk_attn_shared.
//
// Work.  An item is one key/value head of one sequence with up to 8 of the
// query rows that read it (row i of a head's R * G: token i / G, query head
// i % G); a shared prefix is one more sequence with the rows of all others.
// Its keys come in units of 32.  All units of all items, in a fixed order, are
// dealt to the blocks in equal contiguous shares, whatever the lengths are;
// a block's part of an item (a segment) leaves a partial result (running
// maximum, sum, weighted values) in the workspace, in slot block + item,
// which no other segment has; a second launch joins the partials of a row.
//
// Mathematics.  Scores and weighted sums run on m16n8k16 MMAs whose 16 rows
// are 8 query rows twice: rows 0..7 the high and rows 8..15 the low 16-bit
// term of the f32 operand, so that a lane holds both products of its row and
// their sum costs one addition; keys and values enter as stored (Q8: as their
// integer levels, exact in f16, the scales applied in f32 to the scores and
// folded into the weights).  f16 operands are shifted by powers of two so
// that the low terms stay normal: queries to a row maximum of 2^10, weights by
// 2^14 (Q8: after dividing out the unit's largest scale's power of two).  A
// bf16 query has three terms: with two, scores of a few hundred would lose
// the weights' fifth digit.  Each unit's weighted values are summed in a fresh
// accumulator and added in f32, so the MMA's own accumulation never runs over
// more than 32 keys.
//
// Data.  Every warp streams its own units through its own stages of shared
// memory with 16-byte asynchronous copies.  A lane of the 16-bit kernels
// copies exactly the pieces that it will use as MMA operands (the order of the
// inner index of a product is free, so a lane's 8 consecutive values serve two
// k-steps), so stages need no barrier and reads no shuffle; the Q8 kernels
// read 4- and 8-byte pieces, staged with their 16-byte pieces permuted against
// bank conflicts.
#include <cuda_bf16.h>

#include "lk_attn.cuh"

using namespace lk;
using namespace lkh;

namespace lkattn {

constexpr int UNIT = 32;          // keys of a unit
constexpr int TR = 8;             // query rows of an item
constexpr int kMaxWorkers = 512;  // blocks of a launch, at most
constexpr int kMaxSeq = LK_MAX_BATCH + 1;

struct AttnArgs {
  const float* q;
  int n_q, n_kv, G;
  const void* k;
  const void* v;
  const __half* ks;
  const __half* vs;
  int page_log2, n_pages;
  const int* table;
  int table_w;
  const int* lens;
  int B, R;
  const int* ptable;  // prefix: page list, length, tokens it has room for
  int plen, pcap;
  int shared;
  float qscale;  // scale * log2(e)
  float* ml;     // partials: [slot][TR][2] maximum and sum,
  float* o;      //           [slot][TR][D] weighted values
  int W;         // blocks
};

// The deal of the units: sequence s has un[s] units per item, items before it
// item0(s), units before it cum[s]; cum[nseq] is their total.
struct Deal {
  long cum[kMaxSeq + 1];
  int un[kMaxSeq];
  int n[kMaxSeq];
};

__device__ __forceinline__ int rows_of(const AttnArgs& a, int s) { return (s == a.B ? a.B * a.R : a.R) * a.G; }
__device__ __forceinline__ int tiles_of(const AttnArgs& a, int s) { return (rows_of(a, s) + TR - 1) / TR; }
__device__ __forceinline__ int item0(const AttnArgs& a, int s) { return s * a.n_kv * tiles_of(a, 0); }

// Blocks that have a share: none is empty, so an item's segments are in
// consecutive blocks.
__device__ __forceinline__ long shares(const AttnArgs& a, long T) { return T < a.W ? T : a.W; }

// By the block's first warp; the caller synchronizes.
__device__ __forceinline__ void make_deal(const AttnArgs& a, Deal& d) {
  if (threadIdx.x >= 32) return;
  const int lane = threadIdx.x, nseq = a.B + a.shared;
  const int cap = a.table_w << a.page_log2;
  long run = 0;
  for (int s0 = 0; s0 < nseq; s0 += 32) {
    const int s = s0 + lane;
    int n = 0;
    long u = 0;
    if (s < nseq) {
      n = s == a.B ? min(a.plen, a.pcap) : min(max(__ldcg(a.lens + s), 0), cap);
      d.n[s] = n;
      d.un[s] = (n + UNIT - 1) / UNIT;
      u = (long)d.un[s] * a.n_kv * tiles_of(a, s);
    }
    long sum = u;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long up = __shfl_up_sync(FULL, sum, o);
      if (lane >= o) sum += up;
    }
    if (s < nseq) d.cum[s] = run + sum - u;
    run += __shfl_sync(FULL, sum, 31);
  }
  if (lane == 0) d.cum[nseq] = run;
}

// ---- MMA and copies -----------------------------------------------------------------
template <int TYPE>
__device__ __forceinline__ void mma16(float (&c)[4], unsigned a0, unsigned a1, unsigned a2, unsigned a3, unsigned b0,
                                      unsigned b1) {
  if constexpr (TYPE == LK_KV_BF16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// (x, y) rounded to the type, packed, and what the rounding left of them
template <int TYPE>
__device__ __forceinline__ unsigned split2(float& x, float& y) {
  if constexpr (TYPE == LK_KV_BF16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    x -= __low2float(h);
    y -= __high2float(h);
    return *(const unsigned*)&h;
  } else {
    const __half2 h = __floats2half2_rn(x, y);
    x -= __low2float(h);
    y -= __high2float(h);
    return *(const unsigned*)&h;
  }
}

__device__ __forceinline__ unsigned prmt(unsigned a, unsigned b, unsigned s) { return __byte_perm(a, b, s); }

// 16 bytes global -> shared; with bytes 0 nothing is read and zeros are written
__device__ __forceinline__ void cp16(unsigned dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ uint4 lds128(unsigned a) {
  uint4 r;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(a));
  return r;
}
__device__ __forceinline__ uint2 lds64(unsigned a) {
  uint2 r;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(r.x), "=r"(r.y) : "r"(a));
  return r;
}
__device__ __forceinline__ unsigned lds32(unsigned a) {
  unsigned r;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(r) : "r"(a));
  return r;
}

// Bytes c, c+1 (selector) of u = levels ^ 0x80 as a pair of f16 levels: 1024 + u is
// exact in the low mantissa bits of 0x64xx, less 1152.
__device__ __forceinline__ unsigned level_pair(unsigned u, unsigned sel) {
  const unsigned b = prmt(u, 0x64646464u, sel);
  const __half2 h = __hsub2(*(const __half2*)&b, __half2half2(__ushort_as_half(0x6480)));
  return *(const unsigned*)&h;
}

template <int TYPE, int D>
struct Cfg {
  static constexpr int EB = TYPE == LK_KV_Q8 ? 1 : 2;              // bytes of a stored value
  static constexpr int KV = UNIT * D * EB;                         // bytes of a unit's keys
  static constexpr int SC = TYPE == LK_KV_Q8 ? UNIT * D / 16 : 0;  // bytes of their scales
  static constexpr int STAGE = 2 * (KV + SC);
  static constexpr int NW = TYPE != LK_KV_Q8 && D == 128 ? 7 : 8;  // warps
  static constexpr int ST = TYPE != LK_KV_Q8 && D == 128 ? 2 : 3;  // stages a warp
  static constexpr int RING = NW * ST * STAGE;
  static_assert(STAGE * ST >= TR * (D + 4) * 4, "a warp's partial fits in its stages");
  static_assert(RING + 2048 <= 232448, "shared memory of a block");
};

template <int TYPE, int D>
__global__ void __launch_bounds__(32 * Cfg<TYPE, D>::NW, 1) attn_kernel(const AttnArgs a) {
  typedef Cfg<TYPE, D> C;
  constexpr bool Q8 = TYPE == LK_KV_Q8;
  constexpr int KS = D / 16;                       // k-steps of a score
  constexpr int QT = TYPE == LK_KV_BF16 ? 3 : 2;   // terms of a query
  constexpr int NT = D / 8;                        // n-tiles of the output
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ Deal deal;
  __shared__ float wml[C::NW][TR][2];
  asm volatile("griddepcontrol.launch_dependents;" :::);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  make_deal(a, deal);
  __syncthreads();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int nseq = a.B + a.shared;
  const long T = deal.cum[nseq], W = shares(a, T);
  if (blockIdx.x >= W) return;
  long u0 = T * blockIdx.x / W;
  const long u1 = T * (blockIdx.x + 1) / W;
  const unsigned ring = (unsigned)__cvta_generic_to_shared(smem) + warp * C::ST * C::STAGE;
  int s = 0;
  while (u0 < u1) {
    while (deal.cum[s + 1] <= u0) ++s;
    const int un = deal.un[s], n = deal.n[s];
    const long rel = u0 - deal.cum[s];
    const int li = (int)(rel / un), ub = (int)(rel - (long)li * un);
    const int ue = (int)min((long)un, ub + (u1 - u0));
    u0 += ue - ub;
    const int tiles = tiles_of(a, s), kvh = li / tiles, tile = li - kvh * tiles;
    const int slot = (int)blockIdx.x + item0(a, s) + li;
    const bool pre = s == a.B;
    const int nrows = min(TR, rows_of(a, s) - tile * TR);
    const int* table = pre ? a.ptable : a.table + (long)s * a.table_w;

    // the lane's query row (the last row again where there are fewer)
    const int ri = tile * TR + min(g, nrows - 1);
    const int tok = ri / a.G;  // row of the batch (prefix) or of the sequence
    const int row = pre ? tok : s * a.R + tok;
    int vis = n;  // keys that the row sees
    if (!pre) vis = min(n, max(0, __ldcg(a.lens + s) - a.R + 1 + tok));
    unsigned qa[KS][4], qc[QT == 3 ? KS : 1][2];
    float rs = 1.0f;
    {
      const float* q = a.q + ((long)row * a.n_q + kvh * a.G + (ri - tok * a.G)) * D + t * 8;
      float x[D / 4];
      float amax = 0.0f;
#pragma unroll
      for (int j = 0; j < D / 32; ++j) {
        const float4 f0 = __ldcg((const float4*)(q + 32 * j)), f1 = __ldcg((const float4*)(q + 32 * j + 4));
        x[8 * j + 0] = f0.x, x[8 * j + 1] = f0.y, x[8 * j + 2] = f0.z, x[8 * j + 3] = f0.w;
        x[8 * j + 4] = f1.x, x[8 * j + 5] = f1.y, x[8 * j + 6] = f1.z, x[8 * j + 7] = f1.w;
      }
#pragma unroll
      for (int i = 0; i < D / 4; ++i) {
        x[i] *= a.qscale;
        amax = fmaxf(amax, fabsf(x[i]));
      }
      if constexpr (TYPE != LK_KV_BF16) {
        amax = fmaxf(amax, __shfl_xor_sync(FULL, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(FULL, amax, 2));
        const int e = min(max((int)(__float_as_uint(amax) >> 23), 27), 227) - 127;  // amax in [2^e, 2^(e+1))
        rs = __uint_as_float((unsigned)(127 + e - 10) << 23);
        const float up = __uint_as_float((unsigned)(127 - e + 10) << 23);
#pragma unroll
        for (int i = 0; i < D / 4; ++i) x[i] *= up;
      }
      // k-step k: registers 4 k .. 4 k + 3 are the lane's four inner indices
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        qa[k][0] = split2<TYPE>(x[4 * k], x[4 * k + 1]);
        qa[k][2] = split2<TYPE>(x[4 * k + 2], x[4 * k + 3]);
        qa[k][1] = split2<TYPE>(x[4 * k], x[4 * k + 1]);
        qa[k][3] = split2<TYPE>(x[4 * k + 2], x[4 * k + 3]);
        if constexpr (QT == 3) {
          qc[k][0] = split2<TYPE>(x[4 * k], x[4 * k + 1]);
          qc[k][1] = split2<TYPE>(x[4 * k + 2], x[4 * k + 3]);
        }
      }
    }

    // pages of the unit's two halves (-1: none)
    auto pages = [&](int u, int (&pg)[2]) {
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const int key = u * UNIT + 16 * hf;
        pg[hf] = -1;
        if (u < ue && key < n) {
          const int p = __ldg(table + (key >> a.page_log2));
          if ((unsigned)p < (unsigned)a.n_pages) pg[hf] = p;
        }
      }
    };
    // start the copies of unit u into a stage; one commit group
    auto issue = [&](int u, const int (&pg)[2], int stage) {
      const unsigned st = ring + stage * C::STAGE;
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const int key0 = u * UNIT + 16 * hf;
        const int left = pg[hf] < 0 ? 0 : min(16, n - key0);  // tokens there are
        const long r0 =
            (((long)max(pg[hf], 0) * a.n_kv + kvh) << a.page_log2) + (key0 & ((1 << a.page_log2) - 1));
        const char* k = (const char*)a.k + r0 * D * C::EB;
        const char* v = (const char*)a.v + r0 * D * C::EB;
        if constexpr (!Q8) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int kk = 8 * i + g;
#pragma unroll
            for (int j = 0; j < D / 32; ++j)
              cp16(st + (((2 * hf + i) * (D / 32) + j) * 32 + lane) * 16, k + kk * (D * 2) + j * 64 + t * 16,
                   kk < left ? 16 : 0);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int kk = 2 * t + (e & 1) + 8 * (e >> 1);
#pragma unroll
            for (int h = 0; h < D / 64; ++h)
              cp16(st + C::KV + (((4 * hf + e) * (D / 64) + h) * 32 + lane) * 16, v + kk * (D * 2) + h * 128 + g * 16,
                   kk < left ? 16 : 0);
          }
        } else {
          constexpr int PP = D / 16;  // 16-byte pieces of a token
#pragma unroll
          for (int i = 0; i < 16 * PP / 32; ++i) {
            const int c = i * 32 + lane, kk = c / PP, pc = c % PP;
            const int fk = PP == 8 ? 2 * (kk & 3) : kk & 2, fv = PP == 8 ? kk & 6 : kk & 2;
            const int ok = kk < left ? 16 : 0;
            cp16(st + (16 * hf + kk) * D + ((pc ^ fk) * 16), k + c * 16, ok);
            cp16(st + C::KV + (16 * hf + kk) * D + ((pc ^ fv) * 16), v + c * 16, ok);
          }
          // scales: D bytes of each half's keys and as many of its values,
          // 16 / (D / 16) tokens to a piece
          constexpr int SP = D / 16;
          if (lane < 2 * SP) {
            const int pc = lane % SP;
            const char* sc = (const char*)(lane < SP ? a.ks : a.vs) + r0 * (D / 16);
            cp16(st + 2 * C::KV + (lane < SP ? 0 : C::SC) + hf * D + pc * 16, sc + pc * 16,
                 pc * 16 < left * (D / 16) ? 16 : 0);
          }
        }
      }
      cp_commit();
    };

    float O[NT][2], m = -INFINITY, l = 0.0f, dvm = 0.0f, dsc = 1.0f;
#pragma unroll
    for (int i = 0; i < NT; ++i) O[i][0] = O[i][1] = 0.0f;
    int pgq[C::ST][2], pgn[2];
    const int uw = ub + warp;
#pragma unroll
    for (int i = 0; i < C::ST; ++i) {
      pages(uw + i * C::NW, pgq[i]);
    }
#pragma unroll
    for (int i = 0; i < C::ST; ++i) {
      if (uw + i * C::NW < ue) issue(uw + i * C::NW, pgq[i], i);
      else cp_commit();
    }
    pages(uw + C::ST * C::NW, pgn);
    int stage = 0;
    for (int u = uw; u < ue; u += C::NW) {
      cp_wait<C::ST - 1>();
      if constexpr (Q8) __syncwarp();
      const unsigned st = ring + stage * C::STAGE;
      // ---- scores: lane (g, t) has row g with keys 8 i + 2 t, + 1
      float sc[4][2];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (!Q8) {
          float c[4] = {0.f, 0.f, 0.f, 0.f}, c3[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int j = 0; j < D / 32; ++j) {
            const uint4 w = lds128(st + ((i * (D / 32) + j) * 32 + lane) * 16);
            mma16<TYPE>(c, qa[2 * j][0], qa[2 * j][1], qa[2 * j][2], qa[2 * j][3], w.x, w.y);
            mma16<TYPE>(c, qa[2 * j + 1][0], qa[2 * j + 1][1], qa[2 * j + 1][2], qa[2 * j + 1][3], w.z, w.w);
            if constexpr (QT == 3) {
              mma16<TYPE>(c3, qc[2 * j][0], 0u, qc[2 * j][1], 0u, w.x, w.y);
              mma16<TYPE>(c3, qc[2 * j + 1][0], 0u, qc[2 * j + 1][1], 0u, w.z, w.w);
            }
          }
          sc[i][0] = (c[0] + (c[2] + c3[0])) * rs;
          sc[i][1] = (c[1] + (c[3] + c3[1])) * rs;
        } else {
          const int key = 8 * i + g, fk = D == 128 ? 2 * (key & 3) : key & 2;
          // scales of keys 8 i + 2 t, + 1
          __half2 d0[D / 64], d1[D / 64];
          if constexpr (D == 128) {
            const uint4 w = lds128(st + 2 * C::KV + (8 * i + 2 * t) * 8);
            d0[0] = *(const __half2*)&w.x, d0[1] = *(const __half2*)&w.y;
            d1[0] = *(const __half2*)&w.z, d1[1] = *(const __half2*)&w.w;
          } else {
            const uint2 w = lds64(st + 2 * C::KV + (8 * i + 2 * t) * 4);
            d0[0] = *(const __half2*)&w.x, d1[0] = *(const __half2*)&w.y;
          }
          float s0 = 0.f, s1 = 0.f;
#pragma unroll
          for (int b = 0; b < D / 32; ++b) {
            uint2 w = lds64(st + key * D + (((2 * b + (t >> 1)) ^ fk) * 16) + (t & 1) * 8);
            w.x ^= 0x80808080u, w.y ^= 0x80808080u;
            float c[4] = {0.f, 0.f, 0.f, 0.f};
            mma16<TYPE>(c, qa[2 * b][0], qa[2 * b][1], qa[2 * b][2], qa[2 * b][3], level_pair(w.x, 0x4140),
                        level_pair(w.x, 0x4342));
            mma16<TYPE>(c, qa[2 * b + 1][0], qa[2 * b + 1][1], qa[2 * b + 1][2], qa[2 * b + 1][3],
                        level_pair(w.y, 0x4140), level_pair(w.y, 0x4342));
            const float e0 = b & 1 ? __high2float(d0[b >> 1]) : __low2float(d0[b >> 1]);
            const float e1 = b & 1 ? __high2float(d1[b >> 1]) : __low2float(d1[b >> 1]);
            s0 = fmaf(e0, c[0] + c[2], s0);
            s1 = fmaf(e1, c[1] + c[3], s1);
          }
          sc[i][0] = s0 * rs;
          sc[i][1] = s1 * rs;
        }
      }
      // ---- what the row does not see
      const int pg0 = pgq[0][0], pg1 = pgq[0][1];
      const bool whole = (u + 1) * UNIT <= n && pg0 >= 0 && pg1 >= 0;
      if (!__all_sync(FULL, whole && (u + 1) * UNIT <= vis)) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int x = 0; x < 2; ++x)
            if (u * UNIT + 8 * i + 2 * t + x >= vis || (i < 2 ? pg0 : pg1) < 0) sc[i][x] = -INFINITY;
      }
      // ---- running maximum, weights
      float mt = fmaxf(fmaxf(fmaxf(sc[0][0], sc[0][1]), fmaxf(sc[1][0], sc[1][1])),
                       fmaxf(fmaxf(sc[2][0], sc[2][1]), fmaxf(sc[3][0], sc[3][1])));
      mt = fmaxf(mt, __shfl_xor_sync(FULL, mt, 1));
      mt = fmaxf(mt, __shfl_xor_sync(FULL, mt, 2));
      const float mn = fmaxf(m, mt);
      const float ref = mn == -INFINITY ? 0.0f : mn;
      float al = ex2(m - ref);  // 0 from an empty start
      m = mn;
      constexpr float UP = TYPE == LK_KV_BF16 ? 0.0f : Q8 ? 13.0f : 14.0f;
      float p[4][2];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        p[i][0] = ex2(sc[i][0] - (ref - UP));
        p[i][1] = ex2(sc[i][1] - (ref - UP));
      }
      l = l * al + (((p[0][0] + p[0][1]) + (p[1][0] + p[1][1])) + ((p[2][0] + p[2][1]) + (p[3][0] + p[3][1])));
      // ---- weighted values
      if constexpr (Q8) {
        // the largest value scale so far sets the power of two taken out
        constexpr int HW = D / 64;  // words of a token's scales
        unsigned mx = 0;
#pragma unroll
        for (int i = 0; i < HW; ++i) {
          const int w = i * 32 + lane;
          unsigned x = lds32(st + 2 * C::KV + C::SC + w * 4) & 0x7fff7fffu;
          if (u * UNIT + w / HW >= n) x = 0;
          mx = max(mx, max(x & 0xffffu, x >> 16));
        }
        mx = __reduce_max_sync(FULL, mx);
        const float dm = __half2float(__ushort_as_half((unsigned short)mx));
        if (dm > dvm) {  // warp-uniform
          dvm = dm;
          const float ns = __uint_as_float((254u - (__float_as_uint(dm) >> 23)) << 23);
          al *= ns / dsc;  // powers of two; O is 0 before the first
          dsc = ns;
        }
      }
      if (__any_sync(FULL, al != 1.0f)) {
#pragma unroll
        for (int i = 0; i < NT; ++i) O[i][0] *= al, O[i][1] *= al;
      }
      if constexpr (!Q8) {
        unsigned ph[2][4];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          ph[k][0] = split2<TYPE>(p[2 * k][0], p[2 * k][1]);
          ph[k][2] = split2<TYPE>(p[2 * k + 1][0], p[2 * k + 1][1]);
          ph[k][1] = split2<TYPE>(p[2 * k][0], p[2 * k][1]);
          ph[k][3] = split2<TYPE>(p[2 * k + 1][0], p[2 * k + 1][1]);
        }
#pragma unroll
        for (int h = 0; h < D / 64; ++h) {
          unsigned w[8][4];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const uint4 x = lds128(st + C::KV + ((e * (D / 64) + h) * 32 + lane) * 16);
            w[e][0] = x.x, w[e][1] = x.y, w[e][2] = x.z, w[e][3] = x.w;
          }
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const unsigned sel = j & 1 ? 0x7632 : 0x5410;
            float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int k = 0; k < 2; ++k)
              mma16<TYPE>(c, ph[k][0], ph[k][1], ph[k][2], ph[k][3], prmt(w[4 * k][j >> 1], w[4 * k + 1][j >> 1], sel),
                          prmt(w[4 * k + 2][j >> 1], w[4 * k + 3][j >> 1], sel));
            O[8 * h + j][0] += c[0] + c[2];
            O[8 * h + j][1] += c[1] + c[3];
          }
        }
      } else {
        // value scales of keys 8 i + 2 t, + 1, times dsc; 0 for absent tokens
        // (their scales may be anything)
        __half2 d0[4][D / 64], d1[4][D / 64];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if constexpr (D == 128) {
            const uint4 w = lds128(st + 2 * C::KV + C::SC + (8 * i + 2 * t) * 8);
            d0[i][0] = *(const __half2*)&w.x, d0[i][1] = *(const __half2*)&w.y;
            d1[i][0] = *(const __half2*)&w.z, d1[i][1] = *(const __half2*)&w.w;
          } else {
            const uint2 w = lds64(st + 2 * C::KV + C::SC + (8 * i + 2 * t) * 4);
            d0[i][0] = *(const __half2*)&w.x, d1[i][0] = *(const __half2*)&w.y;
          }
          const int key = u * UNIT + 8 * i + 2 * t;
          if (!whole) {
#pragma unroll
            for (int x = 0; x < D / 64; ++x) {
              if (key >= n) d0[i][x] = __half2half2(__ushort_as_half(0));
              if (key + 1 >= n) d1[i][x] = __half2half2(__ushort_as_half(0));
            }
          }
        }
#pragma unroll
        for (int b = 0; b < D / 32; ++b) {
          unsigned ph[2][4];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            float y[4];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float e0 = b & 1 ? __high2float(d0[2 * k + i][b >> 1]) : __low2float(d0[2 * k + i][b >> 1]);
              const float e1 = b & 1 ? __high2float(d1[2 * k + i][b >> 1]) : __low2float(d1[2 * k + i][b >> 1]);
              y[2 * i] = p[2 * k + i][0] * (e0 * dsc);
              y[2 * i + 1] = p[2 * k + i][1] * (e1 * dsc);
            }
            ph[k][0] = split2<TYPE>(y[0], y[1]);
            ph[k][2] = split2<TYPE>(y[2], y[3]);
            ph[k][1] = split2<TYPE>(y[0], y[1]);
            ph[k][3] = split2<TYPE>(y[2], y[3]);
          }
          unsigned w[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int key = 16 * (e >> 2) + 2 * t + (e & 1) + 8 * ((e >> 1) & 1);
            const int fv = D == 128 ? key & 6 : key & 2;
            w[e] = lds32(st + C::KV + key * D + (((2 * b + (g >> 2)) ^ fv) * 16) + (g & 3) * 4) ^ 0x80808080u;
          }
          unsigned z[2][2][2];  // [k-step][half][values 0,1 / 2,3 of the two tokens]
#pragma unroll
          for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              z[k][x][0] = prmt(w[4 * k + 2 * x], w[4 * k + 2 * x + 1], 0x5140);
              z[k][x][1] = prmt(w[4 * k + 2 * x], w[4 * k + 2 * x + 1], 0x7362);
            }
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const unsigned sel = j & 1 ? 0x4342 : 0x4140;
            float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int k = 0; k < 2; ++k)
              mma16<TYPE>(c, ph[k][0], ph[k][1], ph[k][2], ph[k][3], level_pair(z[k][0][j >> 1], sel),
                          level_pair(z[k][1][j >> 1], sel));
            O[4 * b + j][0] += c[0] + c[2];
            O[4 * b + j][1] += c[1] + c[3];
          }
        }
        __syncwarp();  // every lane is done with the stage
      }
      // ---- the stage's next unit
      const int nu = u + C::ST * C::NW;
#pragma unroll
      for (int i = 0; i + 1 < C::ST; ++i) pgq[i][0] = pgq[i + 1][0], pgq[i][1] = pgq[i + 1][1];
      pgq[C::ST - 1][0] = pgn[0], pgq[C::ST - 1][1] = pgn[1];
      if (nu < ue) issue(nu, pgn, stage);
      else cp_commit();
      pages(nu + C::NW, pgn);
      stage = stage + 1 == C::ST ? 0 : stage + 1;
    }
    cp_wait<0>();
    __syncwarp();

    // ---- the warps' partials of the segment, joined in warp order
    if constexpr (Q8) {
      const float back = 1.0f / dsc;
#pragma unroll
      for (int i = 0; i < NT; ++i) O[i][0] *= back, O[i][1] *= back;
    }
    l += __shfl_xor_sync(FULL, l, 1);
    l += __shfl_xor_sync(FULL, l, 2);
    float* mine = (float*)(smem + (size_t)warp * C::ST * C::STAGE);  // [TR][D + 4]
    if (g < nrows) {
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int d = Q8 ? (i >> 2) * 32 + (2 * t + x) * 4 + (i & 3) : (i >> 3) * 64 + (2 * t + x) * 8 + (i & 7);
          mine[g * (D + 4) + d] = O[i][x];
        }
      if (t == 0) wml[warp][g][0] = m, wml[warp][g][1] = l;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < nrows * D; i += 32 * C::NW) {
      const int r = i / D, d = i - r * D;
      float M = wml[0][r][0];
#pragma unroll
      for (int w = 1; w < C::NW; ++w) M = fmaxf(M, wml[w][r][0]);
      const float ref = M == -INFINITY ? 0.0f : M;
      float acc = 0.0f, ls = 0.0f;
#pragma unroll
      for (int w = 0; w < C::NW; ++w) {
        const float f = ex2(wml[w][r][0] - ref);
        const float ov = *(const float*)(smem + (size_t)w * C::ST * C::STAGE + (size_t)(r * (D + 4) + d) * 4);
        acc = fmaf(f, ov, acc);
        ls = fmaf(f, wml[w][r][1], ls);
      }
      __stcg(a.o + ((long)slot * TR + r) * D + d, acc);
      if (d == 0) {
        __stcg(a.ml + ((long)slot * TR + r) * 2, M);
        __stcg(a.ml + ((long)slot * TR + r) * 2 + 1, ls);
      }
    }
    __syncthreads();
  }
}

// ---- the join: one warp per row and query head ---------------------------------------
struct JoinArgs {
  AttnArgs a;
  float* out;
  int8_t* hq;
  int8_t* hl;
  float* hs;
};

template <int Q, int D>
__global__ void __launch_bounds__(128) attn_join_kernel(const JoinArgs j) {
  const AttnArgs& a = j.a;
  __shared__ Deal deal;
  asm volatile("griddepcontrol.launch_dependents;" :::);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  make_deal(a, deal);
  __syncthreads();
  const int lane = threadIdx.x & 31;
  const long w = (long)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (w >= (long)a.B * a.R * a.n_q) return;
  const int row = (int)(w / a.n_q), h = (int)(w - (long)row * a.n_q), kvh = h / a.G, hg = h - kvh * a.G;
  const int b = row / a.R, r = row - b * a.R;
  const long T = deal.cum[a.B + a.shared], W = shares(a, T);
  // the slots of the row's own item, then of its prefix item
  int first[2] = {0, 0}, count[2] = {0, 0}, rt[2] = {0, 0};
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const int s = x == 0 ? b : a.B;
    if (x == 1 && (!a.shared || __ldcg(a.lens + b) < 0)) continue;
    const int un = deal.un[s];
    if (un == 0) continue;
    const int i = (x == 0 ? r : row) * a.G + hg;
    const int li = kvh * tiles_of(a, s) + i / TR;
    const long ub = deal.cum[s] + (long)li * un;
    // the last w with T * w / W <= u has unit u
    const int w0 = (int)(((ub + 1) * W - 1) / T), w1 = (int)(((ub + un) * W - 1) / T);
    first[x] = w0 + item0(a, s) + li;
    count[x] = w1 - w0 + 1;
    rt[x] = i % TR;
  }
  const int total = count[0] + count[1];
  auto at = [&](int i) -> long {
    return i < count[0] ? (long)(first[0] + i) * TR + rt[0] : (long)(first[1] + i - count[0]) * TR + rt[1];
  };
  float M = -INFINITY;
  for (int i = lane; i < total; i += 32) M = fmaxf(M, __ldcg(a.ml + at(i) * 2));
  M = warp_max_xor(M);
  const float ref = M == -INFINITY ? 0.0f : M;
  float acc[D / 32], ls = 0.0f;
#pragma unroll
  for (int c = 0; c < D / 32; ++c) acc[c] = 0.0f;
  for (int i0 = 0; i0 < total; i0 += 32) {
    float f = 0.0f, lf = 0.0f;
    if (i0 + lane < total) {
      const long p = at(i0 + lane) * 2;
      f = ex2(__ldcg(a.ml + p) - ref);
      lf = f * __ldcg(a.ml + p + 1);
    }
    const int n = min(32, total - i0);
#pragma unroll 4
    for (int i = 0; i < n; ++i) {
      const float fi = __shfl_sync(FULL, f, i);
      ls += __shfl_sync(FULL, lf, i);
      const float* o = a.o + at(i0 + i) * D + lane;
#pragma unroll
      for (int c = 0; c < D / 32; ++c) acc[c] = fmaf(fi, __ldcg(o + 32 * c), acc[c]);
    }
  }
#pragma unroll
  for (int c = 0; c < D / 32; ++c) {
    const float y = ls > 0.0f ? __fdiv_rn(acc[c], ls) : 0.0f;
    if (j.out) j.out[w * D + 32 * c + lane] = y;
    if constexpr (Q > 0) quant_lane<Q>(y, j.hq, j.hl, j.hs, w * (D / 32) + c, lane);
  }
}

// ---- host --------------------------------------------------------------------------
long items_of(int n_q, int n_kv, int B, int R, int shared) {
  const int G = n_q / n_kv;
  long n = (long)B * n_kv * ((R * G + TR - 1) / TR);
  if (shared) n += (long)n_kv * (((long)B * R * G + TR - 1) / TR);
  return n;
}

template <typename F>
bool allow_shared(F f, std::atomic<int> (&done)[kMaxDevices], int bytes) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return false;
  if (done[dev].load(std::memory_order_acquire)) return true;
  if (cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) return false;
  done[dev].store(1, std::memory_order_release);
  return true;
}

template <typename A>
cudaError_t launch(void (*f)(A), dim3 grid, dim3 block, int smem, int pdl, cudaStream_t stream, const A& args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, f, args);
}

template <int TYPE, int D>
lk_status run_type(const AttnArgs& a, int pdl, cudaStream_t stream) {
  static std::atomic<int> done[kMaxDevices];
  typedef Cfg<TYPE, D> C;
  if (!allow_shared(attn_kernel<TYPE, D>, done, C::RING)) return LK_ERR_CUDA;
  if (launch(attn_kernel<TYPE, D>, dim3(a.W), dim3(32 * C::NW), C::RING, pdl, stream, a) != cudaSuccess) {
    cudaGetLastError();
    return LK_ERR_CUDA;
  }
  return LK_OK;
}

template <int D>
lk_status run_d(const AttnArgs& a, int type, lk_mode mode, const JoinArgs& j, int pdl, cudaStream_t stream) {
  const lk_status st = type == LK_KV_F16    ? run_type<LK_KV_F16, D>(a, pdl, stream)
                       : type == LK_KV_BF16 ? run_type<LK_KV_BF16, D>(a, pdl, stream)
                                            : run_type<LK_KV_Q8, D>(a, pdl, stream);
  if (st) return st;
  const long heads = (long)a.B * a.R * a.n_q;
  const dim3 grid((unsigned)((heads + 3) / 4)), block(128);
  const cudaError_t e = mode == LK_DEQUANT   ? launch(attn_join_kernel<0, D>, grid, block, 0, 1, stream, j)
                        : mode == LK_INT8ACT ? launch(attn_join_kernel<1, D>, grid, block, 0, 1, stream, j)
                                             : launch(attn_join_kernel<2, D>, grid, block, 0, 1, stream, j);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return LK_ERR_CUDA;
  }
  return LK_OK;
}

size_t ml_bytes(long slots) { return ((size_t)slots * TR * 8 + 255) / 256 * 256; }

}  // namespace lkattn

using namespace lkattn;

extern "C" {

size_t lk_attn_workspace_bytes(int n_q, int n_kv, int head_dim, int B, int R, int shared) {
  if ((head_dim != 64 && head_dim != 128) || n_kv < 1 || n_q < n_kv || n_q % n_kv || n_q > 4096) return 0;
  if (B < 0 || R < 0 || B > LK_MAX_BATCH || R > LK_MAX_BATCH || B * R > LK_MAX_BATCH) return 0;
  const long slots = kMaxWorkers + items_of(n_q, n_kv, B, R, shared != 0);
  return ml_bytes(slots) + (size_t)slots * TR * head_dim * 4;
}

lk_status lk_attn_shared(const lk_kv_cache* cache, const float* q, int n_q, const int32_t* prefix_table,
                         int prefix_w, int prefix_len, const int32_t* table, int table_w, const int32_t* lens, int B,
                         int R, float scale, lk_mode mode, float* out, int8_t* hq, int8_t* hl, float* hs, void* ws,
                         size_t ws_bytes, const lk_launch_cfg* cfg, cudaStream_t stream) {
  if (mode < LK_DEQUANT || mode > LK_TWOPASS || check_launch_cfg(cfg)) return LK_ERR_ARG;
  lk_status st = check_cache(cache, n_q);
  if (st) return st;
  if ((st = check_rows(cache, table, table_w, lens, B, R))) return st;
  if (prefix_len < 0 || prefix_w < 0 || (long)prefix_w * cache->page > 0x40000000L ||
      prefix_len > (long)prefix_w * cache->page)
    return LK_ERR_SHAPE;
  if (!(scale - scale == 0.0f)) return LK_ERR_ARG;  // not finite
  if (B == 0 || R == 0) return LK_OK;
  if (!q || (prefix_len > 0 && !prefix_table)) return LK_ERR_ARG;
  if (!aligned(q, 16) || (prefix_len > 0 && !aligned(prefix_table, 4))) return LK_ERR_ALIGN;
  if (mode == LK_DEQUANT ? !out : false) return LK_ERR_ARG;
  if (out && !aligned(out, 4)) return LK_ERR_ALIGN;
  if (mode != LK_DEQUANT && (st = check_act_out(mode, hq, hl, hs))) return st;
  const int shared = prefix_len > 0;
  if (!ws || ws_bytes < lk_attn_workspace_bytes(n_q, cache->n_kv, cache->head_dim, B, R, shared))
    return LK_ERR_WORKSPACE;
  if (!aligned(ws, 16)) return LK_ERR_ALIGN;
  const DeviceInfo* d = device_info(nullptr);
  if (!d) return LK_ERR_CUDA;
  AttnArgs a = {};
  a.q = q;
  a.n_q = n_q;
  a.n_kv = cache->n_kv;
  a.G = n_q / cache->n_kv;
  a.k = cache->k;
  a.v = cache->v;
  a.ks = (const __half*)cache->ks;
  a.vs = (const __half*)cache->vs;
  a.page_log2 = log2_of(cache->page);
  a.n_pages = cache->n_pages;
  a.table = table;
  a.table_w = table_w;
  a.lens = lens;
  a.B = B;
  a.R = R;
  a.ptable = prefix_table;
  a.plen = prefix_len;
  a.pcap = prefix_len;
  a.shared = shared;
  a.qscale = scale * 1.44269504088896340736f;
  a.W = d->sm_count < kMaxWorkers ? d->sm_count : kMaxWorkers;
  const long slots = kMaxWorkers + items_of(n_q, cache->n_kv, B, R, shared);
  a.ml = (float*)ws;
  a.o = (float*)((char*)ws + ml_bytes(slots));
  JoinArgs j;
  j.a = a;
  j.out = out;
  j.hq = hq;
  j.hl = mode == LK_TWOPASS ? hl : nullptr;
  j.hs = hs;
  const int pdl = cfg_pdl(cfg);
  return cache->head_dim == 128 ? run_d<128>(a, cache->type, mode, j, pdl, stream)
                                : run_d<64>(a, cache->type, mode, j, pdl, stream);
}

lk_status lk_attn(const lk_kv_cache* cache, const float* q, int n_q, const int32_t* table, int table_w,
                  const int32_t* lens, int B, int R, float scale, lk_mode mode, float* out, int8_t* hq, int8_t* hl,
                  float* hs, void* ws, size_t ws_bytes, const lk_launch_cfg* cfg, cudaStream_t stream) {
  return lk_attn_shared(cache, q, n_q, nullptr, 0, 0, table, table_w, lens, B, R, scale, mode, out, hq, hl, hs, ws,
                        ws_bytes, cfg, stream);
}

}  // extern "C"
