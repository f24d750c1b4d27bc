// Attention for many query rows on the same keys (include/lk_attn.h): a
// shared prefix, or several new tokens of a sequence, on the fifth-generation
// tensor cores.
//
// With up to 256 query rows to a key/value head the products, not the cache's
// bytes, set the time: a block takes 256 rows and walks over its share of the
// keys in tiles of 128.  Two streams, each with an S tile (scores, then the
// weights in its place) and an O tile (128 columns each) in tensor memory, and
// a warpgroup of 128 threads, a thread to a row, keep the tensor pipe busy in
// turn: while one stream's warpgroup turns scores into weights, the pipe has
// the other's products.  More than 128 rows: a stream has 128 of the rows and
// both use each tile; else both have the same rows and take the tiles in turn.
//
// Precision as in the streaming kernel, but for bf16's queries: keys and values
// enter as stored, queries and weights as two 16-bit terms (the low term's MMAs
// accumulate on the high term's; a third bf16 term of the queries would take the
// room of the second stream's, or of the ring, for errors of 2e-6 of the
// result's norm that long f32 sums have too); a tile's weighted values start a
// fresh accumulator and are added in f32 registers, 128 keys at a time.
//
// Measured (GPU time of a whole call, 32 query / 8 key heads of 128): 64 new
// tokens behind 32768 in bf16 55 us: 1.25 PFLOP/s of products, twice the plain
// count for the second terms (tensor pipe 57 % busy in the kernel: a 4.9 k cycle
// period of 4.2 k cycles of MMAs, and the first and last tiles).  24 sequences on
// a Q8 prefix of 16384: 56 us with their own tokens' launch before it, the kernel 38,
// bound by the conversion of levels to f16 terms.
//
// Roles: warp 0 issues the MMAs (one thread), warps 2 and 3 fill a ring of
// tile buffers with tensor copies in the 128-byte swizzle of the MMA operands,
// keys as a K-major and values as an MN-major B operand; warpgroups
// 1 and 2 are the streams.  Every wait is bounded (option "wait_us"); one that
// runs out raises the device error word and ends the block.
#include <type_traits>

#include "lk_attn.cuh"
#include "lk_tc.cuh"

using namespace lk;
using namespace lkh;
using namespace lktc;

namespace lkattn {

constexpr int kTileThreads = 384, kTileRegs = 168;

template <int TYPE, int D>
struct TCfg {
  static constexpr bool BF = TYPE == LK_KV_BF16, Q8 = TYPE == LK_KV_Q8;
  static constexpr int KT = Q8 ? 64 : 128;          // keys of a tile
  static constexpr int HALF = 128 * 128;            // 128 rows of 64 16-bit values
  static constexpr int BUF = (D / 64) * HALF;       // a tile of keys or values
  static constexpr int QS = 2 * BUF;                // a stream's queries, high and low terms
  static constexpr int NB = D == 128 ? 3 : 8;       // ring buffers
  // Q8: levels and scales of 64 tokens as they come, two for each of the three
  // warps that convert them; the streams share the queries
  static constexpr int RAW = Q8 ? 64 * D + 64 * D / 16 : 0, NRAW = Q8 ? 6 : 0;
  static constexpr int QX = Q8 ? 0 : QS;            // from stream 0's queries to stream 1's
  static constexpr int SMEM = QS + QX + NB * BUF + NRAW * RAW + 1024;
  // Registers: the launch has kTileThreads * kTileRegs of them; the streams
  // take 2 * 128 * STREAM and leave 128 * REST, the same sum.
  static constexpr int STREAM = Q8 ? 224 : 232, REST = Q8 ? 56 : 40;
  static_assert(kTileThreads * kTileRegs == 2 * 128 * STREAM + 128 * REST, "register split");
};

// Where a tile's K and V are in a segment's order of ring fills (nt tiles):
// the order in which the MMAs use them.
__device__ __forceinline__ int k_at(bool both, int t) { return both ? 2 * t : t == 0 ? 0 : 2 * t - 1; }
__device__ __forceinline__ int v_at(bool both, int t, int nt) {
  return both ? 2 * t + 1 : t == nt - 1 ? 2 * nt - 1 : 2 * t + 2;
}

struct Segment {
  int s, n, kvh, group, ub, nt, rows, slot;
  bool both;  // more than 128 rows: both streams use each tile
};

// The next segment of the share [u0, u1), u0 moved behind it.
__device__ __forceinline__ Segment next_segment(const AttnArgs& a, const Deal& d, int& s, int& u0, int u1) {
  Segment g;
  while (d.cum[s + 1] <= u0) ++s;
  const int un = d.un[s], groups = groups_of<true>(a, s), rel = u0 - d.cum[s], li = rel / un;
  g.s = s;
  g.n = d.n[s];
  g.ub = rel - li * un;
  g.nt = min(un - g.ub, u1 - u0);
  g.kvh = li / groups;
  g.group = li - g.kvh * groups;
  g.rows = min(1 << a.trows_log2, rows_of(a, s) - (g.group << a.trows_log2));
  g.both = g.rows > 128;
  g.slot = (int)blockIdx.x + item0<true>(a, s) + li;
  u0 += g.nt;
  return g;
}

// Fill i of a segment: its tile, and whether it is the values'.
__device__ __forceinline__ int tile_of_fill(const Segment& g, int i, bool& is_v) {
  if (g.both) return is_v = i & 1, i >> 1;
  if (i == 0) return is_v = false, 0;
  if (i == 2 * g.nt - 1) return is_v = true, g.nt - 1;
  is_v = !(i & 1);
  return is_v ? (i - 2) >> 1 : (i + 1) >> 1;
}

// Q8: the power of two that brings the largest scale of a 64-token tile to 64 ..
// 128.  A lane has 16 bytes of the scales (`in`: of tokens that are there), of
// which tokens up to `left` from the tile's first count.
template <int D>
__device__ __forceinline__ float scale_shift(bool in, uint4 w, int left) {
  constexpr int LPG = D / 16, TP = 16 / LPG, WT = D / 64;  // lanes of 16 tokens, tokens of a lane, words of a token
  const int lane = threadIdx.x & 31, k0 = 16 * (lane / LPG) + (lane % LPG) * TP;
  unsigned mx = 0;
  if (in) {
    const unsigned x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (k0 + i / WT < left) mx = max(mx, max(x[i] & 0x7fffu, (x[i] >> 16) & 0x7fffu));
  }
  mx = __reduce_max_sync(FULL, mx);
  const float m = __half2float(__ushort_as_half((unsigned short)mx));  // 0, or at least 2^-24
  return mx ? __uint_as_float((260u - (__float_as_uint(m) >> 23)) << 23) : 1.0f;
}

// The same from the cache.  pg: lanes 0..3 have the pages of the tile's groups of
// 16 tokens (-1: none).
template <int D>
__device__ __forceinline__ uint4 tile_scales(const AttnArgs& a, const uint16_t* sc, int pg, int key0, int kvh, bool& in) {
  constexpr int LPG = D / 16;
  const int lane = threadIdx.x & 31, grp = lane / LPG, k0 = key0 + 16 * grp, p = __shfl_sync(FULL, pg, grp & 3);
  in = grp < 4 && p >= 0;
  const long r = (((long)max(p, 0) * a.n_kv + kvh) << a.page_log2) + (k0 & ((1 << a.page_log2) - 1));
  return in ? __ldca((const uint4*)(sc + r * (D / 32)) + lane % LPG) : make_uint4(0, 0, 0, 0);
}

__device__ __forceinline__ uint4 lds128(unsigned at) {
  uint4 r;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(at) : "memory");
  return r;
}
__device__ __forceinline__ float lds_half(unsigned at) {
  unsigned short r;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(r) : "r"(at) : "memory");
  return __half2float(__ushort_as_half(r));
}
// 32 bytes to global memory
__device__ __forceinline__ void stg256(float* p, const float* v) {
  asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(v[0]), "f"(v[1]), "f"(v[2]),
               "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
               : "memory");
}
__device__ __forceinline__ void sts128(unsigned at, const unsigned* r) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]) : "memory");
}

template <int TYPE, int D>
__global__ void __launch_bounds__(kTileThreads, 1) attn_tile_kernel(const __grid_constant__ AttnArgs a) {
  typedef TCfg<TYPE, D> C;
  constexpr bool BF = C::BF, Q8 = C::Q8;
  constexpr int KT = C::KT;
  extern __shared__ unsigned char raw[];
  __shared__ Deal deal;
  __shared__ __align__(8) unsigned long long bars[2 * C::NB + 11 + C::NRAW];
  __shared__ unsigned tmem_slot;
  __shared__ int abort_flag;
  const unsigned base = (smem_addr(raw) + 1023u) & ~1023u;
  const unsigned ring = base + C::QS + C::QX, raws = ring + C::NB * C::BUF;
  const unsigned bar0 = smem_addr(bars);
  const unsigned b_full = bar0, b_free = bar0 + 8 * C::NB, b_q = bar0 + 16 * C::NB, b_s = b_q + 16, b_p = b_s + 16,
                 b_o = b_p + 16, b_drain = b_o + 16, b_meet = b_drain + 8, b_raw = b_meet + 16;
  const int lane = threadIdx.x & 31, warp = __shfl_sync(FULL, threadIdx.x >> 5, 0);
  if (threadIdx.x == 0) {
    if constexpr (!Q8) {
      map_prefetch(&a.kmap);
      map_prefetch(&a.vmap);
    }
    for (int i = 0; i < C::NB; ++i) bar_init(b_full + 8 * i, Q8 ? 1 : 2), bar_init(b_free + 8 * i, 1);
    for (int x = 0; x < 2; ++x) {
      bar_init(b_q + 8 * x, 128);
      bar_init(b_s + 8 * x, 1);
      bar_init(b_p + 8 * x, 128);
      bar_init(b_o + 8 * x, 1);
    }
    bar_init(b_drain, 1);
    // Q8: of both streams; else of each
    bar_init(b_meet, Q8 ? 256 : 128), bar_init(b_meet + 8, 128);
    for (int i = 0; i < C::NRAW; ++i) bar_init(b_raw + 8 * i, 1);
    abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  // Nothing of the caller's is read before this wait, behind the call's streaming
  // launch either: that one's having waited for the caller's work before it let
  // this one start says nothing of what this one sees.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // Tensor memory is taken behind the wait and ahead of the dependents' start: a
  // launch before or after that wants some on this SM too would wait for this one's,
  // and this one for its end, or for what it took first.
  if (warp == 0) tm_alloc(smem_addr(&tmem_slot), 512);
  if (warp == 1) make_deal<true>(a, deal, lens_pair(a));
  tm_before();
  __syncthreads();
  tm_after();
  asm volatile("griddepcontrol.launch_dependents;" :::);
  const unsigned tmem = __shfl_sync(FULL, *(volatile unsigned*)&tmem_slot, 0);
  const int T = deal.cum[a.B + a.shared];
  int u0 = 0, u1 = 0;
  if (T > 0) {
    const Shares blocks = tile_blocks(a, T);
    if ((int)blockIdx.x < blocks.n) {
      u0 = blocks.begin(blockIdx.x);
      u1 = u0 + blocks.size(blockIdx.x);
    }
  }
  int s = 0;
  auto wait = [&](unsigned bar, unsigned parity) -> bool {
    if (bar_wait(bar, parity & 1u, a.wait_ns, &abort_flag)) return true;
    if (!*(volatile int*)&abort_flag) {
      *(volatile int*)&abort_flag = 1;
      atomicOr(a.err, ERR_TILE_WAIT);
    }
    return false;
  };

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::REST));
    if (warp == 0) {
      // ---- MMA issue: the warp stays together, one elected thread issues ---------------
      constexpr unsigned id_qk = inst_desc(BF, false, 128, 128), id_pv = inst_desc(BF, true, 128, D);
      const bool el = elect_one();
      const unsigned long long q_desc = smem_desc(base, 16, 1024), k_desc = smem_desc(ring, 16, 1024),
                               v_desc = smem_desc(ring, C::HALF, 1024);
      unsigned nb = 0, seg = 0, np0 = 0, np1 = 0;
      bool ok = true;
      while (u0 < u1 && ok) {
        const Segment g = next_segment(a, deal, s, u0, u1);
        const int cnt0 = g.both ? g.nt : (g.nt + 1) / 2, cnt1 = g.both ? g.nt : g.nt / 2;
        // scores of stream x's tile j
        auto qk = [&](int x, int j) -> bool {
          const unsigned f = nb + k_at(g.both, g.both ? j : 2 * j + x), buf = f % C::NB;
          if (!__all_sync(FULL, wait(b_full + 8 * buf, f / C::NB))) return false;
          tm_after();
          const unsigned long long q = q_desc + ((x * C::QX) >> 4), k = k_desc + ((buf * C::BUF) >> 4);
          const unsigned dst = tmem + x * 128;
          if (el) {
#pragma unroll
            for (int i = 0; i < 2 * (D / 16); ++i) {
              const int term = i / (D / 16), st = i % (D / 16), off = (st >> 2) * C::HALF + (st & 3) * 32;
              mma_ss(dst, q + ((term * C::BUF + off) >> 4), k + (off >> 4), id_qk, i > 0);
            }
            mma_commit(b_s + 8 * x);
            if (!g.both || x == 1) mma_commit(b_free + 8 * buf);
          }
          __syncwarp();
          return true;
        };
        // weighted values of stream x's tile j
        auto pv = [&](int x, int j) -> bool {
          const unsigned f = nb + v_at(g.both, g.both ? j : 2 * j + x, g.nt), buf = f % C::NB;
          if (!__all_sync(FULL, wait(b_full + 8 * buf, f / C::NB) && wait(b_p + 8 * x, x ? np1 : np0))) return false;
          x ? ++np1 : ++np0;
          tm_after();
          const unsigned long long v = v_desc + ((buf * C::BUF) >> 4);
          const unsigned p = tmem + x * 128, dst = tmem + 256 + x * 128;
          if (el) {
            // 16 columns hold the two terms of 16 keys' weights
            if constexpr (Q8) {
              // rows 0..63 of the tile are the values' high terms, 64..127 the low
              // ones; low times low is left out (2^-22)
#pragma unroll
              for (int i = 0; i < 12; ++i) {
                const int st = i & 3, term = i >> 2;
                mma_ts(dst, p + st * 16 + (term == 1 ? 8 : 0), v + (((term == 2 ? 4 + st : st) * 2048) >> 4), id_pv, i > 0);
              }
            } else {
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                const int term = i / 8, st = i % 8;
                mma_ts(dst, p + st * 16 + term * 8, v + ((st * 2048) >> 4), id_pv, i > 0);
              }
            }
            mma_commit(b_o + 8 * x);
            if (!g.both || x == 1) mma_commit(b_free + 8 * buf);
          }
          __syncwarp();
          return true;
        };
        ok = __all_sync(FULL, wait(b_q, seg)) && qk(0, 0) && __all_sync(FULL, wait(b_q + 8, seg)) && (!cnt1 || qk(1, 0));
        // a stream without a tile is told all the same: it must not run ahead and
        // complete a second phase of its queries' barrier
        if (!cnt1 && el) mma_commit(b_s + 8);
        __syncwarp();
        for (int i = 0; i < 2 * cnt0 && ok; ++i) {
          const int x = i & 1, j = i >> 1, cnt = x ? cnt1 : cnt0;
          if (j < cnt) ok = pv(x, j);
          if (ok && j + 1 < cnt) ok = qk(x, j + 1);
        }
        nb += 2 * g.nt;
        ++seg;
      }
      // nothing of this block is in flight when its tensor memory is freed
      if (el) mma_commit(b_drain);
      __syncwarp();
      if (!bar_drain(b_drain, 0, a.wait_ns) && lane == 0) atomicOr(a.err, ERR_TILE_WAIT);
    } else if (Q8) {
      // ---- the ring's fills, Q8 ------------------------------------------------------
      // Warps 1 to 3 take the fills in turn: 64 tokens' levels and scales come by
      // bulk copies, a fill ahead, and are written as two f16 terms of level times
      // scale, the high one rounded, the low one what that left (exact), rows 0..63
      // and 64..127 of the tile.  Scales are first shifted so that the tile's largest
      // is 64 .. 128; the streams shift back.
      constexpr int CPR = D / 16, KN = 64 * CPR / 32;  // 16-byte pieces of a token, of a lane
      const unsigned raw0 = raws + (warp - 1) * 2 * C::RAW, raw_bar = b_raw + 16 * (warp - 1);
      unsigned f = 0, n_raw = 0;      // fills, fills of this warp
      unsigned of = 0, o_there = 0;   // the fill before: its number, its groups of 16 tokens that are there,
      int o_left = 0;                 // tokens from its first
      bool ok = true;
      // convert this warp's fill number n
      const auto convert = [&](unsigned n) {
        const unsigned src = raw0 + (n & 1) * C::RAW, buf = of % C::NB, dst0 = ring + buf * C::BUF;
        ok = __all_sync(FULL, wait(raw_bar + 8 * (n & 1), n >> 1));
        if (!ok) return;
        const bool in = lane < 4 * (D / 16) && ((o_there >> (lane / (D / 16))) & 1u);
        const float up = scale_shift<D>(in, in ? lds128(src + 64 * D + lane * 16) : make_uint4(0, 0, 0, 0), o_left);
        ok = __all_sync(FULL, wait(b_free + 8 * buf, (of / C::NB) ^ 1u));
        if (!ok) return;
        constexpr int GB = 4;  // pieces read together
#pragma unroll 1
        for (int k0 = 0; k0 < KN; k0 += GB) {
          uint4 w[GB];
          float e[GB];
#pragma unroll
          for (int k = 0; k < GB; ++k) {
            const int c = lane + 32 * (k0 + k), row = c / CPR;
            w[k] = lds128(src + c * 16);
            e[k] = lds_half(src + 64 * D + (row * (D / 32) + ((c % CPR) >> 1)) * 2);
          }
#pragma unroll
          for (int k = 0; k < GB; ++k) {
            const int c = lane + 32 * (k0 + k), row = c / CPR, ch = c % CPR;
            const bool have = row < o_left && ((o_there >> (row >> 4)) & 1u);
            const __half2 e2 = __half2half2(__float2half_rn(have ? e[k] * up : 0.0f));
            const unsigned x[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
            const unsigned at = dst0 + (ch >> 2) * C::HALF + row * 128;
#pragma unroll
            for (int q = 0; q < 2; ++q) {  // 8 values: 16 bytes of each term
              unsigned hi[4], lo[4];
#pragma unroll
              for (int r = 0; r < 4; ++r) {
                const unsigned pr = level_pair(x[2 * q + (r >> 1)] ^ 0x80808080u, r & 1 ? 0x4342 : 0x4140);
                const __half2 l2 = *(const __half2*)&pr, h2 = __hmul2(l2, e2), r2 = __hfma2(l2, e2, __hneg2(h2));
                hi[r] = *(const unsigned*)&h2;
                lo[r] = *(const unsigned*)&r2;
              }
              const unsigned pc = at + (((2 * (ch & 3) + q) ^ (row & 7)) << 4);
              sts128(pc, hi);
              sts128(pc + 64 * 128, lo);
            }
          }
        }
        fence_async();
        __syncwarp();
        if (lane == 0) bar_arrive(b_full + 8 * buf);
      };
      while (u0 < u1 && ok) {
        const Segment g = next_segment(a, deal, s, u0, u1);
        const int* table = g.s == a.B ? a.ptable : a.table + (long)g.s * a.table_w;
        for (int i = 0; i < 2 * g.nt && ok; ++i, ++f) {
          if (f % 3 != (unsigned)warp - 1) continue;
          bool is_v;
          const int t = tile_of_fill(g, i, is_v), key0 = (g.ub + t) * KT;
          int pg = -1;
          if (lane < 4 && key0 + 16 * lane < g.n) {
            pg = __ldca(table + ((key0 + 16 * lane) >> a.page_log2));
            if ((unsigned)pg >= (unsigned)a.n_pages) pg = -1;
          }
          const unsigned there = __ballot_sync(FULL, pg >= 0), bar = raw_bar + 8 * (n_raw & 1);
          const unsigned dst = raw0 + (n_raw & 1) * C::RAW;
          if (lane == 0) bar_expect(bar, __popc(there) * 17 * D);
          __syncwarp();
          if (pg >= 0) {
            const int k0 = key0 + 16 * lane;
            const long r = (((long)pg * a.n_kv + g.kvh) << a.page_log2) + (k0 & ((1 << a.page_log2) - 1));
            bulk_in(dst + lane * 16 * D, (const char*)(is_v ? a.v : a.k) + r * D, 16 * D, bar);
            bulk_in(dst + 64 * D + lane * D, (is_v ? a.vs : a.ks) + r * (D / 32), D, bar);
          }
          if (n_raw > 0) convert(n_raw - 1);
          of = f, o_there = there, o_left = g.n - key0;
          ++n_raw;
        }
      }
      if (ok && n_raw > 0) convert(n_raw - 1);
      // a block that gave up: its copies have landed before it ends
      if (!ok)
        for (unsigned n = n_raw > 2 ? n_raw - 2 : 0; n < n_raw; ++n) bar_drain(raw_bar + 8 * (n & 1), (n >> 1) & 1u, a.wait_ns);
    } else if (warp >= 2) {
      // ---- the ring's fills ----------------------------------------------------------
      // Warp 2 + h fills part h: of D 128 half h of every token, of D 64 half the
      // tokens.  A tile whose tokens are all there comes by tensor copies; one with
      // trailing or absent tokens by copies of the threads, which write zeros there.
      const int part = warp - 2;
      constexpr int TOK = D == 128 ? KT : KT / 2;  // tokens of a part
      const int tok0 = D == 128 ? 0 : part * TOK;
      unsigned f = 0;
      bool ok = true;
      while (u0 < u1 && ok) {
        const Segment g = next_segment(a, deal, s, u0, u1);
        const int* table = g.s == a.B ? a.ptable : a.table + (long)g.s * a.table_w;
        for (int i = 0; i < 2 * g.nt && ok; ++i, ++f) {
          bool is_v;
          const int t = tile_of_fill(g, i, is_v), key0 = (g.ub + t) * KT + tok0;
          // pages of the part's groups of 16 tokens
          int pg = -1;
          if (lane < TOK / 16 && key0 + 16 * lane < g.n) {
            pg = __ldca(table + ((key0 + 16 * lane) >> a.page_log2));
            if ((unsigned)pg >= (unsigned)a.n_pages) pg = -1;
          }
          const bool all = __all_sync(FULL, lane >= TOK / 16 || pg >= 0) && key0 + TOK <= g.n;
          const unsigned buf = f % C::NB, bar = b_full + 8 * buf;
          const unsigned dst0 = ring + buf * C::BUF + (D == 128 ? part * C::HALF : tok0 * 128);
          ok = __all_sync(FULL, wait(b_free + 8 * buf, (f / C::NB) ^ 1u));
          if (!ok) break;
          if (all) {
            if (lane == 0) bar_expect(bar, TOK * 128);
            __syncwarp();
            // group l's first token begins a box, if the box is not another's
            const int k0 = key0 + 16 * lane, in = k0 & (a.box - 1);
            if (lane < TOK / 16 && in == 0)
              tma_2d(dst0 + lane * 2048, is_v ? &a.vmap : &a.kmap, D == 128 ? part * 64 : 0,
                     ((pg * a.n_kv + g.kvh) << a.page_log2) + (k0 & ((1 << a.page_log2) - 1)), bar);
          } else {
            const char* src0 = (const char*)(is_v ? a.v : a.k) + (D == 128 ? part * 128 : 0);
            const int pc = lane & 7, r_in = lane >> 3;
#pragma unroll 1
            for (int h = 0; h < TOK / 16; ++h) {
              const int p = __shfl_sync(FULL, pg, h), k0 = key0 + 16 * h, left = p >= 0 ? g.n - k0 : 0;
              const long r0 = (((long)max(p, 0) * a.n_kv + g.kvh) << a.page_log2) + (k0 & ((1 << a.page_log2) - 1));
#pragma unroll
              for (int m = 0; m < 4; ++m) {
                const int kk = 4 * m + r_in, row = 16 * h + kk;
                cp16(dst0 + row * 128 + ((pc ^ (row & 7)) << 4), src0 + (r0 + kk) * (2 * D) + pc * 16,
                     kk < left ? 16 : 0);
              }
            }
            cp_commit();
            cp_wait<0>();
            fence_async();
            __syncwarp();
            if (lane == 0) bar_arrive(bar);
          }
        }
      }
      // a block that gave up: its copies have landed before it ends
      if (!ok)
        for (unsigned i = 0; i < C::NB && i < f; ++i)
          if (lane == 0 && !bar_drain(b_full + 8 * ((f - 1 - i) % C::NB), ((f - 1 - i) / C::NB) & 1u, a.wait_ns))
            atomicOr(a.err, ERR_TILE_WAIT);
    }
  } else {
    // ---- a stream: a thread to a row ---------------------------------------------------
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::STREAM));
    const int x = (warp >> 2) - 1, wq = warp & 3, me = threadIdx.x & 127;
    const unsigned tw = tmem + ((unsigned)(32 * wq) << 16);  // the warp's lanes
    const unsigned ts = tw + x * 128, to = tw + 256 + x * 128;
    const unsigned qs = base + x * C::QX;
    constexpr float UP = weight_shift(TYPE);
    unsigned ns = 0, no = 0;  // score and output tiles so far
    bool ok = true, stored = false;
    // the threads of the stream (Q8: of both) meet; a bounded wait as every other
    unsigned met = 0;
    const auto meet = [&]() -> bool {
      const unsigned bar = b_meet + (Q8 ? 0 : 8 * x);
      bar_arrive(bar);
      return __all_sync(FULL, wait(bar, met++));
    };
    while (u0 < u1 && ok) {
      const Segment g = next_segment(a, deal, s, u0, u1);
      const bool pre = g.s == a.B;
      const int* table = pre ? a.ptable : a.table + (long)g.s * a.table_w;
      const int r_first = (g.group << a.trows_log2) + (g.both ? 128 * x : 0);  // row of the head that is the stream's row 0
      const int nr = g.both ? min(128, g.rows - 128 * x) : g.rows;
      const int cnt = g.both ? g.nt : x == 0 ? (g.nt + 1) / 2 : g.nt / 2;
      if (stored) {
        // the last segment's rows have left the queries' place (Q8: both streams
        // are done with the queries)
        if (!Q8 && me == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
        ok = meet();
        if (!ok) break;
      }
      // queries: a warp takes its 32 rows, D / 32 values a lane, all loads first,
      // and writes their two terms swizzled
      float rs = 1.0f;
      {
        // a lane finds its own row's place, rows without a query are zeros
        int off = -1;
        if (me < nr) {
          const int ri = r_first + me, tok = ri / a.G;
          off = (pre ? tok : g.s * a.R + tok) * a.n_q + g.kvh * a.G + (ri - tok * a.G);
        }
        float v[16][D / 32];
#pragma unroll 1
        for (int i0 = 0; i0 < 32; i0 += 16) {
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int at = __shfl_sync(FULL, off, i0 + i);
            const float* q = a.q + (long)at * D + lane * (D / 32);
            float4 f = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (at >= 0) {
              if constexpr (D == 128) f = __ldcg((const float4*)q);
              else *(float2*)&f = __ldcg((const float2*)q);
            }
            v[i][0] = f.x, v[i][1] = f.y;
            if constexpr (D == 128) v[i][2] = f.z, v[i][3] = f.w;
          }
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float am = 0.0f;
#pragma unroll
            for (int c = 0; c < D / 32; ++c) v[i][c] *= a.qscale, am = fmaxf(am, fabsf(v[i][c]));
            if constexpr (!BF) {
              float back;
              const float up = row_shift(warp_absmax(am), back);
              if (lane == i0 + i) rs = back;
#pragma unroll
              for (int c = 0; c < D / 32; ++c) v[i][c] *= up;
            }
            // values lane * D/32 ...: 16-byte piece and place in it
            const int lr = 32 * wq + i0 + i, d0 = lane * (D / 32), piece = (d0 & 63) >> 3;
            const unsigned at = qs + (d0 >> 6) * C::HALF + lr * 128 + ((piece ^ (lr & 7)) << 4) + (d0 & 7) * 2;
#pragma unroll
            for (int term = 0; term < 2; ++term) {
              if (Q8 && x == 1) break;  // stream 0 writes the queries of both
              const unsigned w0 = split2<BF>(v[i][0], v[i][1]);
              if constexpr (D == 128) {
                const unsigned w1 = split2<BF>(v[i][2], v[i][3]);
                asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(at + term * C::BUF), "r"(w0), "r"(w1) : "memory");
              } else {
                asm volatile("st.shared.u32 [%0], %1;" ::"r"(at + term * C::BUF), "r"(w0) : "memory");
              }
            }
          }
        }
      }
      fence_async();
      bar_arrive(b_q + 8 * x);

      int vis = g.n;  // keys that the thread's row sees
      if (!pre && me < nr) {
        const int tok = (r_first + me) / a.G;
        vis = min(g.n, max(0, __ldcg(a.lens + g.s) - a.R + 1 + tok));
      }
      float O[D], m = -INFINITY, l = 0.0f;
#pragma unroll
      for (int i = 0; i < D; ++i) O[i] = 0.0f;
      // what a tile needs beside its products, a tile ahead: its first key, which
      // groups of 16 tokens are there, the powers of two of its scores and values
      int key0 = 0;
      unsigned there = 0;
      float rt = rs, vt = 1.0f;
      const auto look = [&](int j) {
        key0 = (g.ub + (g.both ? j : 2 * j + x)) * KT;
        int pg = -1;
        if (lane < KT / 16 && key0 + 16 * lane < g.n) pg = __ldca(table + ((key0 + 16 * lane) >> a.page_log2));
        if ((unsigned)pg >= (unsigned)a.n_pages) pg = -1;
        there = __ballot_sync(FULL, pg >= 0);
        if constexpr (Q8) {  // reciprocals of powers of two
          bool in;
          const uint4 ks = tile_scales<D>(a, (const uint16_t*)a.ks, pg, key0, g.kvh, in);
          const uint4 vs = tile_scales<D>(a, (const uint16_t*)a.vs, pg, key0, g.kvh, in);
          rt = rs * __frcp_rn(scale_shift<D>(in, ks, g.n - key0));
          vt = __frcp_rn(scale_shift<D>(in, vs, g.n - key0));
        }
      };
      if (cnt > 0) look(0);
      if (cnt == 0) ok = __all_sync(FULL, wait(b_s + 8 * x, ns++));
      for (int j = 0; j < cnt; ++j) {
        const bool whole = __all_sync(FULL, key0 + KT <= vis) && there == (1u << (KT / 16)) - 1;
        const f32x2 vt2 = f2_pack(vt, vt);
        ok = __all_sync(FULL, wait(b_s + 8 * x, ns++));
        if (!ok) break;
        tm_after();
        // The scores' maximum; where some keys are absent or not seen by some row,
        // their scores become -inf on the way.  (Rolled loops: a block runs this
        // code a dozen times, and what is not in the instruction cache yet costs
        // the first tile as much as two later ones.)
        float mx = -INFINITY, mx1 = -INFINITY;
        if (whole) {
#pragma unroll 1
          for (int c = 0; c < KT / 32; ++c) {
            unsigned r[32];
            tm_ld32(ts + 32 * c, r);
            if constexpr (Q8) {
              unsigned r2[16];
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                tm_ld16(ts + 64 + 32 * c + 16 * h, r2);
                tm_ld_wait(r2);
                if (h == 0) tm_ld_wait(r);
#pragma unroll
                for (int k = 0; k < 16; ++k) mx = fmaxf(mx, __uint_as_float(r[16 * h + k]) + __uint_as_float(r2[k]));
              }
            } else {
              tm_ld_wait(r);
#pragma unroll
              for (int k = 0; k < 32; k += 4) {
                mx = max3(mx, __uint_as_float(r[k]), __uint_as_float(r[k + 1]));
                mx1 = max3(mx1, __uint_as_float(r[k + 2]), __uint_as_float(r[k + 3]));
              }
            }
          }
        } else {
#pragma unroll 1
          for (int c = 0; c < KT / 16; ++c) {
            unsigned r[16], r2[16];
            tm_ld16(ts + 16 * c, r);
            if constexpr (Q8) tm_ld16(ts + 64 + 16 * c, r2);
            tm_ld_wait(r);
            if constexpr (Q8) tm_ld_wait(r2);
            const int left = (there >> c) & 1u ? vis - key0 - 16 * c : 0;
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              if (k >= left) {
                r[k] = 0xff800000u;
                if constexpr (Q8) r2[k] = 0u;  // (not a number where the query is none)
              }
              mx = fmaxf(mx, Q8 ? __uint_as_float(r[k]) + __uint_as_float(r2[k]) : __uint_as_float(r[k]));
            }
            tm_st16(ts + 16 * c, r);
            if constexpr (Q8) tm_st16(ts + 64 + 16 * c, r2);
          }
          tm_st_wait();
        }
        const float mn = fmaxf(m, fmaxf(mx, mx1) * rt);
        const float ref = mn == -INFINITY ? 0.0f : mn, al = ex2(m - ref), shift = UP - ref;
        m = mn;
        const f32x2 al2 = f2_pack(al, al);
        // the weights in their place, 16 keys at a time, the next 16 on their way
        f32x2 sum2[2] = {f2_pack(0.0f, 0.0f), f2_pack(0.0f, 0.0f)};
        const f32x2 rt2 = f2_pack(rt, rt), shift2 = f2_pack(shift, shift), minus1 = f2_pack(-1.0f, -1.0f);
        const auto scores = [&](int c, unsigned(&y)[16]) {
          tm_ld16(ts + 16 * c, y);
          if constexpr (Q8) {
            unsigned y2[16];
            tm_ld16(ts + 64 + 16 * c, y2);
            tm_ld_wait(y2);
            tm_ld_wait(y);
#pragma unroll
            for (int k = 0; k < 16; ++k) y[k] = __float_as_uint(__uint_as_float(y[k]) + __uint_as_float(y2[k]));
          }
        };
        const auto weights = [&](int c, const unsigned(&y)[16]) {
          unsigned w[16];
#pragma unroll
          for (int k = 0; k < 16; k += 2) {
            // pairs: one instruction for both halves
            float x0, x1;
            f2_unpack(f2_fma(f2_pack(__uint_as_float(y[k]), __uint_as_float(y[k + 1])), rt2, shift2), x0, x1);
            x0 = ex2(x0), x1 = ex2(x1);
            const f32x2 p = f2_pack(x0, x1);
            sum2[(k >> 1) & 1] = f2_add(sum2[(k >> 1) & 1], p);
            w[k >> 1] = round2<BF>(x0, x1);
            f2_unpack(f2_fma(widen2<BF>(w[k >> 1]), minus1, p), x0, x1);
            w[8 + (k >> 1)] = round2<BF>(x0, x1);
          }
          tm_st16(ts + 16 * c, w);
        };
        {
          unsigned ya[16], yb[16];
          scores(0, ya);
          if constexpr (!Q8) tm_ld_wait(ya);
#pragma unroll 1
          for (int c = 0; c < KT / 16; c += 2) {
            scores(c + 1, yb);
            weights(c, ya);
            if constexpr (!Q8) tm_ld_wait(yb);
            if (c + 2 < KT / 16) scores(c + 2, ya);
            weights(c + 1, yb);
            if constexpr (!Q8) tm_ld_wait(ya);
          }
        }
        float sum0, sum1;
        f2_unpack(f2_add(sum2[0], sum2[1]), sum0, sum1);
        l = fmaf(l, al, sum0 + sum1);
        tm_st_wait();
        tm_before();
        bar_arrive(b_p + 8 * x);
        if (j + 1 < cnt) look(j + 1);
        ok = __all_sync(FULL, wait(b_o + 8 * x, no++));
        if (!ok) break;
        tm_after();
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          unsigned r[32];
          tm_ld32(to + 32 * c, r);
          tm_ld_wait(r);
#pragma unroll
          for (int k = 0; k < 32; k += 2) {
            f32x2 z = f2_pack(__uint_as_float(r[k]), __uint_as_float(r[k + 1]));
            if constexpr (Q8) z = f2_mul(z, vt2);
            f2_unpack(f2_fma(f2_pack(O[32 * c + k], O[32 * c + k + 1]), al2, z), O[32 * c + k], O[32 * c + k + 1]);
          }
        }
        tm_before();
      }
      if (!ok) break;
      // the rows' partials: staged where the queries were (their last product
      // is done), then one bulk store
      const int which = pre ? 1 : 0, sr = tile_slot_rows(rows_of(a, g.s)), row0 = x * (g.both ? 128 : g.rows);
      const long at = (long)g.slot * sr + row0;
      if (me < nr) __stcg((float2*)(a.tml[which] + (at + me) * 2), make_float2(m, l));
      if constexpr (Q8) {  // the queries' place is the other stream's too: each row by its thread
        if (me < nr)
#pragma unroll
          for (int c = 0; c < D / 8; ++c) stg256(a.to[which] + (at + me) * D + 8 * c, O + 8 * c);
      } else {
        if (me < nr)
#pragma unroll
          for (int c = 0; c < D / 4; ++c)
            asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(qs + me * (D * 4) + ((c ^ (me & 7)) << 4)),
                         "f"(O[4 * c]), "f"(O[4 * c + 1]), "f"(O[4 * c + 2]), "f"(O[4 * c + 3])
                         : "memory");
        fence_async();
        ok = meet();
        if (!ok) break;
        if (me == 0) {
          asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(a.to[which] + at * D), "r"(qs),
                       "r"(nr * D * 4)
                       : "memory");
          asm volatile("cp.async.bulk.commit_group;" ::: "memory");
        }
      }
      stored = true;
    }
    if (me == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  }
  tm_before();
  __syncthreads();
  tm_after();
  if (warp == 0) tm_free(tmem, 512);
}

template <int TYPE, int D>
lk_status run_tiles(const AttnArgs& a, int pdl, cudaStream_t stream) {
  typedef TCfg<TYPE, D> C;
  static std::atomic<int> done[kMaxDevices], regs;
  if (!prepare_kernel(attn_tile_kernel<TYPE, D>, done, C::SMEM)) return LK_ERR_CUDA;
  if (!regs.load(std::memory_order_acquire)) {
    // the register split waits forever on a launch with fewer than it assumes
    cudaFuncAttributes fa;
    if (cudaFuncGetAttributes(&fa, attn_tile_kernel<TYPE, D>) != cudaSuccess || fa.numRegs != kTileRegs)
      return LK_ERR_CUDA;
    regs.store(1, std::memory_order_release);
  }
  return launch(attn_tile_kernel<TYPE, D>, dim3(a.TW), dim3(kTileThreads), C::SMEM, pdl, stream, a) == cudaSuccess
             ? LK_OK
             : LK_ERR_CUDA;
}

lk_status launch_tiles(const AttnArgs& a, int type, int D, int pdl, cudaStream_t stream) {
  if (D == 128)
    return type == LK_KV_F16    ? run_tiles<LK_KV_F16, 128>(a, pdl, stream)
           : type == LK_KV_BF16 ? run_tiles<LK_KV_BF16, 128>(a, pdl, stream)
                                : run_tiles<LK_KV_Q8, 128>(a, pdl, stream);
  return type == LK_KV_F16    ? run_tiles<LK_KV_F16, 64>(a, pdl, stream)
         : type == LK_KV_BF16 ? run_tiles<LK_KV_BF16, 64>(a, pdl, stream)
                              : run_tiles<LK_KV_Q8, 64>(a, pdl, stream);
}

}  // namespace lkattn
