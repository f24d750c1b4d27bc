// Attention over the paged cache (include/lk_attn.h): lk_attn,
// lk_attn_shared.
//
// The work and its deal to the blocks are in lk_attn.cuh.  This file has the
// streaming kernel (up to 8 query rows to a key/value head and unit of keys;
// the cache's bytes set its time) and the join of the partials; lk_tile.cu has
// the kernel for many rows on the same keys.
//
// Mathematics.  Scores and weighted sums run on m16n8k16 MMAs whose 16 rows
// are 8 query rows twice: rows 0..7 the high and rows 8..15 the low 16-bit
// term of the f32 operand, so that a lane holds both products of its row and
// their sum costs one addition; keys and values enter as stored (Q8: as their
// integer levels, exact in f16, the scales applied in f32 to the scores and
// folded into the weights).  f16 operands are shifted by powers of two so
// that the low terms stay normal: queries to a row maximum of 2^10, weights by
// 2^14 (Q8: by 2^10, their scales by what brings the largest to 8 .. 16, and the
// product of the two again as two terms).  bf16 has too few bits for two terms
// of a query (errors of 3e-6 of the result's norm where f32 arithmetic has 7e-7):
// a third one has MMAs of its own.  So has a third one of the weights where the
// table has room for few keys (2e-7 instead of 1e-6 to 2e-6); over long
// sequences f32 sums have 5e-7 and more, and it would cost 6 % (16 ragged to
// 16384 100 -> 106 us).  Each unit's weighted values are summed in a fresh
// accumulator and added in f32, so the MMA's own accumulation never runs over
// more than 32 keys.
//
// Data.  Every warp streams its own units through its own stages of shared
// memory: one thread asks for a unit with a few tensor copies (128-byte pieces
// of its tokens' rows, 128-byte swizzle), every lane then reads the operands
// it needs as 16-byte pieces (Q8: 8 and 4 bytes).  The order of the inner index
// of a product is free, so a lane's 8 consecutive values serve two k-steps and
// no value changes lanes.  Copies by the threads themselves (cp.async) were
// measured slower: a warp gets one 512-byte copy instruction through per
// ~190 cycles, 5.1 TB/s with 7 warps.
//
// Few sequences with little room take the same kernel in clusters of up to 8 blocks to
// an item, whose partials stay in shared memory (cluster_size).
//
// Measured (GPU time of a whole call, with its join): 64 x 8192 tokens f16, 32 query /
// 8 key heads of 128: 327 us, 6.6 TB/s; 16 ragged up to 16384 bf16 101 us, 5.6
// TB/s (99 us with two query terms); 1 x 131071 Q8 63 us, 4.5 TB/s, bound by the
// issue of its instructions (58 % of the slots), not by memory; 1 x 1023 f16 in
// clusters 6.2 us (9.1 by the deal and the join), a launch and dependent reads.
#include <cuda_bf16.h>

#include <type_traits>

#include "lk_attn.cuh"
#include "lk_spans.h"
#include "lk_tc.cuh"

using namespace lk;
using namespace lkh;
using namespace lktc;

namespace lkattn {

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

__device__ __forceinline__ unsigned prmt(unsigned a, unsigned b, unsigned s) { return __byte_perm(a, b, s); }

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

// ---- clusters ---------------------------------------------------------------------------
constexpr int kMaxCluster = 8;
// All threads of all blocks of the cluster; every block comes here, whatever
// became of its own waits, which are bounded.
__device__ __forceinline__ void cluster_meet() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ unsigned cluster_addr(unsigned at, unsigned rank) {
  unsigned r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(at), "r"(rank));
  return r;
}
__device__ __forceinline__ void ld_far(unsigned at, float& x, float& y) {
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(x), "=f"(y) : "r"(at) : "memory");
}
__device__ __forceinline__ void ld_far(unsigned at, float (&v)[2]) { ld_far(at, v[0], v[1]); }
__device__ __forceinline__ void ld_far(unsigned at, float (&v)[4]) {
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3])
               : "r"(at)
               : "memory");
}

template <int TYPE, int D>
struct Cfg {
  static constexpr int EB = TYPE == LK_KV_Q8 ? 1 : 2;              // bytes of a stored value
  static constexpr int KV = UNIT * D * EB;                         // bytes of a unit's keys
  static constexpr int SC = TYPE == LK_KV_Q8 ? UNIT * D / 16 : 0;  // bytes of their scales
  static constexpr int STAGE = (2 * (KV + SC) + 1023) / 1024 * 1024;
  static constexpr int ROW = EB * D < 128 ? EB * D : 128;          // bytes of a box row
  static constexpr int PARTS = EB * D / ROW;                       // boxes of a token's row
  static constexpr int NW = TYPE != LK_KV_Q8 && D == 128 ? 7 : 12;  // warps
  static constexpr int ST = TYPE == LK_KV_Q8 && D == 64 ? 3 : 2;     // stages a warp
  static constexpr int RING = NW * ST * STAGE + 1024;  // and the base's alignment
  static_assert(STAGE * ST >= TR * (D + 4) * 4 && NW <= kMaxWarps, "a warp's partial fits in its stages");
  static_assert(RING + 2048 <= 232448, "shared memory of a block");
};

// Where a warp is: unit u of the item of row tile `tile` (of `tiles`) and
// key/value head kvh of sequence s, whose items have un units and n keys.
struct Cursor {
  int s, kvh, tile, tiles, u, un, n;
  __device__ __forceinline__ int item() const { return kvh * tiles + tile; }
};

// By a whole warp.
__device__ __forceinline__ Cursor cursor_at(const AttnArgs& a, const Deal& d, int unit) {
  const int lane = threadIdx.x & 31, nseq = a.B + a.shared;
  Cursor c;
  c.s = 0;
  for (int s0 = 0; s0 < nseq; s0 += 32)
    c.s += __popc(__ballot_sync(FULL, s0 + lane < nseq && d.cum[s0 + lane + 1] <= unit));
  c.un = d.un[c.s];
  c.n = d.n[c.s];
  const int rel = unit - d.cum[c.s], li = rel / c.un;
  c.u = rel - li * c.un;
  c.tiles = groups_of<false>(a, c.s);
  c.kvh = li / c.tiles;
  c.tile = li - c.kvh * c.tiles;
  return c;
}

// To the next unit; behind the last one s is the number of sequences.
__device__ __forceinline__ void advance(const AttnArgs& a, const Deal& d, Cursor& c) {
  if (++c.u < c.un) return;
  c.u = 0;
  if (++c.tile < c.tiles) return;
  c.tile = 0;
  if (++c.kvh < a.n_kv) return;
  c.kvh = 0;
  const int nseq = a.B + a.shared;
  while (++c.s < nseq)
    if ((c.un = d.un[c.s]) > 0) {
      c.n = d.n[c.s];
      c.tiles = groups_of<false>(a, c.s);
      return;
    }
}

// What both ways of joining write: rows, and / or words and scales.
struct JoinArgs {
  AttnArgs a;
  float* out;
  int8_t* hq;
  int8_t* hl;
  float* hs;
  int mode;
  int wide;  // out takes a lane's values in one store
};

// Row and head w (row * n_q + head): a lane's D / 32 neighbouring sums over the
// weights' sum, as f32 and / or quantized.  A sum of 0: the row sees nothing.  One
// that is not a number (the maxima drop such scores, the sums do not) stays so.
template <int Q, int D>
__device__ __forceinline__ void finish(const JoinArgs& j, long w, float (&acc)[D / 32], float ls, int lane) {
  constexpr int V = D / 32;
#pragma unroll
  for (int c = 0; c < V; ++c) acc[c] = ls != 0.0f ? __fdiv_rn(acc[c], ls) : 0.0f;
  if (j.out) {
    float* y = j.out + w * D + lane * V;
    if (j.wide) {
      if constexpr (V == 4) *(float4*)y = *(const float4*)acc;
      else *(float2*)y = *(const float2*)acc;
    } else {
#pragma unroll
      for (int c = 0; c < V; ++c) y[c] = acc[c];
    }
  }
  if constexpr (Q > 0) {
#pragma unroll
    for (int c = 0; c < V; ++c) {
      // value 32 c + lane is in lane (32 c + lane) / V
      float y = 0.0f;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float t = __shfl_sync(FULL, acc[e], (32 * c + lane) / V);
        y = lane % V == e ? t : y;
      }
      quant_lane<Q>(y, j.hq, j.hl, j.hs, w * (D / 32) + c, lane);
    }
  }
}

// CL: the blocks of an item are a cluster and join their parts themselves (j);
// else a is all, and parts go to the workspace.
template <int TYPE, int D, bool CL, bool FINE>
__device__ __forceinline__ void attn_body(const AttnArgs& a, const JoinArgs* j) {
  typedef Cfg<TYPE, D> C;
  constexpr bool Q8 = TYPE == LK_KV_Q8;
  constexpr int KS = D / 16;  // k-steps of a score
  constexpr int NT = D / 8;   // n-tiles of the output
  constexpr bool QT = TYPE == LK_KV_BF16;  // a third term of the queries
  constexpr bool WT = QT && FINE;          // and of the weights
  extern __shared__ unsigned char raw[];
  __shared__ std::conditional_t<CL, int, Deal> deal_place;
  __shared__ float wml[C::NW][TR][2];
  __shared__ __align__(8) unsigned long long bars[C::NW * C::ST];
  __shared__ int abort_flag;
  __shared__ __align__(8) float cml[CL ? TR : 1][2];
  unsigned char* smem = raw + ((1024u - (smem_addr(raw) & 1023u)) & 1023u);
  if (threadIdx.x < C::NW * C::ST) bar_init(smem_addr(bars + threadIdx.x), 1);
  if (threadIdx.x == 0) {
    abort_flag = 0;
    map_prefetch(&a.kmap);
    map_prefetch(&a.vmap);
  }
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  // (a dependent has next to nothing to do before its own wait: started earlier
  // it would only hold its share of the SMs)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" :::);
  if constexpr (!CL)
    if (threadIdx.x < 32) make_deal<false>(a, deal_place, lens_pair(a));
  __syncthreads();
  const int lane = threadIdx.x & 31, warp = __shfl_sync(FULL, threadIdx.x >> 5, 0), g = lane >> 2, t = lane & 3;
  int cn, we, wa, left;  // units of the block, its warps with units; the warp's first and their number
  Cursor cc;
  int pu = 0;  // clusters: units of the prefix, which come before the sequence's own
  bool one;  // the block's units are all one item's: its warps join their parts
  if constexpr (CL) {
    const int item = (int)blockIdx.x / a.C, rank = (int)blockIdx.x - item * a.C;
    cc.tiles = groups_of<false>(a, 0);
    const int items = a.n_kv * cc.tiles, li = item - item / items * items;
    cc.s = item / items;
    cc.kvh = li / cc.tiles;
    cc.tile = li - cc.kvh * cc.tiles;
    const int len = __ldcg(a.lens + cc.s);
    cc.n = min(max(len, 0), a.table_w << a.page_log2);
    if (a.shared && len >= 0) pu = (a.plen + UNIT - 1) / UNIT;
    cc.un = pu + (cc.n + UNIT - 1) / UNIT;
    cc.u = cn = 0;
    if (cc.un > 0) {
      const Shares blocks(cc.un, min(a.C, cc.un));
      cc.u = rank < blocks.k ? blocks.begin(rank) : cc.un;
      cn = rank < blocks.k ? blocks.size(rank) : 0;
    }
    one = true;
  } else {
    const Deal& deal = deal_place;
    const int T = deal.cum[a.B + a.shared];
    if (T == 0) return;
    const Shares blocks = stream_blocks(a, C::NW, T);
    if ((int)blockIdx.x >= blocks.n) return;
    cn = blocks.size(blockIdx.x);
    cc = cursor_at(a, deal, blocks.begin(blockIdx.x));
    one = cc.u + cn <= cc.un;
  }
  we = min(C::NW, cn);
  const Shares warps(cn, max(we, 1));
  wa = warp < we ? warps.begin(warp) : cn;
  left = warp < we ? warps.size(warp) : 0;
  if (one) cc.u += wa;
  else if constexpr (!CL)
    if (left > 0) cc = cursor_at(a, deal_place, stream_blocks(a, C::NW, deal_place.cum[a.B + a.shared]).begin(blockIdx.x) + wa);
  const auto next = [&](Cursor& c) {
    if constexpr (CL) ++c.u;
    else advance(a, deal_place, c);
  };
  const unsigned ring = smem_addr(smem) + warp * C::ST * C::STAGE, bar0 = smem_addr(bars) + 8 * warp * C::ST;

  // pages of a unit's two halves (-1: none)
  auto pages = [&](const Cursor& c, int (&pg)[2]) {
    const bool pre = CL ? c.u < pu : c.s == a.B;
    const int* table = pre ? a.ptable : a.table + (long)c.s * a.table_w;
    const int n = CL && pre ? a.plen : c.n, key0 = (CL && !pre ? c.u - pu : c.u) * UNIT;
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      const int key = key0 + 16 * hf;
      pg[hf] = -1;
      if (key < n) {
        const int p = __ldca(table + (key >> a.page_log2));
        if ((unsigned)p < (unsigned)a.n_pages) pg[hf] = p;
      }
    }
  };
  unsigned there = 0;  // bits 2 i, 2 i + 1: stage i's halves have pages
  unsigned asked = 0;  // bit i: stage i has a unit that was not waited for
  // ask for a unit (one thread of the warp); a.box is 16 or 32 rows
  auto issue = [&](const Cursor& c, const int (&pg)[2], int stage) {
    there = (there & ~(3u << (2 * stage))) | ((pg[0] >= 0 ? 1u : 0u) | (pg[1] >= 0 ? 2u : 0u)) << (2 * stage);
    asked |= 1u << stage;
    if (lane != 0) return;
    const unsigned st = ring + stage * C::STAGE, bar = bar0 + 8 * stage;
    const int n_box = a.box == 32 ? 1 : 2;
    unsigned bytes = 0;
    for (int hf = 0; hf < n_box; ++hf)
      if (pg[hf] >= 0) bytes += 2 * a.box * (D * C::EB + (Q8 ? D / 16 : 0));
    bar_expect(bar, bytes);
    for (int hf = 0; hf < n_box; ++hf) {
      if (pg[hf] < 0) continue;
      const int key0 = (CL && c.u >= pu ? c.u - pu : c.u) * UNIT + 16 * hf;
      const int r0 = ((pg[hf] * a.n_kv + c.kvh) << a.page_log2) + (key0 & ((1 << a.page_log2) - 1));
#pragma unroll
      for (int p = 0; p < C::PARTS; ++p) {
        const unsigned at = st + p * UNIT * C::ROW + 16 * hf * C::ROW;
        tma_2d(at, &a.kmap, p * (C::ROW / C::EB), r0, bar);
        tma_2d(at + C::KV, &a.vmap, p * (C::ROW / C::EB), r0, bar);
      }
      if constexpr (Q8) {
        const unsigned at = st + 2 * C::KV + hf * D, n = a.box * (D / 16);
        bulk_in(at, (const char*)a.ks + (long)r0 * (D / 16), n, bar);
        bulk_in(at + C::SC, (const char*)a.vs + (long)r0 * (D / 16), n, bar);
      }
    }
  };

  // The ring's first units; ac: the unit to ask for next, with its pages.
  Cursor ac = cc;
  int ask = left, pg[2] = {-1, -1};
  {
    Cursor c[C::ST];
    int p[C::ST][2];
#pragma unroll
    for (int i = 0; i < C::ST; ++i) {
      c[i] = ac;
      if (i < ask) {
        pages(ac, p[i]);
        next(ac);
      }
    }
    if (ask > C::ST) pages(ac, pg);
#pragma unroll
    for (int i = 0; i < C::ST; ++i)
      if (i < ask) issue(c[i], p[i], i);
    ask -= min(ask, C::ST);
  }
  unsigned phases = 0;  // bit i: the parity stage i's copies complete next
  int stage = 0;
  bool fail = false;
  while (left > 0) {
    // ---- an item
    const int s = cc.s, kvh = cc.kvh, tile = cc.tile;
    const bool pre = s == a.B;
    const int nrows = min(TR, rows_of(a, s) - tile * TR);
    const long slot = (long)blockIdx.x * C::NW + (one ? 0 : warp) + item0<false>(a, s) + cc.item();
    // the lane's query row (the last row again where there are fewer)
    const int ri = tile * TR + min(g, nrows - 1);
    const int tok = ri / a.G;  // row of the batch (prefix) or of the sequence
    const int row = pre ? tok : s * a.R + tok;
    int row_vis = cc.n;  // keys that the row sees
    if (!pre) row_vis = min(cc.n, max(0, __ldcg(a.lens + s) - a.R + 1 + tok));
    unsigned qa[KS][4], qc[QT ? KS : 1][2];
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
        const float up = row_shift(amax, rs);
#pragma unroll
        for (int i = 0; i < D / 4; ++i) x[i] *= up;
      }
      // k-step k: registers 4 k .. 4 k + 3 are the lane's four inner indices
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        qa[k][0] = split2<TYPE == LK_KV_BF16>(x[4 * k], x[4 * k + 1]);
        qa[k][2] = split2<TYPE == LK_KV_BF16>(x[4 * k + 2], x[4 * k + 3]);
        qa[k][1] = split2<TYPE == LK_KV_BF16>(x[4 * k], x[4 * k + 1]);
        qa[k][3] = split2<TYPE == LK_KV_BF16>(x[4 * k + 2], x[4 * k + 3]);
        if constexpr (QT) {
          qc[k][0] = round2<true>(x[4 * k], x[4 * k + 1]);
          qc[k][1] = round2<true>(x[4 * k + 2], x[4 * k + 3]);
        }
      }
    }

    float O[NT][2], m = -INFINITY, l = 0.0f, dvm = 0.0f, dsc = 1.0f;
#pragma unroll
    for (int i = 0; i < NT; ++i) O[i][0] = O[i][1] = 0.0f;
    const int ue = min(cc.un, cc.u + left);
    left -= ue - cc.u;
    for (int u = cc.u; u < ue; ++u) {
      if (!bar_wait(bar0 + 8 * stage, (phases >> stage) & 1u, a.wait_ns, &abort_flag)) {
        if (lane == 0 && !*(volatile int*)&abort_flag) {
          *(volatile int*)&abort_flag = 1;
          atomicOr(a.err, ERR_ATTN_WAIT);
        }
        fail = true;
      }
      fail = __any_sync(FULL, fail);
      if (fail) break;
      phases ^= 1u << stage;
      asked &= ~(1u << stage);
      const unsigned st = ring + stage * C::STAGE;
      // ---- scores: lane (g, t) has row g with keys 8 i + 2 t, + 1
      float sc[4][2];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (!Q8) {
          float c[4] = {0.f, 0.f, 0.f, 0.f}, c3[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int j = 0; j < D / 32; ++j) {
            // piece 4 (j & 1) + t of the token's part j >> 1
            const uint4 w = lds128(st + (j >> 1) * (UNIT * 128) + (8 * i + g) * 128 + (((4 * (j & 1) + t) ^ g) << 4));
            mma16<TYPE>(c, qa[2 * j][0], qa[2 * j][1], qa[2 * j][2], qa[2 * j][3], w.x, w.y);
            mma16<TYPE>(c, qa[2 * j + 1][0], qa[2 * j + 1][1], qa[2 * j + 1][2], qa[2 * j + 1][3], w.z, w.w);
            if constexpr (QT) {
              mma16<TYPE>(c3, qc[2 * j][0], 0u, qc[2 * j][1], 0u, w.x, w.y);
              mma16<TYPE>(c3, qc[2 * j + 1][0], 0u, qc[2 * j + 1][1], 0u, w.z, w.w);
            }
          }
          sc[i][0] = (c[0] + (c[2] + c3[0])) * rs;
          sc[i][1] = (c[1] + (c[3] + c3[1])) * rs;
        } else {
          const int key = 8 * i + g, fk = D == 128 ? g : (key >> 1) & 3;  // the swizzle
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
      const bool in0 = (there >> (2 * stage)) & 1u, in1 = (there >> (2 * stage + 1)) & 1u;  // the halves' pages
      const bool of_pre = CL && u < pu;
      const int k0 = (CL && !of_pre ? u - pu : u) * UNIT, n = of_pre ? a.plen : cc.n, vis = of_pre ? a.plen : row_vis;
      const bool whole = k0 + UNIT <= n && in0 && in1;
      if (!__all_sync(FULL, whole && k0 + UNIT <= vis)) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int x = 0; x < 2; ++x)
            if (k0 + 8 * i + 2 * t + x >= vis || !(i < 2 ? in0 : in1)) sc[i][x] = -INFINITY;
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
      constexpr float UP = weight_shift(TYPE);
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
          if (k0 + w / HW >= n || !(w / HW < 16 ? in0 : in1)) x = 0;
          mx = max(mx, max(x & 0xffffu, x >> 16));
        }
        mx = __reduce_max_sync(FULL, mx);
        const float dm = __half2float(__ushort_as_half((unsigned short)mx));
        if (dm > dvm) {  // warp-uniform
          dvm = dm;
          // as an f16 factor that brings the largest scale to 8 .. 16 (2^14 at
          // most): smaller ones stay normal down to 2^-18 of it
          const float ns = fminf(__uint_as_float((257u - (__float_as_uint(dm) >> 23)) << 23), 16384.0f);
          al *= ns / dsc;  // powers of two; O is 0 before the first
          dsc = ns;
        }
      }
      if (__any_sync(FULL, al != 1.0f)) {
#pragma unroll
        for (int i = 0; i < NT; ++i) O[i][0] *= al, O[i][1] *= al;
      }
      if constexpr (!Q8) {
        unsigned ph[2][4], pc[WT ? 2 : 1][2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          ph[k][0] = split2<TYPE == LK_KV_BF16>(p[2 * k][0], p[2 * k][1]);
          ph[k][2] = split2<TYPE == LK_KV_BF16>(p[2 * k + 1][0], p[2 * k + 1][1]);
          ph[k][1] = split2<TYPE == LK_KV_BF16>(p[2 * k][0], p[2 * k][1]);
          ph[k][3] = split2<TYPE == LK_KV_BF16>(p[2 * k + 1][0], p[2 * k + 1][1]);
          if constexpr (WT) {
            pc[k][0] = round2<true>(p[2 * k][0], p[2 * k][1]);
            pc[k][1] = round2<true>(p[2 * k + 1][0], p[2 * k + 1][1]);
          }
        }
#pragma unroll
        for (int h = 0; h < D / 64; ++h) {
          unsigned w[8][4];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int key = 16 * (e >> 2) + 2 * t + (e & 1) + 8 * ((e >> 1) & 1);
            uint4 x = lds128(st + C::KV + h * (UNIT * 128) + key * 128 + ((g ^ (key & 7)) << 4));
            // what lies behind the tokens may be anything: 0 * NaN is not 0
            if (!whole && (k0 + key >= n || !(e < 4 ? in0 : in1))) x = make_uint4(0, 0, 0, 0);
            w[e][0] = x.x, w[e][1] = x.y, w[e][2] = x.z, w[e][3] = x.w;
          }
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const unsigned sel = j & 1 ? 0x7632 : 0x5410;
            float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const unsigned b0 = prmt(w[4 * k][j >> 1], w[4 * k + 1][j >> 1], sel),
                             b1 = prmt(w[4 * k + 2][j >> 1], w[4 * k + 3][j >> 1], sel);
              mma16<TYPE>(c, ph[k][0], ph[k][1], ph[k][2], ph[k][3], b0, b1);
              if constexpr (WT) mma16<TYPE>(c, pc[k][0], 0u, pc[k][1], 0u, b0, b1);
            }
            O[8 * h + j][0] += c[0] + c[2];
            O[8 * h + j][1] += c[1] + c[3];
          }
        }
      } else {
        // weights as two f16 terms, keys 8 i + 2 t, + 1 in a pair
        __half2 p_hi[4], p_lo[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const unsigned h = split2<false>(p[i][0], p[i][1]), r = split2<false>(p[i][0], p[i][1]);
          p_hi[i] = *(const __half2*)&h;
          p_lo[i] = *(const __half2*)&r;
        }
        // value scales of those keys times dsc (exact above 2^-24); 0 for absent
        // tokens, whose scales may be anything
        __half2 d0[4][D / 64], d1[4][D / 64];
        const __half2 ds2 = __float2half2_rn(dsc);
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
          const int key = k0 + 8 * i + 2 * t;
#pragma unroll
          for (int x = 0; x < D / 64; ++x) {
            if (!whole) {
              if (key >= n || !(i < 2 ? in0 : in1)) d0[i][x] = __half2half2(__ushort_as_half(0));
              if (key + 1 >= n || !(i < 2 ? in0 : in1)) d1[i][x] = __half2half2(__ushort_as_half(0));
            }
            d0[i][x] = __hmul2(d0[i][x], ds2);
            d1[i][x] = __hmul2(d1[i][x], ds2);
          }
        }
#pragma unroll
        for (int b = 0; b < D / 32; ++b) {
          // weight times scale, again as two terms: the high one rounded, the
          // low one what that left (exact) and the weight's low term
          unsigned ph[2][4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const __half2 e = b & 1 ? __highs2half2(d0[i][b >> 1], d1[i][b >> 1]) : __lows2half2(d0[i][b >> 1], d1[i][b >> 1]);
            const __half2 hi = __hmul2(p_hi[i], e);
            const __half2 lo = __hfma2(p_lo[i], e, __hfma2(p_hi[i], e, __hneg2(hi)));
            ph[i >> 1][2 * (i & 1)] = *(const unsigned*)&hi;
            ph[i >> 1][2 * (i & 1) + 1] = *(const unsigned*)&lo;
          }
          unsigned w[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int key = 16 * (e >> 2) + 2 * t + (e & 1) + 8 * ((e >> 1) & 1);
            const int fv = D == 128 ? key & 7 : (key >> 1) & 3;
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
      }
      // ---- the stage's next unit
      __syncwarp();  // every lane is done with the stage
      if (ask > 0) {
        issue(ac, pg, stage);
        next(ac);
        if (--ask > 0) pages(ac, pg);
      }
      stage = stage + 1 == C::ST ? 0 : stage + 1;
    }
    if (fail) break;
    cc.u = ue - 1;
    if (left > 0) next(cc);

    // ---- its partial
    if constexpr (Q8) {
      const float back = 1.0f / dsc;
#pragma unroll
      for (int i = 0; i < NT; ++i) O[i][0] *= back, O[i][1] *= back;
    }
    l += __shfl_xor_sync(FULL, l, 1);
    l += __shfl_xor_sync(FULL, l, 2);
    if (g < nrows) {
      // of several items to a block, straight to the workspace; of one, beside
      // the other warps' in the stages, which are done with
      float* to = one ? (float*)(smem + (size_t)warp * C::ST * C::STAGE) + g * (D + 4) : a.o + (slot * TR + g) * D;
      constexpr int E = Q8 ? 4 : 8;  // neighbouring values of a lane
#pragma unroll
      for (int b = 0; b < NT / E; ++b)
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int i = 0; i < E; i += 4)
            *(float4*)(to + b * 8 * E + (2 * t + x) * E + i) =
                make_float4(O[b * E + i][x], O[b * E + i + 1][x], O[b * E + i + 2][x], O[b * E + i + 3][x]);
      if (t == 0) {
        if (one) wml[warp][g][0] = m, wml[warp][g][1] = l;
        else *(float2*)(a.ml + (slot * TR + g) * 2) = make_float2(m, l);
      }
    }
  }
  if (fail) {
    // nothing of the warp's copies is in flight when the block ends
    for (int i = 0; i < C::ST; ++i)
      if ((asked >> i) & 1u) bar_drain(bar0 + 8 * i, (phases >> i) & 1u, a.wait_ns);
  }
  if constexpr (CL) __syncthreads();
  else if (!one || __syncthreads_or(abort_flag)) return;

  // ---- one item: the warps' partials, joined in warp order
  {
    const int s = cc.s, nrows = min(TR, rows_of(a, s) - cc.tile * TR);
    const long slot = CL ? 0 : (long)blockIdx.x * C::NW + item0<false>(a, s) + cc.item();
    for (int i = threadIdx.x; i < nrows * D; i += 32 * C::NW) {
      const int r = i / D, d = i - r * D;
      float M = -INFINITY;
      for (int w = 0; w < we; ++w) M = fmaxf(M, wml[w][r][0]);
      const float ref = M == -INFINITY ? 0.0f : M;
      float acc = 0.0f, ls = 0.0f;
      for (int w = 0; w < we; ++w) {
        const float f = ex2(wml[w][r][0] - ref);
        const float ov = *(const float*)(smem + (size_t)w * C::ST * C::STAGE + (size_t)(r * (D + 4) + d) * 4);
        acc = fmaf(f, ov, acc);
        ls = fmaf(f, wml[w][r][1], ls);
      }
      if constexpr (CL) {
        // in the first warp's place: each value's only reader is its writer
        *(float*)(smem + (size_t)(r * (D + 4) + d) * 4) = acc;
        if (d == 0) cml[r][0] = M, cml[r][1] = ls;
      } else {
        a.o[(slot * TR + r) * D + d] = acc;
        if (d == 0) *(float2*)(a.ml + (slot * TR + r) * 2) = make_float2(M, ls);
      }
    }
    if constexpr (CL) {
      // ---- the cluster's partials, joined in rank order: row r by block r % C
      cluster_meet();
      for (int r = (int)blockIdx.x % a.C + warp * a.C; r < nrows; r += C::NW * a.C) {
        constexpr int V = D / 32;
        float m[kMaxCluster], l[kMaxCluster], o[kMaxCluster][V], M = -INFINITY;
#pragma unroll
        for (int c = 0; c < kMaxCluster; ++c) {
          // (a rank that is not there: the last one's again, with weight 0)
          const unsigned from = min(c, a.C - 1);
          ld_far(cluster_addr(smem_addr(&cml[r][0]), from), m[c], l[c]);
          ld_far(cluster_addr(smem_addr(smem) + (r * (D + 4) + lane * V) * 4, from), o[c]);
          if (c >= a.C) m[c] = -INFINITY;
          M = fmaxf(M, m[c]);
        }
        const float ref = M == -INFINITY ? 0.0f : M;
        float acc[V], ls = 0.0f;
#pragma unroll
        for (int e = 0; e < V; ++e) acc[e] = 0.0f;
#pragma unroll
        for (int c = 0; c < kMaxCluster; ++c) {
          const float f = ex2(m[c] - ref);
          ls = fmaf(f, l[c], ls);
#pragma unroll
          for (int e = 0; e < V; ++e) acc[e] = fmaf(f, o[c][e], acc[e]);
        }
        const int ri = cc.tile * TR + r, tok = ri / a.G;
        const long w = (long)(s * a.R + tok) * a.n_q + cc.kvh * a.G + (ri - tok * a.G);
        if (j->mode == LK_DEQUANT) finish<0, D>(*j, w, acc, ls, lane);
        else if (j->mode == LK_INT8ACT) finish<1, D>(*j, w, acc, ls, lane);
        else finish<2, D>(*j, w, acc, ls, lane);
      }
      cluster_meet();  // a block's parts are there until all have read them
    }
  }
}

template <int TYPE, int D, bool FINE>
__global__ void __launch_bounds__(32 * Cfg<TYPE, D>::NW, 1) attn_kernel(const __grid_constant__ AttnArgs a) {
  attn_body<TYPE, D, false, FINE>(a, nullptr);
}
template <int TYPE, int D>
__global__ void __launch_bounds__(32 * Cfg<TYPE, D>::NW, 1) attn_cluster_kernel(const __grid_constant__ JoinArgs j) {
  attn_body<TYPE, D, true, true>(j.a, &j);
}

// ---- the join: one warp per row and query head ---------------------------------------
// Partials of a row from one item: entry i (0 <= i < n) has its maximum and
// sum at ml + 2 at(i), its values at o + D at(i); the values' 16-byte pieces are
// permuted by flip (tile partials).  Streaming: n0 warps of the item's first
// block, nm blocks that have nothing else, warps of its last block.  Tile: a
// block each, with `per` partials of the row.
struct Source {
  const float* ml;
  const float* o;
  int first, mid, last;
  int n, n0, nm, step, per, hop, flip;
  __device__ __forceinline__ int at(int i) const {  // (rows of the workspace: 32 bits)
    const int k = i - n0, j = per == 1 ? k : k >> 1;
    const int x = first + i * TR, y = mid + j * step + (k - j * per) * hop, w = last + (k - nm) * TR;
    const int yw = j < nm ? y : w;
    return i < n0 ? x : yw;
  }
};

// Row i of key/value head kvh in sequence s of the streaming deal.
__device__ __forceinline__ Source stream_source(const AttnArgs& a, const Deal& d, int s, int kvh, int i) {
  Source r = {};
  const int un = d.un[s];
  if (un == 0) return r;
  const int T = d.cum[a.B + a.shared];
  const Shares blocks = stream_blocks(a, a.NW, T);
  const int tile = i / TR, li = kvh * groups_of<false>(a, s) + tile, item = item0<false>(a, s) + li;
  const int ib = d.cum[s] + li * un, ie = ib + un;  // the item's units
  const int c0 = blocks.holder(ib), c1 = blocks.holder(ie - 1);
  // entries of block c: one if it has nothing else, else one of each warp with units of the item
  const auto part = [&](int c, int& at, int& n) {
    const int ca = blocks.begin(c), cn = blocks.size(c);
    int w0 = 0, w1 = 0;
    if (ca < ib || ca + cn > ie) {
      const Shares warps(cn, min(a.NW, cn));
      w0 = warps.holder(max(ca, ib) - ca);
      w1 = warps.holder(min(ca + cn, ie) - ca - 1);
    }
    at = (c * a.NW + w0 + item) * TR + i % TR;
    n = w1 - w0 + 1;
  };
  int n2 = 0;
  part(c0, r.first, r.n0);
  if (c1 > c0) part(c1, r.last, n2);
  r.nm = c1 > c0 ? c1 - c0 - 1 : 0;
  r.mid = ((c0 + 1) * a.NW + item) * TR + i % TR;
  r.step = a.NW * TR;
  r.per = 1;
  r.n = r.n0 + r.nm + n2;
  r.ml = a.ml;
  r.o = a.o;
  return r;
}

// The same of the tile deal.
__device__ __forceinline__ Source tile_source(const AttnArgs& a, const Deal& d, int s, int kvh, int i) {
  Source r = {};
  const int un = d.un[s];
  if (un == 0) return r;
  const int T = d.cum[a.B + a.shared], trows = 1 << a.trows_log2;
  const Shares blocks = tile_blocks(a, T);
  const int group = i >> a.trows_log2, li = kvh * groups_of<true>(a, s) + group, ig = i - group * trows;
  const int ub = d.cum[s] + li * un, w0 = blocks.holder(ub), w1 = blocks.holder(ub + un - 1);
  const int rows = rows_of(a, s), rg = min(trows, rows - group * trows), which = s == a.B ? 1 : 0;
  r.step = tile_slot_rows(rows);
  r.mid = (w0 + item0<true>(a, s) + li) * r.step + ig;
  r.nm = w1 - w0 + 1;
  r.per = rg <= 128 ? 2 : 1;
  r.hop = rg;
  r.n = r.nm * r.per;
  r.ml = a.tml[which];
  r.o = a.to[which];
  r.flip = a.tflip ? ig & 7 : 0;
  return r;
}

// Values through L2; volatile, so that a batch of loads stays together ahead of
// its sums (moved down to them, each waits alone: 14.8 against 9.9 us).
__device__ __forceinline__ void ld_cg(const float* p, float (&v)[4]) {
  asm volatile("ld.global.cg.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]) : "l"(p));
}
__device__ __forceinline__ void ld_cg(const float* p, float (&v)[2]) {
  asm volatile("ld.global.cg.v2.f32 {%0, %1}, [%2];" : "=f"(v[0]), "=f"(v[1]) : "l"(p));
}

template <int Q, int D>
__global__ void __launch_bounds__(128) attn_join_kernel(const JoinArgs j) {
  const AttnArgs& a = j.a;
  __shared__ Deal deal, tdeal;
  asm volatile("griddepcontrol.launch_dependents;" :::);
  const int lane = threadIdx.x & 31;
  // The deal and the first partials' places are worked out ahead of the wait,
  // from lengths that nobody vouches for there (in bounds whatever they are);
  // behind it they are read again, and where they are others all is done anew.
  // With all of it behind the wait 7 x 5 drafts take 15.3 instead of 13.7 us, 64 new
  // rows 57.8 instead of 55.1: much of it is fetching code.
  int2 lens = lens_pair(a);
  const auto deals = [&] {
    if (threadIdx.x < 32) make_deal<false>(a, deal, lens);
    else if (threadIdx.x < 64 && (a.own_tiled || a.pre_tiled)) make_deal<true>(a, tdeal, lens);
    __syncthreads();
  };
  deals();
  const long heads = (long)a.B * a.R * a.n_q, w0 = (long)blockIdx.x * 4 + (threadIdx.x >> 5);
  const long w = w0 < heads ? w0 : heads - 1;
  const int row = (int)(w / a.n_q), h = (int)(w - (long)row * a.n_q), kvh = h / a.G, hg = h - kvh * a.G;
  const int b = row / a.R, r = row - b * a.R;
  // A lane has V neighbouring values.  Partials come in batches of NB whose
  // loads are all in flight at once, the values' not waiting for the maxima's.
  constexpr int V = D / 32, NB = 16;
  float M = -INFINITY, acc[V], ls = 0.0f;
#pragma unroll
  for (int c = 0; c < V; ++c) acc[c] = 0.0f;
  // the row's own item, then its prefix item (a rolled loop: this code runs
  // once, and what it takes to fetch it counts)
  bool waited = false;
#pragma unroll 1
  for (int x = 0; x < 2; ++x) {
    if (x == 1 && (!a.shared || __ldcg(a.lens + b) < 0)) break;
    const int s = x ? a.B : b, i = (x ? row : r) * a.G + hg;
    const Source z = (x ? a.pre_tiled : a.own_tiled) ? tile_source(a, tdeal, s, kvh, i) : stream_source(a, deal, s, kvh, i);
    if (!waited) {
      waited = true;
      asm volatile("griddepcontrol.wait;" ::: "memory");
      const int2 now = lens_pair(a);
      const bool other = now.x != lens.x || now.y != lens.y;
      if (__syncthreads_or(other)) {
        lens = now;
        deals();
        --x;
        continue;
      }
    }
    const int at = V == 4 ? (lane ^ z.flip) * 4 : ((lane >> 1) ^ z.flip) * 4 + (lane & 1) * 2;
#pragma unroll 1
    for (int i0 = 0; i0 < z.n; i0 += NB) {
      // lane i < NB: partial i0 + i's place, maximum and sum
      const bool in = lane < NB && i0 + lane < z.n;
      const int mine = z.at(min(i0 + (lane & (NB - 1)), z.n - 1));
      const float2 p = in ? __ldcg((const float2*)(z.ml + (long)mine * 2)) : make_float2(-INFINITY, 0.0f);
      float o[NB][V];
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        ld_cg(z.o + (long)__shfl_sync(FULL, mine, i) * D + at, o[i]);
      }
      const float m = fmaxf(M, warp_max_xor(p.x)), ref = m == -INFINITY ? 0.0f : m;
      const float al = ex2(M - ref), f = ex2(p.x - ref), lf = f * p.y;
      M = m;
      ls *= al;
#pragma unroll
      for (int c = 0; c < V; ++c) acc[c] *= al;
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        const float fi = __shfl_sync(FULL, f, i);
        ls += __shfl_sync(FULL, lf, i);
        if (i0 + i < z.n) {
#pragma unroll
          for (int c = 0; c < V; ++c) acc[c] = fmaf(fi, o[i][c], acc[c]);
        }
      }
    }
  }
  if (w0 < heads) finish<Q, D>(j, w, acc, ls, lane);
}

// ---- host --------------------------------------------------------------------------
// Whether rows on the same keys go to the tile kernel.  The streaming kernel
// reads the keys once per 8 rows (from L2), the tile kernel once, at a fixed
// cost of some 10 us; a sequence's length is not known here, a prefix's is.
// Measured (whole call, streaming / tile, us; 8 kv heads):
//   sequences, f16 D 128: 24 rows 1 x 8000 20.2 / 21.0, 4 x 8000 48.6 / 38.9, 20
//     rows 8 x 1000 21.0 / 20.3; 64 rows 1 x 8000 39.4 / 21.9, 1 x 1000 13.9 / 14.0
//   Q8 D 128: 24 rows 4 x 8000 48.0 / 60.9, 36 rows 67.9 / 61.7, 64 rows 101 / 64
//   prefix, f16 D 128: 96 rows 2000 25.5 / 27.8, 128 rows 29.5 / 28.5; 32 rows 8000
//     27.9 / 31.1, 48 rows 34.3 / 32.1; 24 rows 32000 55.5 / 48.5; bf16 96 rows 2000
//     29.9 / 27.1, 32 rows 8000 29.4 / 30.0
//   D 64: 64 rows 8000 26.8 / 26.6; 24 rows 32000 32.8 / 34.6
//   Q8 D 128: 256 rows 2000 42.9 / 37.9, 48 rows 8000 34.4 / 38.8, 64 rows 41.1 /
//     39.6; D 64: 96 rows 8000 38.3 / 32.2, 64 rows 26.8 / 30.9
bool tiled(long rows, int type, int D, long keys) {
  const bool q8 = type == LK_KV_Q8;
  if (rows <= (q8 ? 32 : 16)) return false;
  return keys < 0 || rows * keys * D >= (q8 ? 1L << 26 : 1L << 25);
}

// Blocks of an item (up to 8 rows of one key/value head and sequence) where they
// are a cluster that joins its own partials: one launch, no deal, and a shared
// prefix is read by every sequence, from L2.  0 where the equal deal to all SMs
// and the join launch, or the tile kernel, do better.  `room`: tokens the table
// has room for; how many there are is not known here.  All clusters run at
// once: a block has an SM, and 15 clusters of 8, 23 of 6, 28 of 5, 36 of 4, 46 of 3,
// 76 of 2 fit (cudaOccupancyMaxActiveClusters; 16 of 8 took two rounds: 5.8 us
// became 10.1).  Measured (GPU time, cluster / deal and join, us; 8 kv heads of
// 128, 4 query heads each; f16, Q8 nearly the same where it is not named):
//   B 1, C 8: 256 tokens 5.5 / 8.3, 1000 6.2 / 9.3, 4000 9.5 / 12.3, 8000 12.7 / 15.9,
//     12700 17.2 / 17.4; D 64 12700 f16 10.2 / 13.6, Q8 12.3 / 11.6, 20000 f16 12.8 / 14.8
//   B 2, C 6: 250 6.1 / 9.4, 1000 6.9 / 9.7, 4000 10.4 / 15.2 (12.8 with C 4)
//   B 4, C 4: 256 5.9 / 9.4, 1000 8.3 / 10.5, 4000 13.6 / 17.8
//   B 5, C 3: 250 6.3 / 9.4, 1000 8.6 / 13.1, 2000 11.0 / 15.3
//   B 16, C 1: 256 8.3 / 12.2, 1000 13.3 / 17.5
// against the tile kernel and its join, rows on the same keys:
//   32 rows, C 4: f16 500 7.3 / 12.4, 4000 14.7 / 18.1; Q8 4000 14.4 / 17.1
//   64 rows, C 2: f16 500 9.3 / 12.8, 2000 14.8 / 16.3; bf16 16.6 / 15.8; Q8 14.2 / 19.8
//   256 rows, 2 kv heads, C 2: f16 500 9.1 / 14.9, 2000 14.2 / 15.6; Q8 14.0 / 23.3
// on a prefix, 8 sequences of 77, C 2: f16 300 7.2 / 14.6, 1900 13.1 / 18.1, 2900
//   16.4 / 19.7; bf16 1900 15.6 / 18.4; Q8 2900 16.6 / 21.8; D 64 f16 2900 10.1 / 18.9
// fewer than 8 items, to which clusters give 8 blocks each and the deal all SMs, so
// their number bounds the tokens too (number: tokens; f16 where not named):
//   1: 4000 9.5 / 10.1, 6000 10.9 / 10.2, 8000 12.6 / 11.1, 12700 17.1 / 12.4
//   2: 6000 11.1 / 10.6, 12700 17.2 / 13.5; 4: 8000 12.7 / 12.9, 12700 17.1 / 15.7
//   6: 10000 14.3 / 14.6, 12700 17.3 / 15.7
//   bf16 1: 3000 9.9 / 9.3, 6000 12.8 / 10.5; 4: 4000 10.9 / 11.1, 6000 13.0 / 11.9
//   Q8 1: 6000 11.1 / 11.0, 10000 14.9 / 12.2
//   D 64 f16 1: 10000 8.9 / 8.7, 18000 11.8 / 10.0; 4: 18000 11.9 / 12.7; Q8 1: 8000
//     8.9 / 9.4, 10000 10.3 / 9.8 (its bound is near enough as it is)
// One sequence full, the others 100: B 4 4000 12.6 / 14.1, B 16 1000 12.6 / 10.1: a
// long sequence among short ones loses at small C, and more so beyond that room.
int cluster_size(long items, bool alone, int type, int D, long prefix, long room) {
  const long C = items <= 14   ? 8
                 : items <= 22 ? 6
                 : items <= 27 ? 5
                 : items <= 34 ? 4
                 : items <= 44 ? 3
                 : items <= 74 ? 2
                 : items <= 150 ? 1
                                : 0;
  const bool half = D == 64 && type != LK_KV_Q8;  // half the time a token; Q8's is not the bytes'
  const long few = items >= 8 || (D == 64 && type == LK_KV_Q8) ? 14 : items + 6;  // 14ths
  const long most = (type == LK_KV_BF16 ? 1024 : type == LK_KV_Q8 ? 1400 : 1600) * (half ? 2 : 1) * C * few / 14;
  return room + prefix <= most && (alone || room <= (half ? 1536 : 1024) * C) ? (int)C : 0;
}

// Up to as many keys bf16's weights have a third term too.
constexpr long kFineKeys = 4096;

struct Plan {
  long slots, tslots[2];  // streaming partials; tile partials of sequences, prefix
  int tsr[2];             // rows of a tile slot
  int C;                  // blocks of a cluster, 0: no clusters
};

// type < 0: the most that any call of the sizes takes.
Plan plan(int n_q, int n_kv, int B, int R, int type, int D, long prefix, long room) {
  const long G = n_q / n_kv, rows[2] = {R * G, (long)B * R * G}, many[2] = {(long)B * n_kv, prefix ? n_kv : 0};
  Plan p = {};
  if (type >= 0) p.C = cluster_size(many[0] * ((rows[0] + TR - 1) / TR), B == 1, type, D, prefix, room);
  p.slots = (long)kMaxWorkers * kMaxWarps;
  for (int x = 0; x < 2; ++x) {
    p.slots += many[x] * ((rows[x] + TR - 1) / TR);
    if (!many[x] || p.C || !(type < 0 ? rows[x] > 16 : tiled(rows[x], type, D, x ? prefix : -1))) continue;
    p.tsr[x] = tile_slot_rows(rows[x]);
    p.tslots[x] = kTileWorkers + many[x] * ((rows[x] + 127) / 128);  // items of 128 rows or of 256
  }
  return p;
}

size_t up256(size_t n) { return (n + 255) / 256 * 256; }

// Byte offsets of the workspace's parts; returns its size.
size_t layout(const Plan& p, int D, size_t (&ml)[3], size_t (&o)[3]) {
  size_t at = 0;
  for (int x = 0; x < 3; ++x) {
    const size_t rows = x == 0 ? (size_t)p.slots * TR : (size_t)p.tslots[x - 1] * p.tsr[x - 1];
    ml[x] = at;
    at += up256(rows * 8);
    o[x] = at;
    at += up256(rows * D * 4);
  }
  return at;
}

lk_status make_maps(AttnArgs& a, int type, int D, int box) {
  typedef CUresult (*encode_fn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
  static std::atomic<encode_fn> known;
  encode_fn encode = known.load(std::memory_order_acquire);
  if (!encode) {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &r) != cudaSuccess ||
        r != cudaDriverEntryPointSuccess || !f) {
      cudaGetLastError();
      return LK_ERR_CUDA;
    }
    encode = (encode_fn)f;
    known.store(encode, std::memory_order_release);
  }
  const int eb = type == LK_KV_Q8 ? 1 : 2, row = D * eb < 128 ? D * eb : 128;
  const cuuint64_t dim[2] = {(cuuint64_t)D, ((cuuint64_t)a.n_pages * a.n_kv) << a.page_log2};
  const cuuint64_t pitch[1] = {(cuuint64_t)D * eb};
  const cuuint32_t shape[2] = {(cuuint32_t)(row / eb), (cuuint32_t)box}, step[2] = {1, 1};
  for (int x = 0; x < 2; ++x)
    if (encode(x ? &a.vmap : &a.kmap, eb == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_UINT16, 2,
               const_cast<void*>(x ? a.v : a.k), dim, pitch, shape, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
               row == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return LK_ERR_CUDA;
  a.box = box;
  return LK_OK;
}

template <int TYPE, int D, bool FINE>
lk_status run_type(const AttnArgs& a, int pdl, cudaStream_t stream) {
  static std::atomic<int> done[kMaxDevices];
  typedef Cfg<TYPE, D> C;
  if (!prepare_kernel(attn_kernel<TYPE, D, FINE>, done, C::RING)) return LK_ERR_CUDA;
  return launch(attn_kernel<TYPE, D, FINE>, dim3(a.W), dim3(32 * C::NW), C::RING, pdl, stream, a) == cudaSuccess
             ? LK_OK
             : LK_ERR_CUDA;
}

template <int TYPE, int D>
lk_status run_cluster(const JoinArgs& j, int pdl, cudaStream_t stream) {
  static std::atomic<int> done[kMaxDevices];
  typedef Cfg<TYPE, D> C;
  if (!prepare_kernel(attn_cluster_kernel<TYPE, D>, done, C::RING)) return LK_ERR_CUDA;
  const int items = j.a.B * j.a.n_kv * (int)((j.a.R * j.a.G + TR - 1) / TR);
  return launch(attn_cluster_kernel<TYPE, D>, dim3(items * j.a.C), dim3(32 * C::NW), C::RING, pdl, stream, j, j.a.C) ==
                 cudaSuccess
             ? LK_OK
             : LK_ERR_CUDA;
}

template <int Q, int D>
lk_status run_join(const JoinArgs& j, cudaStream_t stream) {
  static std::atomic<int> done[kMaxDevices];
  if (!prepare_kernel(attn_join_kernel<Q, D>, done, 0)) return LK_ERR_CUDA;
  const long heads = (long)j.a.B * j.a.R * j.a.n_q;
  return launch(attn_join_kernel<Q, D>, dim3((unsigned)((heads + 3) / 4)), dim3(128), 0, 1, stream, j) == cudaSuccess
             ? LK_OK
             : LK_ERR_CUDA;
}

template <int D>
lk_status run_d(JoinArgs& j, int type, lk_mode mode, int pdl, cudaStream_t stream) {
  AttnArgs& a = j.a;
  lk_status st = LK_OK;
  a.NW = type == LK_KV_Q8 ? Cfg<LK_KV_Q8, D>::NW : Cfg<LK_KV_F16, D>::NW;
  const int page = 1 << a.page_log2;
  if (a.C) {
    if ((st = make_maps(a, type, D, page < UNIT ? page : UNIT))) return st;
    return type == LK_KV_F16    ? run_cluster<LK_KV_F16, D>(j, pdl, stream)
           : type == LK_KV_BF16 ? run_cluster<LK_KV_BF16, D>(j, pdl, stream)
                                : run_cluster<LK_KV_Q8, D>(j, pdl, stream);
  }
  // the launches after the first are dependents of the one before
  if (!a.own_tiled || (a.shared && !a.pre_tiled)) {
    if ((st = make_maps(a, type, D, page < UNIT ? page : UNIT))) return st;
    // (beside the tile kernel's partials, which have two, it would be lost)
    const bool fine = !a.own_tiled && !a.pre_tiled && (long)a.table_w << a.page_log2 <= kFineKeys && a.plen <= kFineKeys;
    st = type == LK_KV_F16  ? run_type<LK_KV_F16, D, false>(a, pdl, stream)
         : type == LK_KV_Q8 ? run_type<LK_KV_Q8, D, false>(a, pdl, stream)
         : fine             ? run_type<LK_KV_BF16, D, true>(a, pdl, stream)
                            : run_type<LK_KV_BF16, D, false>(a, pdl, stream);
    pdl = 1;
  }
  if (!st && (a.own_tiled || a.pre_tiled)) {
    const int part = D == 128 ? 128 : 64;  // tokens that a warp of the tile kernel fetches
    if (type != LK_KV_Q8 && (st = make_maps(a, type, D, page < part ? page : part))) return st;
    st = launch_tiles(a, type, D, pdl, stream);
  }
  if (st) return st;
  return mode == LK_DEQUANT   ? run_join<0, D>(j, stream)
         : mode == LK_INT8ACT ? run_join<1, D>(j, stream)
                              : run_join<2, D>(j, stream);
}

}  // namespace lkattn

using namespace lkattn;

extern "C" {

size_t lk_attn_workspace_bytes(int n_q, int n_kv, int head_dim, int B, int R, int shared) {
  if ((head_dim != 64 && head_dim != 128) || n_kv < 1 || n_q < n_kv || n_q % n_kv || n_q > 4096) return 0;
  if (B < 0 || R < 0 || B > LK_MAX_BATCH || R > LK_MAX_BATCH || B * R > LK_MAX_BATCH) return 0;
  size_t ml[3], o[3];
  return layout(plan(n_q, n_kv, B, R, -1, head_dim, shared != 0, 0), head_dim, ml, o);
}

int lk_attn_launches(int type, int n_q, int n_kv, int head_dim, int B, int R, int prefix_len, int room) {
  if (type < LK_KV_F16 || type > LK_KV_Q8 || prefix_len < 0 || room < 0 || !lk_attn_workspace_bytes(n_q, n_kv, head_dim, B, R, 0)) return 0;
  if (B == 0 || R == 0) return 0;
  const Plan p = plan(n_q, n_kv, B, R, type, head_dim, prefix_len, room);
  const bool tile = p.tslots[0] || p.tslots[1], stream = !p.tslots[0] || (prefix_len && !p.tslots[1]);
  return p.C ? 1 : 1 + tile + stream;
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
  // units of 32 keys, all items' together, are 32-bit numbers
  const long cap_units = ((long)table_w * cache->page + UNIT - 1) / UNIT, pre_units = ((long)prefix_len + UNIT - 1) / UNIT;
  const long G = n_q / cache->n_kv;
  if (cache->n_kv * (B * ((R * G + TR - 1) / TR) * cap_units + (B * R * G + TR - 1) / TR * pre_units) > 0x7fffffffL)
    return LK_ERR_SHAPE;
  if (!ws || ws_bytes < lk_attn_workspace_bytes(n_q, cache->n_kv, cache->head_dim, B, R, shared))
    return LK_ERR_WORKSPACE;
  if (!aligned(ws, 16)) return LK_ERR_ALIGN;
  // what is written apart from all else that is given (out in place of q excepted:
  // a row's head is written by those that read it, when they have)
  const size_t rows = (size_t)B * R * n_q * cache->head_dim, tokens = (size_t)cache->n_pages * cache->n_kv * cache->page;
  const size_t kv = tokens * cache->head_dim * (cache->type == LK_KV_Q8 ? 1 : 2), sc = tokens * (cache->head_dim / 32) * 2;
  const bool words = mode != LK_DEQUANT, q8 = cache->type == LK_KV_Q8;
  const Span spans[] = {{out, rows * 4},
                        {words ? hq : nullptr, rows},
                        {mode == LK_TWOPASS ? hl : nullptr, rows},
                        {words ? hs : nullptr, rows / 8},
                        {ws, lk_attn_workspace_bytes(n_q, cache->n_kv, cache->head_dim, B, R, shared)},
                        {out == q ? nullptr : q, rows * 4},
                        {cache->k, kv},
                        {cache->v, kv},
                        {q8 ? cache->ks : nullptr, sc},
                        {q8 ? cache->vs : nullptr, sc},
                        {table, (size_t)B * table_w * 4},
                        {lens, (size_t)B * 4},
                        {shared ? prefix_table : nullptr, (size_t)prefix_w * 4}};
  if (spans_clash(spans, 5, sizeof spans / sizeof *spans)) return LK_ERR_ARG;
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
  a.shared = shared;
  a.qscale = scale * 1.44269504088896340736f;
  const Plan p = plan(n_q, cache->n_kv, B, R, cache->type, cache->head_dim, prefix_len, (long)table_w * cache->page);
  size_t ml[3], o[3];
  layout(p, cache->head_dim, ml, o);
  a.own_tiled = p.tslots[0] > 0;
  a.pre_tiled = p.tslots[1] > 0;
  a.C = p.C;
  a.ml = (float*)((char*)ws + ml[0]);
  a.o = (float*)((char*)ws + o[0]);
  for (int x = 0; x < 2; ++x) {
    a.tml[x] = (float*)((char*)ws + ml[x + 1]);
    a.to[x] = (float*)((char*)ws + o[x + 1]);
  }
  a.tunit_log2 = cache->type == LK_KV_Q8 ? 6 : 7;
  a.trows_log2 = cache->type == LK_KV_Q8 ? 7 : 8;
  a.tflip = cache->type != LK_KV_Q8;
  a.W = d->sm_count < kMaxWorkers ? d->sm_count : kMaxWorkers;
  a.TW = d->sm_count < kTileWorkers ? d->sm_count : kTileWorkers;
  a.wait_ns = opt_wait_us > 0 ? (unsigned long long)opt_wait_us * 1000ull : 2000000000ull;
  a.err = error_word_ptr();
  if (!a.err) return LK_ERR_CUDA;
  JoinArgs j;
  j.a = a;
  j.out = out;
  j.wide = aligned(out, 16);
  j.hq = hq;
  j.hl = mode == LK_TWOPASS ? hl : nullptr;
  j.hs = hs;
  j.mode = mode;
  const int pdl = cfg_pdl(cfg);
  return cache->head_dim == 128 ? run_d<128>(j, cache->type, mode, pdl, stream)
                                : run_d<64>(j, cache->type, mode, pdl, stream);
}

lk_status lk_attn(const lk_kv_cache* cache, const float* q, int n_q, const int32_t* table, int table_w,
                  const int32_t* lens, int B, int R, float scale, lk_mode mode, float* out, int8_t* hq, int8_t* hl,
                  float* hs, void* ws, size_t ws_bytes, const lk_launch_cfg* cfg, cudaStream_t stream) {
  return lk_attn_shared(cache, q, n_q, nullptr, 0, 0, table, table_w, lens, B, R, scale, mode, out, hq, hl, hs, ws,
                        ws_bytes, cfg, stream);
}

}  // extern "C"
