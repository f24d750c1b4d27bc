// Host checks and work partition shared by the attention step's kernels.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>

#include "lk_attn.h"
#include "lk_device.cuh"
#include "lk_host.h"

namespace lkattn {

// Bits of the device error word that a wait which ran out sets: the streaming
// kernel's (clusters included) and the tile kernel's (1 to 16 are the GEMV
// kernels', 32 the chain's barrier).
constexpr int ERR_ATTN_WAIT = 64, ERR_TILE_WAIT = 128;

inline int log2_of(int p) {
  int n = 0;
  while ((1 << n) < p) ++n;
  return n;
}

inline lk_status check_cache(const lk_kv_cache* c, int n_q) {
  if (!c) return LK_ERR_ARG;
  if (c->type < LK_KV_F16 || c->type > LK_KV_Q8) return LK_ERR_ARG;
  if (c->head_dim != 64 && c->head_dim != 128) return LK_ERR_SHAPE;
  if (c->page < 16 || c->page > 1024 || (c->page & (c->page - 1))) return LK_ERR_SHAPE;
  // rows of the cache are coordinates of a tensor map
  if ((long)c->n_pages * c->page > 0x7fffffffL / (c->n_kv > 0 ? c->n_kv : 1)) return LK_ERR_SHAPE;
  if (c->n_kv < 1 || c->n_pages < 1 || n_q < c->n_kv || n_q % c->n_kv || n_q > 4096) return LK_ERR_SHAPE;
  if (!c->k || !c->v || (c->type == LK_KV_Q8 && (!c->ks || !c->vs))) return LK_ERR_ARG;
  if (!lkh::aligned(c->k, 16) || !lkh::aligned(c->v, 16)) return LK_ERR_ALIGN;
  if (c->type == LK_KV_Q8 && (!lkh::aligned(c->ks, 16) || !lkh::aligned(c->vs, 16))) return LK_ERR_ALIGN;
  return LK_OK;
}

// B, R, table and lens (the pointers only where there are rows)
inline lk_status check_rows(const lk_kv_cache* c, const int32_t* table, int table_w, const int32_t* lens, int B,
                            int R) {
  if (B < 0 || R < 0 || B > LK_MAX_BATCH || R > LK_MAX_BATCH || B * R > LK_MAX_BATCH) return LK_ERR_SHAPE;
  if (table_w < 0 || (long)table_w * c->page > 0x40000000L) return LK_ERR_SHAPE;
  if (B == 0 || R == 0) return LK_OK;
  if (!lens || (table_w > 0 && !table)) return LK_ERR_ARG;
  if (!lkh::aligned(lens, 4) || (table && !lkh::aligned(table, 4))) return LK_ERR_ALIGN;
  return LK_OK;
}

// ---- the work of a call and its deal ---------------------------------------------------
// An item is one key/value head of one sequence (a shared prefix is one more,
// number B) with a group of the query rows that read it: row i of a head's
// R * G (prefix: B * R * G): token i / G, query head i % G.  The streaming
// kernel's items have up to 8 rows and their keys come in units of 32, the tile
// kernel's 256 rows (Q8: 128) and units of 128 (Q8: 64).  A sequence belongs to one of the two.
// All units of a kernel's items, in a fixed order, are dealt to its blocks in
// equal contiguous shares, whatever the lengths are, and a streaming block's
// share to its warps in the same way; the part of an item that a block (warp)
// has, a segment, leaves a partial result (running maximum, sum, weighted
// values) in the workspace, in slot block (warp) + item, which no other segment
// has; a last launch joins the partials of a row.  A streaming block whose
// whole share is one item's joins its warps' partials itself.
constexpr int UNIT = 32;           // keys of a unit, streaming kernel
constexpr int TR = 8;              // its query rows of an item
constexpr int kMaxWorkers = 192;   // blocks of the streaming launch, at most
constexpr int kMaxWarps = 12;      // and their warps
constexpr int kTileWorkers = 192;  // blocks of a tile launch, at most
constexpr int kMaxSeq = LK_MAX_BATCH + 1;

// Rows of a tile slot: of more than 128 query rows each has one partial, else
// the keys' tiles are halved between two streams with a partial of the rows each.
__host__ __device__ inline int tile_slot_rows(long rows) { return rows <= 128 ? 2 * (int)rows : 256; }

struct AttnArgs {
  CUtensorMap kmap, vmap;  // [pages * heads * page rows][D], boxes of 128 bytes (Q8, D 64: 64) by box rows
  int box;
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
  const int* ptable;  // prefix: page list, length
  int plen;
  int shared;
  float qscale;       // scale * log2(e)
  int own_tiled, pre_tiled;  // which kernel has the sequences, the prefix
  float* ml;          // streaming partials: [slot][TR][2] maximum and sum,
  float* o;           //   [slot][TR][D] weighted values
  float* tml[2];      // tile partials of the sequences, the prefix: [slot][slot rows][2],
  float* to[2];       //   [slot][slot rows][D], tflip: 16-byte pieces permuted in 128 bytes by row & 7
  int C;              // blocks of a cluster (attn_cluster_kernel), else 0
  int W, NW, TW;      // blocks and warps of the streaming launch, blocks of the tile launch
  int tunit_log2, trows_log2;  // keys of a unit, rows of an item of the tile kernel
  int tflip;          // whether its partials' pieces are permuted
  unsigned long long wait_ns;
  int* err;
};

// Sequence s has un[s] units per item (0 where the other kernel has it) and
// n[s] keys; units before it cum[s]; cum[nseq] is their total.  32 bits: the
// host refuses sizes whose units could pass them (64-bit quotients would be half
// the time of a short call).
struct Deal {
  int cum[kMaxSeq + 1];
  int un[kMaxSeq];
  int n[kMaxSeq];
};

__device__ __forceinline__ int rows_of(const AttnArgs& a, int s) { return (s == a.B ? a.B * a.R : a.R) * a.G; }
template <bool TILED>
__device__ __forceinline__ int groups_of(const AttnArgs& a, int s) {
  const int lg = TILED ? a.trows_log2 : 3;
  static_assert(TR == 8, "3 is its logarithm");
  return (rows_of(a, s) + (1 << lg) - 1) >> lg;
}
// Items before sequence s: of the streaming kernel in one row, of the tile
// kernel the prefix's apart.
template <bool TILED>
__device__ __forceinline__ int item0(const AttnArgs& a, int s) {
  if (TILED && s == a.B) return 0;
  return s * a.n_kv * groups_of<TILED>(a, 0);
}

// Units dealt to holders in contiguous shares: groups of G units to k holders
// each, the first G % k of them having one more.  One group of all units is the
// general deal; where all items are one sequence's, a group is an item, and no
// share has pieces of two (a second piece costs the tile kernel some 5 us).
// With k <= G no share is empty, so an item's segments are in consecutive holders.
// There are n holders; begin and size are theirs (behind the last one begin
// would be up to twice the units, which can pass 32 bits).
struct Shares {
  int G, k, n, base, more;
  __host__ __device__ __forceinline__ Shares(int G, int k, int groups = 1)
      : G(G), k(k), n(groups * k), base(G / k), more(G - base * k) {}
  __host__ __device__ __forceinline__ int begin(int c) const {
    const int i = c / k, j = c - i * k;
    return i * G + j * base + (j < more ? j : more);
  }
  __host__ __device__ __forceinline__ int size(int c) const { return base + (c % k < more ? 1 : 0); }
  __host__ __device__ __forceinline__ int holder(int u) const {
    const int i = u / G, r = u - i * G, first = more * (base + 1);
    return i * k + (r < first ? r / (base + 1) : more + (r - first) / base);
  }
};
// The deal of T units to at most W blocks, each with at least `least` units
// where there are enough; `one`: they are one sequence's, in `items` equal items.
// T is any number up to 2^31 - 1, but not 0.
__host__ __device__ __forceinline__ Shares deal_blocks(int T, int W, int least, bool one, int items) {
  const bool each = one && items <= W;
  const int G = each ? T / items : T, most = each ? W / items : W, full = (G - 1) / least + 1;
  return Shares(G, most < full ? most : full, each ? items : 1);
}
__device__ __forceinline__ Shares tile_blocks(const AttnArgs& a, int T) {
  const bool pre = !a.own_tiled;
  return deal_blocks(T, a.TW, 1, pre || (a.B == 1 && !a.pre_tiled), a.n_kv * groups_of<true>(a, pre ? a.B : 0));
}
// (a unit for each of a block's warps)
__device__ __forceinline__ Shares stream_blocks(const AttnArgs& a, int NW, int T) {
  return deal_blocks(T, a.W, NW, a.B == 1 && (a.pre_tiled || !a.shared) && !a.own_tiled, a.n_kv * groups_of<false>(a, 0));
}

// The lengths of sequences 2 l and 2 l + 1 in lane l.
__device__ __forceinline__ int2 lens_pair(const AttnArgs& a) {
  static_assert(LK_MAX_BATCH <= 64, "two sequences to a lane");
  const int s = 2 * (threadIdx.x & 31);
  return make_int2(s < a.B ? __ldcg(a.lens + s) : 0, s + 1 < a.B ? __ldcg(a.lens + s + 1) : 0);
}

// By one whole warp; the caller synchronizes.
template <bool TILED>
__device__ __forceinline__ void make_deal(const AttnArgs& a, Deal& d, int2 lens) {
  const int lane = threadIdx.x & 31, cap = a.table_w << a.page_log2, lu = TILED ? a.tunit_log2 : 5;
  static_assert(UNIT == 32, "5 is its logarithm");
  int n[2] = {lens.x, lens.y}, u[2];
  const bool own = (a.own_tiled != 0) == TILED, pre = (a.pre_tiled != 0) == TILED;
  const int items = a.n_kv * groups_of<TILED>(a, 0);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int s = 2 * lane + i;
    n[i] = min(max(n[i], 0), cap);
    const int un = own ? (n[i] + (1 << lu) - 1) >> lu : 0;
    if (s < a.B) d.n[s] = n[i], d.un[s] = un;
    u[i] = un * items;
  }
  int sum = u[0] + u[1];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int up = __shfl_up_sync(lk::FULL, sum, o);
    if (lane >= o) sum += up;
  }
  const int before = sum - u[0] - u[1];
  if (2 * lane < a.B) d.cum[2 * lane] = before;
  if (2 * lane + 1 < a.B) d.cum[2 * lane + 1] = before + u[0];
  if (lane == 31) {
    d.cum[a.B] = sum;
    if (a.shared) {
      const int un = pre ? (a.plen + (1 << lu) - 1) >> lu : 0;
      d.n[a.B] = a.plen;
      d.un[a.B] = un;
      d.cum[a.B + 1] = sum + un * a.n_kv * groups_of<TILED>(a, a.B);
    }
  }
}

// ---- instructions both kernels use ----------------------------------------------------
// (x, y) rounded to the 16-bit type, packed, and what the rounding left of them
template <bool BF>
__device__ __forceinline__ unsigned split2(float& x, float& y) {
  if constexpr (BF) {
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
// The rounded pair as two f32.
template <bool BF>
__device__ __forceinline__ lk::f32x2 widen2(unsigned h) {
  if constexpr (BF) return lk::f2_pack(__uint_as_float(h << 16), __uint_as_float(h & 0xffff0000u));
  const __half2 v = *(const __half2*)&h;
  return lk::f2_pack(__low2float(v), __high2float(v));
}
template <bool BF>
__device__ __forceinline__ unsigned round2(float x, float y) {
  if constexpr (BF) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    return *(const unsigned*)&h;
  }
  const __half2 h = __floats2half2_rn(x, y);
  return *(const unsigned*)&h;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
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
// Bytes of u = levels ^ 0x80 that the selector names as a pair of f16 levels: 1024 + u
// is exact in the low mantissa bits of 0x64xx, less 1152.
__device__ __forceinline__ unsigned level_pair(unsigned u, unsigned sel) {
  const unsigned b = __byte_perm(u, 0x64646464u, sel);
  const __half2 h = __hsub2(*(const __half2*)&b, __half2half2(__ushort_as_half(0x6480)));
  return *(const unsigned*)&h;
}
// log2 of what a row's largest weight is, sums and weighted values with it: the
// two kernels' partials are joined as they are.
__host__ __device__ constexpr float weight_shift(int type) {
  return type == LK_KV_BF16 ? 0.0f : type == LK_KV_Q8 ? 10.0f : 14.0f;
}
// Shift of a row's queries before f16 splitting: 2^10 / amax's power of two
// (returned), and its inverse for the scores.
__device__ __forceinline__ float row_shift(float amax, float& back) {
  const int e = min(max((int)(__float_as_uint(amax) >> 23), 27), 227) - 127;  // amax in [2^e, 2^(e+1))
  back = __uint_as_float((unsigned)(127 + e - 10) << 23);
  return __uint_as_float((unsigned)(127 - e + 10) << 23);
}

// ---- host -------------------------------------------------------------------------------
template <typename A>
cudaError_t launch(void (*f)(A), dim3 grid, dim3 block, int smem, int pdl, cudaStream_t stream, const A& args,
                   int cluster = 0) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  int n = 0;
  if (pdl) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n++].val.programmaticStreamSerializationAllowed = 1;
  }
  if (cluster) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = cluster;
    attr[n].val.clusterDim.y = attr[n].val.clusterDim.z = 1;
    ++n;
  }
  cfg.attrs = attr;
  cfg.numAttrs = n;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, f, args);
  if (e != cudaSuccess) cudaGetLastError();
  return e;
}

// Once per kernel and device: its dynamic shared memory (0: none) and the
// carveout of the GEMV kernels around it.
template <typename F>
bool prepare_kernel(F f, std::atomic<int> (&done)[lkh::kMaxDevices], int smem) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= lkh::kMaxDevices) return false;
  if (done[dev].load(std::memory_order_acquire)) return true;
  if (smem && cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) return false;
  if (cudaFuncSetAttribute(f, cudaFuncAttributePreferredSharedMemoryCarveout, (int)cudaSharedmemCarveoutMaxShared) !=
      cudaSuccess)
    return false;
  done[dev].store(1, std::memory_order_release);
  return true;
}

// Tensor maps of a's keys and values with boxes of `box` rows: 128-byte
// pieces of a row in the 128-byte swizzle (rows of 64 bytes: the 64-byte one).
lk_status make_maps(AttnArgs& a, int type, int D, int box);

// The tile kernel (lk_tile.cu): launched for the sequences that a marks as tiled.
lk_status launch_tiles(const AttnArgs& a, int type, int D, int pdl, cudaStream_t stream);

}  // namespace lkattn
