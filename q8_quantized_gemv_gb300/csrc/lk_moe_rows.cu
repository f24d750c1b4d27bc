// The experts' products for several rows in the quantized modes (include/lk_moe.h),
// on the tensor cores.
//
// Rows that chose the same expert share the read of its weights.  Every block
// sorts the pairs by expert (the same sort in all of them: it takes about a
// microsecond, nothing is handed on) into bundles of one expert's up to 8 pairs
// (TwoPass 4), and takes its share of all bundles' weight rows, the same rows of an expert's
// bundles one after the other: an expert's weights come from HBM once, for more bundles again
// from L2 (bundle after bundle TwoPass took 262 us for 64 rows gate/up of 128 experts, so 234).  A tile is 16 weight
// rows x 8 columns, a column a pair's words (TwoPass: neighbouring columns its high and low
// words, which the same lane then has the dots of); a warp streams its tiles through its
// own shared-memory stages, each one slice of K of the 16 rows and of the bundle's activation
// rows, by the lanes' own asynchronous copies: a bulk copy a row goes out one lane at a
// time, about 20 cycles each, and 24 of them were a good part of a stage's time (64 rows down
// 145 us against 128).  Slices are as large as 16 warps have room for: halves of it, two
// stages a warp, took 159 us.
// Each row is 16 bytes longer than its slice, which keeps ldmatrix's eight rows in
// different banks.  A 32-block is one mma m16n8k32 of int8
// levels with the exact dots as result, combined in f32 as every other kernel
// of the library does (partial b mod 4 ascending, (p0 + p2) + (p1 + p3)):
// the products have lk_gemv_q8's bits.
//
// Gate/up: a tile is 8 gate rows over the 8 up rows of the same outputs, so a lane has
// both values of an output.  Words: groups of 32 outputs, finished by the block that
// has them whole, or by the last of its blocks to count in.
//
// Down: a block has a range of output rows and streams it from every expert;
// its products stay in shared memory until all of a row's pairs are there, then
// are added in the order of the pairs.
//
// Bound: HBM for few pairs an expert.  The int8 MMA takes 16 cycles of an SM's
// tensor pipe, 70 % of it at the copy bandwidth.
#include "lk_moe.cuh"

using namespace lk;
using namespace lkh;
using namespace lkring;

namespace lkmoe {

namespace {

constexpr int TR = 16;        // weight rows of a tile
constexpr int TC = 8;         // columns of a tile: activation rows of a stage
constexpr int NW = 16;        // warps of a block at most
constexpr int DEPTH = 2;      // stages of a warp at most
constexpr int STATIC = 1024;  // static shared memory, at most
constexpr int ROOM_D = 65536; // bytes of products that a block keeps, about

struct RowsArgs {
  MoeArgs a;
  int M, P;                        // rows, pairs M * k
  unsigned rs, srs, ars, xsr;      // stage: bytes of a level, scale, activation and activation-scale row
  unsigned x_off, xs_off;
  unsigned o_ids, o_rank, o_order, o_cnt, o_off, o_bundle, o_d, o_ring;  // offsets in shared memory
  int rows_d;                      // down: output rows of a pass
  int nw;                          // warps
};

__device__ __forceinline__ void ldmatrix4(unsigned (&r)[4], unsigned addr) {
  // (volatile: in order with the waits and the copies; no other memory is concerned)
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
// d = A (16 x 32) * B (32 x 8) + 0x4B400000: as a float, 1.5 * 2^23 + the dot (|dot| < 2^20)
__device__ __forceinline__ void dot_bits(int (&d)[4], const unsigned (&w)[4], unsigned b0, unsigned b1) {
  constexpr int base = 0x4B400000;
  asm("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=r"(d[0]), "=r"(d[1]), "=r"(d[2]), "=r"(d[3])
      : "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(b0), "r"(b1), "r"(base));
}
__device__ __forceinline__ float dot_of(int bits) { return __fadd_rn(__int_as_float(bits), -12582912.0f); }

// A bundle: expert, its first place in the sorted pairs, pairs.
__device__ __forceinline__ unsigned bundle_of(int e, int start, int n) {
  return (unsigned)e | (unsigned)start << 10 | (unsigned)(n - 1) << 21;
}

template <int Q, bool GLU>
__global__ void __launch_bounds__(NW * 32, 1) moe_rows_kernel(const RowsArgs ra) {
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ unsigned long long bars[NW * DEPTH];
  __shared__ int totals[2][NW];
  __shared__ int aborted, n_bundles;
  constexpr int TP = TC / Q;  // pairs of a bundle
  const MoeArgs& a = ra.a;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = ra.nw;
  const int g = lane >> 2, t4 = lane & 3;
  volatile int* abort_flag = &aborted;
  short* ids = (short*)(smem + ra.o_ids);
  unsigned short* rank = (unsigned short*)(smem + ra.o_rank);
  unsigned short* order = (unsigned short*)(smem + ra.o_order);
  const unsigned short* from = GLU ? rank : order;  // later: the activation row of order's pairs
  unsigned short* cnt = (unsigned short*)(smem + ra.o_cnt);
  unsigned short* off = (unsigned short*)(smem + ra.o_off);  // first place, first bundle of an expert
  unsigned* bundle = (unsigned*)(smem + ra.o_bundle);
  float* dd = (float*)(smem + ra.o_d);
  unsigned char* ring = smem + ra.o_ring + (size_t)warp * a.depth * a.stage_bytes;
  const unsigned full0 = smem_u32(bars + warp * DEPTH);
  if (lane == 0)
    for (int s = 0; s < a.depth; ++s) mbar_init(full0 + 8 * s, 32);
  for (int e = threadIdx.x; e < a.E; e += blockDim.x) cnt[e] = 0;
  if (threadIdx.x == 0) {
    aborted = 0;
    asm volatile("griddepcontrol.launch_dependents;" :::);
  }
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  griddep_wait();
  for (int p = threadIdx.x; p < ra.P; p += blockDim.x) {
    const int e = __ldcg(a.ids + p);
    ids[p] = (unsigned)e < (unsigned)a.E ? (short)e : (short)-1;
  }
  __syncthreads();

  // ---- the pairs by expert: how many of its expert come before each (one warp) ----
  if (warp == 0) {
    for (int p0 = 0; p0 < ra.P; p0 += 32) {
      const int e = p0 + lane < ra.P ? ids[p0 + lane] : -1;
      const unsigned same = __match_any_sync(FULL, e);
      const int before = __popc(same & ((1u << lane) - 1u));
      int base = 0;
      if (e >= 0) {
        base = cnt[e];
        rank[p0 + lane] = (unsigned short)(base + before);
      }
      __syncwarp();
      if (e >= 0 && before == 0) cnt[e] = (unsigned short)(base + __popc(same));
      __syncwarp();
    }
  }
  __syncthreads();
  // first places and bundles: sums over the experts before (a thread has neighbours)
  {
    const int per = (a.E + nw * 32 - 1) / (nw * 32), e0 = min(a.E, (int)threadIdx.x * per), e1 = min(a.E, e0 + per);
    int n = 0, b = 0;
    for (int e = e0; e < e1; ++e) {
      n += cnt[e];
      b += (cnt[e] + TP - 1) / TP;
    }
    int in = n, ib = b;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int yn = __shfl_up_sync(FULL, in, o), yb = __shfl_up_sync(FULL, ib, o);
      if (lane >= o) {
        in += yn;
        ib += yb;
      }
    }
    if (lane == 31) {
      totals[0][warp] = in;
      totals[1][warp] = ib;
    }
    __syncthreads();
    int bn = in - n, bb = ib - b;
    for (int w = 0; w < nw; ++w) {
      if (w < warp) {
        bn += totals[0][w];
        bb += totals[1][w];
      }
      if (threadIdx.x == 0) n_bundles = (w ? n_bundles : 0) + totals[1][w];
    }
    for (int e = e0; e < e1; ++e) {
      off[e] = (unsigned short)bn;
      for (int i = 0; i < cnt[e]; i += TP) bundle[bb++] = bundle_of(e, bn + i, min(TP, cnt[e] - i));
      bn += cnt[e];
    }
  }
  __syncthreads();
  for (int p = threadIdx.x; p < ra.P; p += blockDim.x)
    if (ids[p] >= 0) order[off[ids[p]] + rank[p]] = (unsigned short)p;
  __syncthreads();
  if (GLU) {
    for (int i = threadIdx.x; i < ra.P; i += blockDim.x) rank[i] = (unsigned short)(order[i] / a.k);
    __syncthreads();
  }
  const int nbu = n_bundles;

  const int nb = a.K >> 5, odd = (nb >> 2) & 1;  // odd: rows of scales begin at 8 bytes in turn
  const int G = gridDim.x;
  // this block's output rows (down), in passes; its tiles (gate/up)
  const int per = a.rows / 8;  // gate/up: tiles of a bundle
  const int r_lo = GLU ? 0 : (int)((long)a.rows * blockIdx.x / G), r_hi = GLU ? 0 : (int)((long)a.rows * (blockIdx.x + 1) / G);
  const int t_lo = GLU ? (int)((long)nbu * per * blockIdx.x / G) : 0;
  const int t_hi = GLU ? (int)((long)nbu * per * (blockIdx.x + 1) / G) : 0;
  // Gate/up: tiles (and groups of four, for the words) go expert by expert, of an expert by its
  // rows, the same rows of its bundles one after the other: they come from HBM once.
  struct Place {
    int first, n;  // the expert's first bundle, its bundles
    int step, v;   // its rows' tile (group), bundle
  };
  auto place_of = [&](int i, int each) {
    Place s;
    const int v0 = i / each;
    const unsigned bu = bundle[v0];
    const int e = bu & 1023;
    s.n = (cnt[e] + TP - 1) / TP;
    s.first = v0 - ((int)((bu >> 10) & 2047) - off[e]) / TP;
    const int r = i - s.first * each;
    s.step = s.n == 1 ? r : r / s.n;
    s.v = s.first + r - s.step * s.n;
    return s;
  };
  const unsigned a_row = (lane & 15) * ra.rs + (lane >> 4) * 16;
  const unsigned b_row = (lane & 7) * ra.ars + (lane >> 3) * 16;
  int slot = 0;
  unsigned phase = 0;
  bool ok = true;

  for (int r0 = r_lo; GLU ? r0 == 0 : r0 < r_hi; r0 += GLU ? 1 : ra.rows_d) {
    const int rn = GLU ? 0 : min(ra.rows_d, r_hi - r0);  // down: rows of this pass
    const int rt = GLU ? per : (rn + TR - 1) / TR;
    const int lo = GLU ? t_lo : 0, hi = GLU ? t_hi : nbu * rt;
    struct Cursor {
      int tile, c;  // gate/up: tile, down: bundle; slice
      int w;        // the tile's rows
      unsigned bu;  // its bundle
    };
    const int dv = nw / rt, dw = nw - dv * rt;
    auto place = [&](Cursor& s) {
      const Place at = place_of(s.tile, per);
      s.w = at.step;
      s.bu = bundle[at.v];
    };
    auto next = [&](Cursor& s) {  // (no divisions but a gate/up tile's)
      if (++s.c < a.nsl) return;
      s.c = 0;
      if (GLU) {
        s.tile += nw;
        if (s.tile < hi) place(s);
      } else {
        s.tile += dv;
        s.w += dw;
        if (s.w >= rt) {
          s.w -= rt;
          ++s.tile;
        }
        if (s.tile < nbu) s.bu = bundle[s.tile];
      }
    };
    auto issue = [&](const Cursor& s, int to) {
      const int e = s.bu & 1023, start = (s.bu >> 10) & 2047, n = (int)(s.bu >> 21) + 1;
      const int k0 = s.c * a.tk, len = a.K - k0 < a.tk ? a.K - k0 : a.tk;
      const unsigned bar = full0 + 8 * to;
      unsigned char* st = ring + (size_t)to * a.stage_bytes;
      const int rows = GLU ? TR : min(TR, rn - TR * s.w);
      const long row0 = (long)e * a.rows + (GLU ? 8 * s.w : r0 + TR * s.w);
      auto stack_row = [&](int i) { return row0 + (GLU ? i & 7 : i); };
      if (16 * lane < len) {
        unsigned char* to_w = st + 16 * lane;
        const int8_t* w = a.wa + row0 * a.K + k0 + 16 * lane;
        if (GLU) {
          const int8_t* u = a.wb + row0 * a.K + k0 + 16 * lane;
#pragma unroll
          for (int i = 0; i < 8; ++i, w += a.K) copy16(to_w + i * ra.rs, w);
#pragma unroll
          for (int i = 8; i < TR; ++i, u += a.K) copy16(to_w + i * ra.rs, u);
        } else {
#pragma unroll
          for (int i = 0; i < TR; ++i, w += a.K)
            if (i < rows) copy16(to_w + i * ra.rs, w);
        }
#pragma unroll
        for (int x = 0; x < TC / Q; ++x) {
          if (x >= n) break;
          const long at = (long)from[start + x] * a.K + k0 + 16 * lane;
          copy16(to_w + ra.x_off + Q * x * ra.ars, a.xq + at);
          if (Q == 2) copy16(to_w + ra.x_off + (Q * x + 1) * ra.ars, a.xl + at);
        }
      }
      // scales: 2 bytes a block of a weight row, 16 or (where rows begin at 8) 8 at a time,
      // and 4 bytes a block of an activation row
      auto scale16 = [&](int i, int at) {
        copy16(st + a.s_off + i * ra.srs + at, (GLU && i >= 8 ? a.sb : a.sa) + (stack_row(i) * nb + (k0 >> 5)) * 2 + at);
      };
      auto act_scale = [&](int x, int at) {
        copy16(st + ra.xs_off + x * ra.xsr + 4 * at, a.xs + (long)from[start + x] * nb + (k0 >> 5) + at);
      };
      if (len == 512 && !odd) {
        if (lane >> 1 < rows) scale16(lane >> 1, 16 * (lane & 1));
        if (lane >> 2 < n) act_scale(lane >> 2, 4 * (lane & 3));
      } else {
        const int per_row = len / 128, half = per_row / 2;
        if (!odd && len % 256 == 0) {
          for (int c = lane; c < rows * half; c += 32) scale16(c / half, 16 * (c % half));
        } else {
          for (int c = lane; c < rows * per_row; c += 32) {
            const int i = c / per_row, at = 8 * (c - i * per_row);
            copy8(st + a.s_off + i * ra.srs + at, (GLU && i >= 8 ? a.sb : a.sa) + (stack_row(i) * nb + (k0 >> 5)) * 2 + at);
          }
        }
        for (int c = lane; c < n * per_row; c += 32) act_scale(c / per_row, 4 * (c % per_row));
      }
      arrive_with_copies(bar);
      __syncwarp();
    };
    const int first = lo + warp;
    Cursor head{GLU ? first : first / rt, 0, first % rt, 0};
    if (first < hi) {
      if (GLU) place(head);
      else head.bu = bundle[head.tile];
    }
    Cursor at = head;
    const int total = ok && first < hi ? ((hi - 1 - first) / nw + 1) * a.nsl : 0;
    int issued = 0;
    for (int s = slot; issued < total && issued < a.depth; ++issued, next(head)) {
      issue(head, s);
      if (++s == a.depth) s = 0;
    }
    // partials of a lane's products: [partial][row g or g + 8][its pairs]: Int8Act pairs 2 t4 and
    // 2 t4 + 1, TwoPass pair t4
    constexpr int LP = Q == 1 ? 2 : 1;
    float p[4][2][LP];
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int c = 0; c < LP; ++c) p[q][e][c] = 0.f;
    int n = 0;
    for (; ok && n < total; ++n) {
      if (!__all_sync(FULL, mbar_wait(full0 + 8 * slot, phase, a.wait_ns, abort_flag))) {
        if (lane == 0) raise_error(a.err, ERR_MOE_WAIT, abort_flag);
        ok = false;
        break;
      }
      const int k0 = at.c * a.tk, len = a.K - k0 < a.tk ? a.K - k0 : a.tk;
      unsigned char* st = ring + (size_t)slot * a.stage_bytes;
      const unsigned W = smem_u32(st) + a_row, X = smem_u32(st + ra.x_off) + b_row;
      const unsigned char* S = st + a.s_off + g * ra.srs;
      const unsigned char* XS = st + ra.xs_off + LP * t4 * ra.xsr;
      const int groups = len >> 7;
      // two groups of four blocks at a time: their MMAs before the first combine
#pragma unroll 1
      for (int gi = 0; gi < groups; gi += 2) {
        int d[2][4][4];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          if (gi + u >= groups) break;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const unsigned at = 128 * (gi + u) + 64 * h;
            unsigned x[4], w0[4], w1[4];
            ldmatrix4(w0, W + at);
            ldmatrix4(w1, W + at + 32);
            ldmatrix4(x, X + at);
            dot_bits(d[u][2 * h], w0, x[0], x[1]);
            dot_bits(d[u][2 * h + 1], w1, x[2], x[3]);
          }
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          if (gi + u >= groups) break;
          const uint2 s0 = *(const uint2*)(S + 8 * (gi + u)), s8 = *(const uint2*)(S + 8 * ra.srs + 8 * (gi + u));
          const float2 wa0 = __half22float2(*(const __half2*)&s0.x), wa1 = __half22float2(*(const __half2*)&s0.y);
          const float2 wb0 = __half22float2(*(const __half2*)&s8.x), wb1 = __half22float2(*(const __half2*)&s8.y);
          const float ws[2][4] = {{wa0.x, wa0.y, wa1.x, wa1.y}, {wb0.x, wb0.y, wb1.x, wb1.y}};
          float xs[LP][4];
#pragma unroll
          for (int c = 0; c < LP; ++c) {
            const float4 v = *(const float4*)(XS + c * ra.xsr + 16 * (gi + u));
            xs[c][0] = v.x;
            xs[c][1] = v.y;
            xs[c][2] = v.z;
            xs[c][3] = v.w;
          }
#pragma unroll
          for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int* dq = d[u][q] + 2 * e;  // columns 2 t4, 2 t4 + 1 of row g + 8 e
              if constexpr (Q == 1) {
#pragma unroll
                for (int c = 0; c < 2; ++c)
                  p[q][e][c] = __fmaf_rn(__fmul_rn(ws[e][q], xs[c][q]), dot_of(dq[c]), p[q][e][c]);
              } else {
                const float v = __fmaf_rn(xs[0][q], dot_of(dq[0]), __fmul_rn(__fmul_rn(xs[0][q], 0.0078125f), dot_of(dq[1])));
                p[q][e][0] = __fmaf_rn(ws[e][q], v, p[q][e][0]);
              }
            }
        }
      }
      __syncwarp();
      if (issued < total) {
        issue(head, slot);
        next(head);
        ++issued;
      }
      if (at.c == a.nsl - 1) {
        const int w = at.w, start = (at.bu >> 10) & 2047, np = (int)(at.bu >> 21) + 1;
#pragma unroll
        for (int c = 0; c < LP; ++c) {
          float y[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            y[e] = __fadd_rn(__fadd_rn(p[0][e][c], p[2][e][c]), __fadd_rn(p[1][e][c], p[3][e][c]));
#pragma unroll
            for (int q = 0; q < 4; ++q) p[q][e][c] = 0.f;
          }
          if (LP * t4 + c >= np) continue;
          const long pair = order[start + LP * t4 + c];
          if (GLU) {
            a.out[pair * a.rows + 8 * w + g] = swiglu(y[0], y[1]);
          } else {
            float* to = dd + pair * ra.rows_d + TR * w + g;
            if (TR * w + g < rn) to[0] = y[0];
            if (TR * w + g + 8 < rn) to[8] = y[1];
          }
        }
      }
      next(at);
      if (++slot == a.depth) {
        slot = 0;
        phase ^= 1u;
      }
    }
    // copies in flight land before the block may end
    for (int m = n; m < issued; ++m) {
      if (lane == 0) drain_wait(full0 + 8 * slot, phase, a.wait_ns, a.err);
      __syncwarp();
      if (++slot == a.depth) {
        slot = 0;
        phase ^= 1u;
      }
    }
    if constexpr (!GLU) {
      __syncthreads();
      for (int i = threadIdx.x; i < ra.M * rn; i += blockDim.x) {
        const int t = i / rn, r = i - t * rn;
        float y = 0.f;
        for (int j = 0; j < a.k; ++j) {
          const int pr = t * a.k + j;
          if (ids[pr] >= 0) y = __fmaf_rn(__ldcg(a.weights + pr), dd[(size_t)pr * ra.rows_d + r], y);
        }
        a.out[(long)t * a.rows + r0 + r] = y;
      }
      __syncthreads();
    }
  }
  if constexpr (GLU) {
    if (!a.hq) return;
    __threadfence();  // this block's h before its counts
    __syncthreads();
    if (*abort_flag || t_hi <= t_lo) return;
    const int groups = a.rows / 32;  // of a pair
    // the expert's groups of the same rows as the first tile's, to those of the last one's
    const Place from_tile = place_of(t_lo, per), to_tile = place_of(t_hi - 1, per);
    const int x0 = from_tile.first * groups + from_tile.step / 4 * from_tile.n;
    const int x1 = to_tile.first * groups + (to_tile.step / 4 + 1) * to_tile.n;
    for (int x = x0 + warp; x < x1; x += nw) {
      const Place at = place_of(x, groups);
      const int gi = at.step, t0 = at.first * per + 4 * gi * at.n + at.v - at.first;  // its first tile of four
      int mine = 0;
      for (int i = 0; i < 4; ++i) mine += t0 + i * at.n >= t_lo && t0 + i * at.n < t_hi;
      if (mine == 0) continue;
      if (mine < 4) {
        int old = 0;
        if (lane == 0) old = atomicAdd(a.cnt + x, mine);
        old = __shfl_sync(FULL, old, 0);
        if (old + mine != 4) continue;  // another block finishes it
        if (lane == 0) a.cnt[x] = 0;
        __threadfence();  // the others' h after their counts
      }
      const int v = at.v;
      const unsigned bu = bundle[v];
      const int start = (bu >> 10) & 2047, np = (int)(bu >> 21) + 1;
      for (int c = 0; c < np; ++c) {
        const long pair = order[start + c];
        quant_lane<Q>(__ldcg(a.out + pair * a.rows + 32 * gi + lane), a.hq + pair * a.rows,
                      Q == 2 ? a.hl + pair * a.rows : nullptr, a.hs + pair * (a.rows >> 5), gi, lane);
      }
    }
  }
}

unsigned up16(unsigned n) { return (n + 15u) & ~15u; }

// The layout of shared memory; false where it does not fit.
bool fit_rows(RowsArgs& r, int Q, bool glu, int blocks, int smem_optin, int* smem) {
  MoeArgs& a = r.a;
  unsigned o = 0;
  auto take = [&](unsigned bytes) {
    const unsigned at = o;
    o = up16(o + bytes);
    return at;
  };
  r.o_ids = take(2u * r.P);
  r.o_rank = take(2u * r.P);
  r.o_order = take(2u * r.P);
  r.o_cnt = take(2u * a.E);
  r.o_off = take(2u * a.E);
  r.o_bundle = take(4u * r.P);
  r.rows_d = 0;
  if (!glu) {
    // rows of a pass: all of a block's where they fit, else a multiple of a tile's
    const int rows = (a.rows + blocks - 1) / blocks;
    const int most = ROOM_D / (4 * r.P);  // at least 8
    r.rows_d = rows <= most ? rows : most < TR ? most : most / TR * TR;
  }
  r.o_d = take(4u * r.P * r.rows_d);
  r.o_ring = (o + 127u) & ~127u;
  const int room = smem_optin - STATIC - (int)r.o_ring;
  // slices of 512 for as many warps as have room (two warps a scheduler left it waiting
  // for the MMAs; slices begin at multiples of 8 scales)
  r.nw = 0;
  for (int tk = 512; tk >= 256 && r.nw < 8; tk /= 2) {
    a.tk = tk < a.K ? tk : a.K;
    a.nsl = (a.K + a.tk - 1) / a.tk;
    r.rs = a.tk + 16u;
    r.srs = up16(a.tk / 16u + 8u);
    r.ars = a.tk + 16u;
    r.xsr = a.tk / 8u + 16u;
    a.s_off = TR * r.rs;
    r.x_off = a.s_off + TR * r.srs;
    r.xs_off = r.x_off + TC * r.ars;
    a.stage_bytes = (r.xs_off + TC * r.xsr + 127u) & ~127u;
    const int fits = room / (int)a.stage_bytes;
    r.nw = fits < NW ? fits : NW;
    a.depth = r.nw ? fits / r.nw : 0;
    if (a.depth > DEPTH) a.depth = DEPTH;
  }
  if (a.depth < 1) return false;
  *smem = (int)r.o_ring + r.nw * a.depth * (int)a.stage_bytes;
  return true;
}

template <int Q, bool GLU>
lk_status run(RowsArgs& r, const DeviceInfo* d, int pdl, cudaStream_t stream) {
  static std::atomic<int> done[kMaxDevices];
  int smem = 0;
  if (!fit_rows(r, Q, GLU, d->sm_count, d->smem_optin, &smem)) return LK_ERR_SHAPE;
  return launch_moe_kernel(moe_rows_kernel<Q, GLU>, done, dim3(d->sm_count), r.nw * 32, smem, d->smem_optin - STATIC, pdl,
                           stream, r);
}

}  // namespace

lk_status moe_rows(const MoeArgs& a, bool glu, int mode, int M, int pdl, cudaStream_t stream) {
  const DeviceInfo* d = device_info(nullptr);
  if (!d) return LK_ERR_CUDA;
  RowsArgs r = {};
  r.a = a;
  r.M = M;
  r.P = M * a.k;
  return glu ? (mode == 1 ? run<1, true>(r, d, pdl, stream) : run<2, true>(r, d, pdl, stream))
             : (mode == 1 ? run<1, false>(r, d, pdl, stream) : run<2, false>(r, d, pdl, stream));
}

}  // namespace lkmoe
