// The experts' products of a mixture-of-experts token (include/lk_moe.h):
// lk_moe_glu_q8, lk_moe_down_q8.
//
// Bound: the chosen experts' weights, read once from HBM.  Like the ring GEMV,
// a block has a share of rows, every warp streams its own groups of four rows
// ("quads") by bulk copies into its own shared-memory stages and refills a
// stage when it has consumed it; the activation stays in shared memory.  The
// rows' arithmetic is lk_gemv_q8's (8 lanes to a row, lane pair b mod 4 with
// block b's exact dot, (p0 + p2) + (p1 + p3)), so each product has its bits.
//
// Stages are few and large: a bulk copy goes out in about 20 cycles whatever its size, one
// lane at a time, and a warp takes as long again around each stage (gate/up of 8 rows, 4096 x 1024:
// slices of 512 170 us, 1024 107, 2048 85, whole rows 83).  So rows that are whole in a
// stage are one copy of neighbouring rows (gate/up two), up to four quads of short
// rows, and the scales come by the lanes' own asynchronous copies.
//
// Gate/up: a quad is the gate rows and the up rows of two neighbouring outputs
// of one pair, so the warp that has them has what the SwiGLU needs.  A row's
// pairs lie one after the other, and its blocks share their outputs evenly.  The
// words of h need 32 outputs: after its last quad a block quantizes the groups
// of 32 it has whole, and a group that it has in part if it is the last of its
// blocks to count in (cnt).
//
// Down: a block has a range of output rows for all pairs of the row of activations,
// a quad is four of them of one pair's expert.  The products stay in shared memory until
// all are there, then are added in the order of the pairs: no second launch.
#include "lk_moe.cuh"

using namespace lk;
using namespace lkh;
using namespace lkring;
using namespace lkmoe;

namespace {

constexpr int NW = 12;             // warps of a block
constexpr int SLICE = 4096;        // bytes of K in a stage at most
constexpr int DEPTH = 8;           // stages of a warp at most
constexpr int kStatic = 1536;      // static shared memory, at most

template <int Q>
__host__ __device__ constexpr unsigned act_bytes(unsigned len) {
  return Q == 0 ? 4u * len : len * Q + len / 8u;
}

// The activation rows of a block in shared memory, one after the other: words, low
// words and scales, or f32 values.  All threads load 16-byte runs; batch b is runs
// [b, b + 1) * RUNS * blockDim.x, so that the first can be under way while the first weights are
// asked for (behind those a load would wait for all of them).
template <int Q>
struct ActLoad {
  static constexpr int RUNS = 4;
  const MoeArgs& a;
  const int* row_of;  // the rows' numbers
  int rows, per;      // runs of a row
  uint4 v[RUNS];
  __device__ __forceinline__ ActLoad(const MoeArgs& args, const int* numbers, int n)
      : a(args), row_of(numbers), rows(n), per((int)(act_bytes<Q>(args.K) / 16)) {}
  __device__ __forceinline__ const void* source(int i) const {
    const int r = i / per, c = i - r * per;
    const long row = row_of[r];
    if constexpr (Q == 0) {
      return a.x + row * a.K + 4 * c;
    } else {
      const int w = a.K / 16;
      if (c < w) return a.xq + row * a.K + 16 * c;
      if (Q == 2 && c < 2 * w) return a.xl + row * a.K + 16 * (c - w);
      return a.xs + row * (a.K >> 5) + 4 * (c - Q * w);
    }
  }
  __device__ __forceinline__ void load(int b) {
#pragma unroll
    for (int u = 0; u < RUNS; ++u) {
      const int i = (b * RUNS + u) * blockDim.x + threadIdx.x;
      if (i < rows * per) v[u] = ld_cg16(source(i));
    }
  }
  __device__ __forceinline__ void store(int b, unsigned char* act) {
#pragma unroll
    for (int u = 0; u < RUNS; ++u) {
      const int i = (b * RUNS + u) * blockDim.x + threadIdx.x;
      if (i < rows * per) *(uint4*)(act + 16 * (size_t)place(i)) = v[u];
    }
  }
  // where run i goes: f32 values of a stretch of 256 so that the eight neighbours a lane
  // takes lie in two runs, each next to those of the lanes beside it
  __device__ __forceinline__ int place(int i) const {
    if constexpr (Q != 0) return i;
    const int r = i / per, c = i - r * per, j = c & 63;
    return c < (a.K >> 8) * 64 ? i - j + (j & 1) * 32 + (j >> 1) : i;
  }
  __device__ __forceinline__ bool more(int b) const { return b * RUNS * (int)blockDim.x < rows * per; }
};

// What a lane has of its item's four rows: under Dequant its part of each row, in packed
// halves, and for rows in several slices what rounding took off it; else partial (lane & 7) / 2
// of row lane / 8, in the even lanes.
template <int Q>
struct Partial {
  float p;
  __device__ __forceinline__ void clear() { p = 0.f; }
};
template <>
struct Partial<0> {
  f32x2 p[QR], rest[QR];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int r = 0; r < QR; ++r) p[r] = rest[r] = f2_pack(0.f, 0.f);
  }
};

// Four levels (u = their bytes ^ 0x80) as f32 pairs.
__device__ __forceinline__ void levels4(unsigned u, f32x2& w01, f32x2& w23) {
  const f32x2 neg = f2_pack(-8388736.0f, -8388736.0f);  // 2^23 + 128, as in i8_as_f32
  w01 = f2_add(f2_pack(i8_bits_f32(u, 0), i8_bits_f32(u, 1)), neg);
  w23 = f2_add(f2_pack(i8_bits_f32(u, 2), i8_bits_f32(u, 3)), neg);
}

// A stage's part of four rows against the activation at `act` (K its whole length); row r
// of the four is row base + (r & 1) + hop * (r >> 1) of the stage.
// Dequant: lane l has values 8l .. 8l + 7 of a stretch of 256, of one block, of all four rows
// (4l .. 4l + 3 of a last 128).  The stage's sums are f32, over 16 steps at most; what is
// rounded off when they are added to the item's is kept beside these (D. E. Knuth's two-sum), so a
// value passes 16 + 4 roundings, and 7 behind: within 2e-6 of sum |w x| whatever the number of slices
// (in f32 alone the chain was as long as the slices are many: 195 at most, 1.2e-5).
// (SLICED: rows in several slices.  The two-sum of rows in one took 2 %.)
template <int Q, bool SLICED>
__device__ __forceinline__ void quad_stage(Partial<Q>& p, const unsigned char* st, const MoeArgs& a, int k0, int len,
                                           int base, int hop, const unsigned char* act, int lane) {
  if constexpr (Q == 0) {
    const float* X = (const float*)act + k0 + 4 * lane;
    const unsigned char* S = st + a.s_off;
    f32x2 acc[QR];
#pragma unroll
    for (int r = 0; r < QR; ++r) acc[r] = f2_pack(0.f, 0.f);
    const int n = len >> 8;
#pragma unroll 2
    for (int s = 0; s < n; ++s) {
      const float4 xa = *(const float4*)(X + 256 * s), xb = *(const float4*)(X + 256 * s + 128);
#pragma unroll
      for (int r = 0; r < QR; ++r) {
        const int row = base + (r & 1) + hop * (r >> 1);
        const uint2 u = *(const uint2*)(st + row * a.ld + 256 * s + 8 * lane);
        const float ws = __half2float(*(const __half*)(S + row * a.srow + 16 * s + 2 * (lane >> 2)));
        f32x2 w0, w1, w2, w3;
        levels4(u.x ^ 0x80808080u, w0, w1);
        levels4(u.y ^ 0x80808080u, w2, w3);
        f32x2 d = f2_mul(w0, f2_pack(xa.x, xa.y));
        d = f2_fma(w1, f2_pack(xa.z, xa.w), d);
        d = f2_fma(w2, f2_pack(xb.x, xb.y), d);
        d = f2_fma(w3, f2_pack(xb.z, xb.w), d);
        acc[r] = f2_fma(f2_pack(ws, ws), d, acc[r]);
      }
    }
    if (len & 128) {
      const float4 xx = *(const float4*)(X + 256 * n);
#pragma unroll
      for (int r = 0; r < QR; ++r) {
        const int row = base + (r & 1) + hop * (r >> 1);
        const unsigned u = *(const unsigned*)(st + row * a.ld + 256 * n + 4 * lane);
        const float ws = __half2float(*(const __half*)(S + row * a.srow + 16 * n + 2 * (lane >> 3)));
        f32x2 w0, w1;
        levels4(u ^ 0x80808080u, w0, w1);
        const f32x2 d = f2_fma(w1, f2_pack(xx.z, xx.w), f2_mul(w0, f2_pack(xx.x, xx.y)));
        acc[r] = f2_fma(f2_pack(ws, ws), d, acc[r]);
      }
    }
#pragma unroll
    for (int r = 0; r < QR; ++r) {
      const f32x2 a0 = p.p[r], minus = f2_pack(-1.f, -1.f), sum = f2_add(a0, acc[r]);
      p.p[r] = sum;
      if constexpr (!SLICED) continue;
      auto less = [&](f32x2 x, f32x2 y) { return f2_fma(y, minus, x); };  // x - y
      const f32x2 b = less(sum, a0);
      p.rest[r] = f2_add(p.rest[r], f2_add(less(a0, less(sum, b)), less(acc[r], b)));
    }
  } else {
    const int nseg = len >> 7;
    const int rr = lane >> 3, j = lane & 7, q = j >> 1, row = base + (rr & 1) + hop * (rr >> 1);
    const unsigned char* W = st + row * a.ld + 16 * j;
    const unsigned char* S = st + a.s_off + row * a.srow + 2 * q;
    const unsigned char* XQ = act + k0 + 16 * j;
    const float* XS = (const float*)(act + (size_t)a.K * Q) + (k0 >> 5) + q;
#pragma unroll 8
    for (int seg = 0; seg < nseg; ++seg) {
      const int4 w = *(const int4*)(W + 128 * seg);
      const float ws = __half2float(*(const __half*)(S + 8 * seg));
      int d = dot16(w, *(const int4*)(XQ + 128 * seg));
      d += __shfl_xor_sync(FULL, d, 1);
      int e = 0;
      if constexpr (Q == 2) {
        e = dot16(w, *(const int4*)(XQ + a.K + 128 * seg));
        e += __shfl_xor_sync(FULL, e, 1);
      }
      p.p = q8_step<Q>(p.p, ws, XS[4 * seg], d, e);
    }
  }
}

// The product of each row r, in lane 8 r: Dequant the sum over the lanes, else
// (p0 + p2) + (p1 + p3).
template <int Q, bool SLICED>
__device__ __forceinline__ float row_sum(const Partial<Q>& p, int lane) {
  if constexpr (Q == 0) {
    float v[QR];
#pragma unroll
    for (int r = 0; r < QR; ++r) {
      float lo, hi;
      f2_unpack(p.p[r], lo, hi);
      v[r] = __fadd_rn(lo, hi);
    }
    if constexpr (SLICED) {
#pragma unroll
      for (int r = 0; r < QR; ++r) {
        float lo, hi;
        f2_unpack(p.rest[r], lo, hi);
        if (v[r] - v[r] == 0.f) v[r] = __fadd_rn(v[r], __fadd_rn(lo, hi));  // (not finite: it has no rest)
      }
    }
    // lanes 16 apart take two rows each, lanes 8 apart one of these
    const bool up = lane & 16, odd = lane & 8;
    const float a0 = __shfl_xor_sync(FULL, up ? v[0] : v[2], 16), a1 = __shfl_xor_sync(FULL, up ? v[1] : v[3], 16);
    const float k0 = __fadd_rn(up ? v[2] : v[0], a0), k1 = __fadd_rn(up ? v[3] : v[1], a1);
    float s = __fadd_rn(odd ? k1 : k0, __shfl_xor_sync(FULL, odd ? k0 : k1, 8));
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) s = __fadd_rn(s, __shfl_xor_sync(FULL, s, o));
    return s;
  } else {
    float v = p.p + __shfl_down_sync(FULL, p.p, 4);
    return v + __shfl_down_sync(FULL, v, 2);
  }
}

template <int Q, bool GLU, bool SLICED>
__global__ void __launch_bounds__(NW * 32, 1) moe_kernel(const MoeArgs a) {
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ unsigned long long bars[NW * DEPTH];
  __shared__ int pair_of[LK_MOE_MAX_K], expert_of[LK_MOE_MAX_K], row_of[LK_MOE_MAX_K];
  __shared__ float weight_of[LK_MOE_MAX_K];
  __shared__ int n_pairs;
  __shared__ int aborted;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long t = blockIdx.y;
  volatile int* abort_flag = &aborted;
  float* products = (float*)(smem + a.s_products);  // down: [pair][this block's rows]
  unsigned char* ring = smem + a.ring_off + (size_t)warp * a.depth * a.stage_bytes;
  const unsigned full0 = smem_u32(bars + warp * DEPTH);
  if (lane == 0)
    for (int s = 0; s < a.depth; ++s) mbar_init(full0 + 8 * s, 33);  // the bulk copies', and each lane's
  if (threadIdx.x == 0) {
    aborted = 0;
    asm volatile("griddepcontrol.launch_dependents;" :::);
  }
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  griddep_wait();

  // the row's pairs that are there
  if (warp == 0) {
    const int e = lane < a.k ? __ldcg(a.ids + t * a.k + lane) : -1;
    const unsigned there = __ballot_sync(FULL, (unsigned)e < (unsigned)a.E);
    if ((there >> lane) & 1u) {
      const int i = __popc(there & ((1u << lane) - 1u));
      pair_of[i] = lane;
      expert_of[i] = e;
      row_of[i] = (int)(GLU ? t : t * a.k + lane);
      if (!GLU) weight_of[i] = __ldcg(a.weights + t * a.k + lane);
    }
    if (lane == 0) n_pairs = __popc(there);
  }
  __syncthreads();
  const int np = n_pairs;
  ActLoad<Q> act(a, row_of, GLU ? np > 0 : np);
  act.load(0);

  // this block's quads: gate/up, of all pairs' outputs; down, of its rows of all pairs.  An
  // item is up to G of them side by side (gate/up: blocks begin at whole items)
  const int G = a.group;
  const int per = GLU ? a.rows / 2 : a.rows / 4;  // quads of a pair
  const int units = GLU ? np * per / G : per;
  const int q0 = (int)((long)units * blockIdx.x / gridDim.x) * (GLU ? G : 1);
  const int q1 = (int)((long)units * (blockIdx.x + 1) / gridDim.x) * (GLU ? G : 1);
  const int nq = q1 - q0, ipp = (nq + G - 1) / G, items = GLU ? ipp : ipp * np;
  struct Cursor {
    int c;         // slice
    int i, q, n;   // the item's pair (of those that are there), its first quad (gate/up: of the pair's; down:
                   // of the block's), its quads
  };
  const int whole = ipp * G, di = GLU || !ipp ? 0 : NW / ipp, dq = (NW - di * ipp) * G;
  auto next = [&](Cursor& s) {
    if (++s.c < a.nsl) return;
    s.c = 0;
    s.i += di;
    s.q += GLU ? NW * G : dq;
    if (s.q >= (GLU ? per : whole)) {  // (gate/up: a pair has at least 64 quads, a round at most 48)
      s.q -= GLU ? per : whole;
      ++s.i;
    }
    if (!GLU) s.n = min(G, nq - s.q);
  };
  const int nb = a.K >> 5;
  const int hop = GLU ? 2 * G : 2;               // (quad_stage; gate/up: up rows behind the gate rows)
  auto issue = [&](const Cursor& s, int slot) {
    const int k0 = s.c * a.tk, len = a.K - k0 < a.tk ? a.K - k0 : a.tk;
    const unsigned bar = full0 + 8 * slot;
    unsigned char* st = ring + (size_t)slot * a.stage_bytes;
    const int rows = 4 * s.n, half = 2 * s.n;  // of the stage; gate/up: of each matrix
    const long row0 = (long)expert_of[s.i] * a.rows + (GLU ? 2 * s.q : 4 * (q0 + s.q));
    if (lane == 0) mbar_arrive_expect_tx(bar, (unsigned)rows * len);
    __syncwarp();
    if (a.nsl == 1) {
      if (lane < (GLU ? 2 : 1))
        bulk_g2s_nohint(st + (size_t)lane * hop * a.ld, (lane ? a.wb : a.wa) + row0 * a.K, (GLU ? half : rows) * a.K, bar);
    } else if (lane < 4) {
      const bool up = GLU && lane >= 2;
      bulk_g2s_nohint(st + lane * a.ld, (up ? a.wb : a.wa) + (row0 + (up ? lane - 2 : lane)) * a.K + k0, len, bar);
    }
    // the scales, 2 bytes a block: a row has up to 256 bytes and begins at a multiple of 8
    if (8 * lane < len / 16) {
      const long at = 2 * (row0 * nb + (k0 >> 5)) + 8 * lane;
      unsigned char* to = st + a.s_off + 8 * lane;
#pragma unroll 1
      for (int i = 0; i < (GLU ? half : rows); i += 2) {
        copy8(to + i * a.srow, a.sa + at + 2 * i * nb);
        copy8(to + (i + 1) * a.srow, a.sa + at + 2 * (i + 1) * nb);
        if (GLU) {
          copy8(to + (hop + i) * a.srow, a.sb + at + 2 * i * nb);
          copy8(to + (hop + i + 1) * a.srow, a.sb + at + 2 * (i + 1) * nb);
        }
      }
    }
    arrive_with_copies(bar);
    __syncwarp();
  };
  const int first = GLU ? q0 + warp * G : warp;
  Cursor head{0, 0, 0, G};
  if (warp < items) {
    head.i = first / (GLU ? per : ipp);
    head.q = GLU ? first - head.i * per : (first - head.i * ipp) * G;
    if (!GLU) head.n = min(G, nq - head.q);
  }
  Cursor at = head;
  const int total = warp < items ? ((items - 1 - warp) / NW + 1) * a.nsl : 0;
  int issued = 0;
  for (; issued < total && issued < a.depth; ++issued, next(head)) issue(head, issued);
  act.store(0, smem);
  for (int b = 1; act.more(b); ++b) {
    act.load(b);
    act.store(b, smem);
  }
  __syncthreads();

  bool ok = true;
  Partial<Q> p;
  p.clear();
  int n = 0, slot = 0;
  unsigned phase = 0;
  for (; n < total; ++n) {
    if (!__all_sync(FULL, mbar_wait(full0 + 8 * slot, phase, a.wait_ns, abort_flag))) {
      if (lane == 0) raise_error(a.err, ERR_MOE_WAIT, abort_flag);
      ok = false;
      break;
    }
    const int k0 = at.c * a.tk, len = a.K - k0 < a.tk ? a.K - k0 : a.tk;
    unsigned char* st = ring + (size_t)slot * a.stage_bytes;
    const unsigned char* x = smem + (GLU ? 0 : at.i * act_bytes<Q>(a.K));
    for (int q = 0; q < at.n; ++q) {
      quad_stage<Q, SLICED>(p, st, a, k0, len, (GLU ? 2 : 4) * q, hop, x, lane);
      if (at.c < a.nsl - 1) break;  // (a slice: one quad, its sums go on)
      const float v = row_sum<Q, SLICED>(p, lane);
      p.clear();
      if (GLU) {
        const float u = __shfl_down_sync(FULL, v, 16);
        if (lane == 0 || lane == 8)
          a.out[(t * a.k + pair_of[at.i]) * a.rows + 2 * (at.q + q) + (lane >> 3)] = swiglu(v, u);
      } else if ((lane & 7) == 0) {
        products[4 * (at.i * nq + at.q + q) + (lane >> 3)] = v;
      }
    }
    __syncwarp();
    if (issued < total) {
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      issue(head, slot);
      next(head);
      ++issued;
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
    if (++slot == a.depth) {
      slot = 0;
      phase ^= 1u;
    }
  }
  if constexpr (!GLU) {
    __syncthreads();
    for (int r = threadIdx.x; r < 4 * nq; r += blockDim.x) {
      float y = 0.f;
      for (int i = 0; i < np; ++i) y = __fmaf_rn(weight_of[i], products[4 * nq * i + r], y);
      a.out[t * a.rows + 4 * q0 + r] = y;
    }
  }
  if constexpr (GLU && Q > 0) {
    if (!a.hq) return;
    __threadfence();  // this block's h before its counts
    __syncthreads();
    if (!ok || *abort_flag || q1 <= q0) return;
    for (int g = q0 / 16 + warp; g <= (q1 - 1) / 16; g += NW) {
      const int lo = q0 > 16 * g ? q0 : 16 * g, hi = q1 < 16 * g + 16 ? q1 : 16 * g + 16;
      const int i = g / (per / 16), gi = g - i * (per / 16);
      const long pair = t * a.k + pair_of[i];
      if (hi - lo < 16) {
        int old = 0;
        int* cnt = a.cnt + pair * (a.rows >> 5) + gi;
        if (lane == 0) old = atomicAdd(cnt, hi - lo);
        old = __shfl_sync(FULL, old, 0);
        if (old + hi - lo != 16) continue;  // another block finishes it
        if (lane == 0) *cnt = 0;
        __threadfence();  // the others' h after their counts
      }
      quant_lane<Q>(__ldcg(a.out + pair * a.rows + 32 * gi + lane), a.hq + pair * a.rows,
                    Q == 2 ? a.hl + pair * a.rows : nullptr, a.hs + pair * (a.rows >> 5), gi, lane);
    }
  }
}

// ---- host --------------------------------------------------------------------------

// Bytes of `rows` activation rows in a block's shared memory (past 32 bits for rows of 2^30), and
// as many as leave the stages room.
constexpr unsigned long long kHeld = 200000;
unsigned long long held_bytes(int mode, int K, int rows) {
  return (mode == 0 ? 4ull * K : (unsigned long long)K * mode + K / 8u) * rows;
}

// Stages: whole rows up to SLICE bytes, else the fewest equal slices, and up to four quads of
// short rows; `quads` of them come to a warp.  Where these are few, two smaller stages a warp
// instead of one, so that its copies go on while it computes (8 experts of 1024 x 4096 for one
// row: 15.0 us against 17.0; 64 pairs: 85 against 83).
bool fit(MoeArgs& a, int mode, int rows_held, int products, long quads, int smem_optin, int* smem) {
  a.s_products = (unsigned)held_bytes(mode, a.K, rows_held);  // (a multiple of 16)
  a.ring_off = (a.s_products + 4u * products + 127u) & ~127u;
  const int room = smem_optin - kStatic - (int)a.ring_off;
  const int unit = mode == 0 ? 256 : 128;
  bool found = false;
  for (int n = (a.K + SLICE - 1) / SLICE; n <= a.K / 128; ++n) {
    const int tk = ((a.K + n - 1) / n + unit - 1) & ~(unit - 1);
    int group = 1;
    while (n == 1 && group < 4 && 8 * group * a.K <= 4 * SLICE && quads >= 8 * group) group *= 2;
    for (; group > 0; group /= 2) {
      const int ld = n == 1 ? a.K : tk;
      const unsigned srow = (tk / 16u + 31u) & ~15u;  // (padded: the rows of a quad in different banks)
      const unsigned bytes = (4u * group * (ld + srow) + 127u) & ~127u;
      int depth = room / (int)(NW * bytes);
      if (depth > DEPTH) depth = DEPTH;
      if (depth < 1 || (found && depth < 2)) continue;
      found = true;
      a.tk = tk;
      a.nsl = (a.K + tk - 1) / tk;
      a.ld = ld;
      a.group = group;
      a.srow = srow;
      a.s_off = 4u * group * ld;
      a.stage_bytes = bytes;
      a.depth = depth;
      *smem = (int)a.ring_off + NW * depth * (int)bytes;
      break;
    }
    // large enough, or as deep as it gets
    if (found && (a.depth >= 2 || quads >= 4 || 2 * tk < SLICE)) break;
  }
  return found;
}

template <int Q, bool GLU, bool SLICED = false>
lk_status run(const MoeArgs& a, dim3 grid, int smem, int optin, int pdl, cudaStream_t stream) {
  static std::atomic<int> done[kMaxDevices];
  return launch_moe_kernel(moe_kernel<Q, GLU, SLICED>, done, grid, NW * 32, smem, optin - kStatic, pdl, stream, a);
}

template <bool GLU>
lk_status launch_moe(MoeArgs& a, int mode, int M, int held, const lk_launch_cfg* cfg, cudaStream_t stream) {
  const int path = cfg ? cfg->path : 0;
  if (path == 1 || (path == 3 && mode == 0)) return LK_ERR_SHAPE;
  const bool held_fits = held_bytes(mode, a.K, held) <= kHeld;
  // (the tensor-core kernel streams the activation with the weights: it takes any length)
  bool rows = path == 3 || (path == 0 && mode != 0 && !held_fits);
  if (!rows && !held_fits) return LK_ERR_SHAPE;
  const DeviceInfo* d = device_info(nullptr);
  if (!d) return LK_ERR_CUDA;
  a.wait_ns = opt_wait_us > 0 ? (unsigned long long)opt_wait_us * 1000ull : 2000000000ull;
  a.err = error_word_ptr();
  if (!a.err) return LK_ERR_CUDA;
  if (path == 0 && mode != 0 && !rows) rows = rows_favoured(a.E, a.rows, a.K, a.k, M, mode, GLU, d->sm_count);
  if (rows) return moe_rows(a, GLU, mode, M, cfg_pdl(cfg), stream);
  int smem = 0;
  const int gx = row_blocks(a.rows, a.k, M, d->sm_count, GLU);
  const int products = GLU ? 0 : a.k * 4 * ((a.rows / 4 + gx - 1) / gx);
  const long quads = (GLU ? (long)a.k * a.rows / 2 : (long)a.k * a.rows / 4) / gx / NW;  // of a warp, about
  if (!fit(a, mode, held, products, quads, d->smem_optin, &smem)) return LK_ERR_SHAPE;
  const dim3 grid(gx, M);
  const int pdl = cfg_pdl(cfg);
  return mode == 0   ? (a.nsl > 1 ? run<0, GLU, true>(a, grid, smem, d->smem_optin, pdl, stream)
                                  : run<0, GLU>(a, grid, smem, d->smem_optin, pdl, stream))
         : mode == 1 ? run<1, GLU>(a, grid, smem, d->smem_optin, pdl, stream)
                     : run<2, GLU>(a, grid, smem, d->smem_optin, pdl, stream);
}

// Checks that both calls make of a stack's shape, the mode, the rows and k.
lk_status check_shape(int E, int rows, int K, lk_mode mode, int M, int k, const lk_launch_cfg* cfg) {
  if (mode < LK_DEQUANT || mode > LK_TWOPASS || check_launch_cfg(cfg)) return LK_ERR_ARG;
  if (E < 1 || E > LK_MOE_MAX_E || rows < 128 || rows % 128 || K < 128 || K % 128 || K > LK_MOE_MAX_LEN || M < 0 ||
      M > LK_MAX_BATCH || k < 1 || k > LK_MOE_MAX_K)
    return LK_ERR_SHAPE;
  // rows of a stack, and tiles of all pairs, are 32-bit numbers
  if ((long)E * rows > 0x7fffffffL || (long)k * rows > 0x1fffffffL) return LK_ERR_SHAPE;
  return LK_OK;
}
// Activation rows by mode: present and aligned.
lk_status check_act_in(lk_mode mode, const float* x, const int8_t* xq, const int8_t* xl, const float* xs) {
  if (mode == LK_DEQUANT ? !x : (!xq || !xs || (mode == LK_TWOPASS && !xl))) return LK_ERR_ARG;
  if (mode == LK_DEQUANT ? !aligned(x, 16) : (!aligned(xq, 16) || !aligned(xs, 16) || (mode == LK_TWOPASS && !aligned(xl, 16))))
    return LK_ERR_ALIGN;
  return LK_OK;
}

}  // namespace

extern "C" {

lk_status lk_moe_glu_q8(const int8_t* wg, const uint16_t* wsg, const int8_t* wu, const uint16_t* wsu, int E, int F,
                        int K, lk_mode mode, const float* x, const int8_t* xq, const int8_t* xl, const float* xs, int M,
                        const int32_t* ids, int k, float* h, int8_t* hq, int8_t* hl, float* hs, int* cnt,
                        const lk_launch_cfg* cfg, cudaStream_t stream) {
  lk_status st = check_shape(E, F, K, mode, M, k, cfg);
  if (st) return st;
  if (M == 0) return LK_OK;
  if (!wg || !wsg || !wu || !wsu || !ids || !h) return LK_ERR_ARG;
  if (!aligned(wg, 16) || !aligned(wsg, 16) || !aligned(wu, 16) || !aligned(wsu, 16) || !aligned(ids, 4) || !aligned(h, 16))
    return LK_ERR_ALIGN;
  if ((st = check_act_in(mode, x, xq, xl, xs))) return st;
  if (mode == LK_DEQUANT) hq = nullptr;
  if (hq) {
    if (!hs || !cnt || (mode == LK_TWOPASS && !hl)) return LK_ERR_ARG;
    if (!aligned(hq, 16) || !aligned(hs, 16) || !aligned(cnt, 4) || (mode == LK_TWOPASS && !aligned(hl, 16)))
      return LK_ERR_ALIGN;
  }
  const size_t n = (size_t)M * k * F, mat = (size_t)E * F * K, act = (size_t)M * K;
  const bool words = mode != LK_DEQUANT, two = mode == LK_TWOPASS;
  const Span spans[] = {{h, n * 4},
                        {hq, n},
                        {hq && two ? hl : nullptr, n},
                        {hq ? hs : nullptr, n / 8},
                        {hq ? cnt : nullptr, n / 8},
                        {wg, mat},
                        {wsg, mat / 16},
                        {wu, mat},
                        {wsu, mat / 16},
                        {words ? nullptr : x, act * 4},
                        {words ? xq : nullptr, act},
                        {two ? xl : nullptr, act},
                        {words ? xs : nullptr, act / 8},
                        {ids, (size_t)M * k * 4}};
  if (spans_clash(spans, 5, sizeof spans / sizeof *spans)) return LK_ERR_ARG;
  MoeArgs a = {};
  a.wa = wg;
  a.sa = (const unsigned char*)wsg;
  a.wb = wu;
  a.sb = (const unsigned char*)wsu;
  a.E = E;
  a.rows = F;
  a.K = K;
  a.x = x;
  a.xq = xq;
  a.xl = xl;
  a.xs = xs;
  a.ids = ids;
  a.k = k;
  a.out = h;
  a.hq = hq;
  a.hl = hl;
  a.hs = hs;
  a.cnt = cnt;
  return launch_moe<true>(a, mode, M, 1, cfg, stream);
}

lk_status lk_moe_down_q8(const int8_t* wd, const uint16_t* wsd, int E, int N, int F, lk_mode mode, const float* h,
                         const int8_t* hq, const int8_t* hl, const float* hs, int M, const int32_t* ids,
                         const float* weights, int k, float* y, const lk_launch_cfg* cfg, cudaStream_t stream) {
  lk_status st = check_shape(E, N, F, mode, M, k, cfg);
  if (st) return st;
  if (M == 0) return LK_OK;
  if (!wd || !wsd || !ids || !weights || !y) return LK_ERR_ARG;
  if (!aligned(wd, 16) || !aligned(wsd, 16) || !aligned(ids, 4) || !aligned(weights, 4) || !aligned(y, 16))
    return LK_ERR_ALIGN;
  if ((st = check_act_in(mode, h, hq, hl, hs))) return st;
  const size_t mat = (size_t)E * N * F, act = (size_t)M * k * F;
  const bool words = mode != LK_DEQUANT, two = mode == LK_TWOPASS;
  const Span spans[] = {{y, (size_t)M * N * 4},
                        {wd, mat},
                        {wsd, mat / 16},
                        {words ? nullptr : h, act * 4},
                        {words ? hq : nullptr, act},
                        {two ? hl : nullptr, act},
                        {words ? hs : nullptr, act / 8},
                        {ids, (size_t)M * k * 4},
                        {weights, (size_t)M * k * 4}};
  if (spans_clash(spans, 1, sizeof spans / sizeof *spans)) return LK_ERR_ARG;
  MoeArgs a = {};
  a.wa = wd;
  a.sa = (const unsigned char*)wsd;
  a.E = E;
  a.rows = N;
  a.K = F;
  a.x = h;
  a.xq = hq;
  a.xl = hl;
  a.xs = hs;
  a.ids = ids;
  a.weights = weights;
  a.k = k;
  a.out = y;
  return launch_moe<false>(a, mode, M, k, cfg, stream);
}

}  // extern "C"
