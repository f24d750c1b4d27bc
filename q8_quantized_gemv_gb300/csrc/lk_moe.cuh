// What the kernels of the experts' products share (lk_moe.cu, lk_moe_rows.cu).
#pragma once

#include <math.h>

#include "lk_moe.h"
#include "lk_ring_kernel.cuh"
#include "lk_spans.h"

namespace lkmoe {

constexpr int ERR_MOE_WAIT = 256;  // bit of the device error word

struct MoeArgs {
  const int8_t* wa;            // gate, or down
  const unsigned char* sa;     // f16 scales, as bytes
  const int8_t* wb;            // up
  const unsigned char* sb;
  int E, rows, K;              // a matrix: [rows][K]
  const float* x;              // activation rows: M (gate/up) or M * k (down)
  const int8_t* xq;
  const int8_t* xl;
  const float* xs;
  const int* ids;
  const float* weights;
  int k;
  float* out;                  // h [M * k][rows], or y [M][rows]
  int8_t* hq;
  int8_t* hl;
  float* hs;
  int* cnt;
  int tk, nsl;                 // bytes of K in a stage, stages of a row
  int ld, group;               // single rows: bytes between a stage's rows, quads of an item
  int depth;                   // stages of a warp
  unsigned srow, s_off, stage_bytes, ring_off, s_products;
  unsigned long long wait_ns;
  int* err;
};

// Blocks of an activation row of the single-row kernel, `sms` SMs for M rows: all of them on the
// SMs at once (a second wave of blocks doubles the time); down: enough that a block's products
// are few.
constexpr int kProducts = 16384;  // down: bytes of a block's products, about
inline int row_blocks(int rows, int k, int M, int sms, bool glu) {
  int gx = sms / M;
  if (gx < 1) gx = 1;
  if (!glu) {
    const int least = (int)(((long)k * rows * 4 + kProducts - 1) / kProducts);
    if (gx < least) gx = least;
    if (gx > rows / 4) gx = rows / 4;
  }
  return gx;
}

// Whether the tensor-core kernel, which reads a shared expert once, is faster than single rows.
// By the bytes that each reads, in us (MB by TB/s): single rows a pair's matrices for each of
// the pairs, from HBM or L2, wave after wave of blocks; the tensor cores those of the experts
// touched, as uniform routing has it (absent pairs count: the host does not know them), and
// a start and an end that grow with a matrix.  The constants are fitted to the times of 90
// shapes in both modes (1 to 64 rows, 4 to 512 experts, matrices of 35 KB to 62 MB): the kernel
// chosen takes 0.3 to 0.7 % more than the better one on the mean, 19 % at the worst.  Single
// rows against tensor cores, us, gate/up and down: 128 experts 4096 x 1024, k 8, Int8Act 8 rows
// 79 / 84 and 42 / 50, 16 rows 150 / 132 and 84 / 72, TwoPass 8 rows 83 / 87 and 50 / 51; 60
// experts 2048 x 1408, k 4, Int8Act 16 rows 51 / 52 and 30 / 35, 32 rows 97 / 66 and 59 / 45;
// 256 experts 4096 x 1024, k 8, Int8Act 16 rows 159 / 156 and 85 / 86, 20 rows 194 / 175 and
// 178 (two waves) / 98; 4 experts 1024 x 1024, k 1, 32 rows 16 / 9 and 10 / 9; 8 experts
// 4096 x 14336, k 2, 1 row 41 / 56 and 33 / 59.
inline bool rows_favoured(int E, int rows, int K, int k, int M, int mode, bool glu, int sms) {
  const double mb = (double)rows * K * (glu ? 2 : 1) * 1.0625e-6, pairs = (double)M * k;
  const double touched = k < E ? E * (1.0 - pow(1.0 - (double)k / E, M)) : E;  // (a row's are different ones)
  const int waves = (int)(((long)row_blocks(rows, k, M, sms, glu) * M + sms - 1) / sms);
  struct Fit {
    double rate, start, grows, to;  // TB/s; us, us a MB, up to so many
  };
  constexpr Fit fits[2][2] = {{{7.4, 2.0, 1.75, 6.0}, {7.8, 0.0, 1.25, 20.0}},   // Int8Act: down, gate/up
                              {{4.4, 2.0, 4.75, 3.0}, {7.2, 1.0, 1.0, 12.0}}};  // TwoPass
  const Fit& f = fits[mode - 1][glu];
  return waves * pairs * mb / f.rate >= touched * mb / 6.0 + f.start + f.grows * (mb < f.to ? mb : f.to);
}

// A kernel with `smem` bytes of dynamic shared memory, of `most` at most.
template <typename A>
lk_status launch_moe_kernel(void (*f)(A), std::atomic<int> (&done)[lkh::kMaxDevices], dim3 grid, int threads, int smem,
                            int most, int pdl, cudaStream_t stream, const A& a) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= lkh::kMaxDevices) return LK_ERR_CUDA;
  if (!done[dev].load(std::memory_order_acquire)) {
    if (cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, most) != cudaSuccess) return LK_ERR_CUDA;
    lkh::carveout_max_shared(f);
    done[dev].store(1, std::memory_order_release);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, f, a) == cudaSuccess ? LK_OK : LK_ERR_CUDA;
}

// A lane's own copies, and its arrival at `bar` when they are there.
__device__ __forceinline__ void copy16(void* to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(lkring::smem_u32(to)), "l"(from) : "memory");
}
__device__ __forceinline__ void copy8(void* to, const void* from) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(lkring::smem_u32(to)), "l"(from) : "memory");
}
__device__ __forceinline__ void arrive_with_copies(unsigned bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

// The quantized modes for several rows (lk_moe_rows.cu).
lk_status moe_rows(const MoeArgs& a, bool glu, int mode, int M, int pdl, cudaStream_t stream);

}  // namespace lkmoe
