// What the kernels of the experts' products share (lk_moe.cu, lk_moe_rows.cu).
#pragma once

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
