// Device helpers shared by the dense attention kernels (attn_dense.cu,
// attn_window.cu).
#pragma once
#include <limits.h>

#include <atomic>

#include "common.cuh"

namespace csa2 {

constexpr int kRows = 128;                   // flattened (query, head) rows of a unit
constexpr int kMaxQ = kRows + 1;             // queries that 128 rows can touch
constexpr int kMaxPos = INT_MAX - 4096;      // sums of a position with a tile or a window stay in 32 bits
constexpr float kLog2e = 1.4426950408889634f;
constexpr uint32_t kWaitLimit = 1u << 22;

// Byte offset of 16-byte piece `pc` (8 fp16 elements) of row `r` in a K-major
// 128B-swizzled operand whose chunks of 64 elements hold `rows` rows.
__device__ __forceinline__ uint32_t sw_off(int r, int pc, int rows) {
  return (uint32_t)((pc >> 3) * rows * 128 + r * 128 + (((pc & 7) ^ (r & 7)) << 4));
}

// 2^x by the hardware's approximate exponential (relative error ~2^-22, far
// below the fp16 rounding of P it feeds).
__device__ __forceinline__ float ex2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two fp32 operations per instruction.
__device__ __forceinline__ uint64_t f32x2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 unpack_f32x2(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// Bounded wait that also gives up early once another role raised `abort`.
__device__ __forceinline__ bool wait_or_abort(uint64_t *bar, uint32_t parity, volatile int *abort) {
  for (uint32_t i = 0; i < kWaitLimit; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 255u) == 255u && *abort) return false;
  }
  *abort = 1;
  return false;
}

// Raises a kernel's dynamic shared memory limit, once per device (bit d of
// `done`; the attribute belongs to the device's context).
template <typename K>
inline cudaError_t allow_smem_once(K kernel, size_t smem, std::atomic<uint64_t> *done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || (dev < 64 && ((done->load(std::memory_order_relaxed) >> dev) & 1u))) return e;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e == cudaSuccess && dev < 64) done->fetch_or((uint64_t)1 << dev, std::memory_order_relaxed);
  return e;
}

}  // namespace csa2
