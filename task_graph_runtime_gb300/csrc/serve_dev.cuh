// Device helpers shared by the serving operators' kernels.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "mpk.h"
#include "serve.h"

namespace mpk {

__device__ __forceinline__ float sv_lo(uint32_t w) {
  return __uint_as_float(w << 16);
}
__device__ __forceinline__ float sv_hi(uint32_t w) {
  return __uint_as_float(w & 0xffff0000u);
}
// two fp32 to packed bf16, nearest even (lo in the low half)
__device__ __forceinline__ uint32_t sv_pack(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t sv_div(uint32_t n, const FastDiv& f) {
  return (__umulhi(n, f.mul) + n) >> f.shift;
}
// The first error of a call stays in the caller's status word.
__device__ __forceinline__ void sv_latch(uint32_t* status, uint32_t code) {
  if (status) atomicCAS(status, 0u, code);
}
// Programmatic dependent launch: wait until the kernels before this one in
// the stream have finished and their writes are visible / let the next
// kernel of the stream start its preamble.
__device__ __forceinline__ void sv_grid_wait() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ void sv_grid_launch() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// First token row of sequence b (clamped to the batch's rows, so that a bad
// array cannot lead outside the tensors).
__device__ __forceinline__ int sv_row(const int32_t* q_start, int per, int n,
                                      int b) {
  const int r = q_start ? __ldg(q_start + b) : b * per;
  return min(max(r, 0), n);
}
// Sequence that owns token row t; -1 when t lies behind the last sequence.
__device__ __forceinline__ int sv_seq_of(const int32_t* q_start, int per,
                                         int batch, int t) {
  if (!q_start) {
    const int b = per > 0 ? t / per : batch;
    return b < batch ? b : -1;
  }
  if (t < __ldg(q_start) || t >= __ldg(q_start + batch)) return -1;
  int lo = 0, hi = batch;          // q_start[lo] <= t < q_start[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(q_start + mid) <= t) lo = mid;
    else hi = mid;
  }
  return lo;
}

// The same by a whole warp: the sequences that end at or before row t are
// counted 32 at a time, one load's latency for all (a search takes one for
// each halving).  Large batches are searched.
__device__ __forceinline__ int sv_seq_of_warp(const int32_t* q_start, int per,
                                              int batch, int t) {
  if (!q_start || batch > 512) return sv_seq_of(q_start, per, batch, t);
  if (t < __ldg(q_start)) return -1;
  int n = 0;
#pragma unroll 4
  for (int b0 = 0; b0 < batch; b0 += 32) {
    const int b = b0 + (int)(threadIdx.x & 31);
    const bool done = b < batch && __ldg(q_start + b + 1) <= t;
    n += __popc(__ballot_sync(0xffffffffu, done));
  }
  return n < batch ? n : -1;
}

// Raises a kernel's limit of dynamic shared memory, once a device.
struct SmemLimit {
  std::atomic<bool> done[64] = {};
  cudaError_t set(const void* kernel, int bytes) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const bool known = dev < 64;
    if (known && done[dev].load(std::memory_order_relaxed)) return e;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             bytes);
    if (e == cudaSuccess && known) done[dev].store(true);
    return e;
  }
};

// Launch with the attribute that lets the kernel's preamble overlap the end
// of the kernel before it in the stream (which must call sv_grid_wait before
// it touches what that kernel writes).
template <typename... KArgs, typename... Args>
inline cudaError_t sv_launch(void (*k)(KArgs...), dim3 grid, int threads,
                             size_t smem, cudaStream_t s, Args... args) {
  cudaLaunchConfig_t c = {};
  c.gridDim = grid;
  c.blockDim = dim3(threads);
  c.dynamicSmemBytes = smem;
  c.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  c.attrs = at;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, k, args...);
}

}  // namespace mpk
