// attend_kernel for head_dim 32.
#include "attend_kernel.cuh"

namespace mpk {
cudaError_t launch_attend_32(const AttendArgs& a, cudaStream_t s) {
  return run_attend<32>(a, s);
}
}  // namespace mpk
