// attend_kernel for head_dim 64.
#include "attend_kernel.cuh"

namespace mpk {
cudaError_t launch_attend_64(const AttendArgs& a, cudaStream_t s) {
  return run_attend<64>(a, s);
}
}  // namespace mpk
