// attend_kernel for head_dim 128.
#include "attend_kernel.cuh"

namespace mpk {
cudaError_t launch_attend_128(const AttendArgs& a, cudaStream_t s) {
  return run_attend<128>(a, s);
}
}  // namespace mpk
