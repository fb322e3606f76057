// The experts' weight gradients (see expert_backward_device.h).
#include "expert_backward_device.h"

namespace moe {

hipError_t launch_weight_gradients(const BwdParams& P, bool long_rows, int G, hipStream_t s) {
  hipError_t e = hipSuccess;
  auto go = [&](auto kern, int grid, int threads) {
    if (e != hipSuccess) return;
    hipLaunchKernelGGL(kern, dim3(grid), dim3(threads), 0, s, P);
    e = hipGetLastError();
  };
  if (long_rows) {
    go(expert_backward_kernel<BWD_DW2>, G, kBwdThreads);
    go(expert_backward_kernel<BWD_DW1>, G, kBwdThreads);
  } else {
    go(weight_backward_short_kernel<BWD_DW2>, 2 * G, 256);
    go(weight_backward_short_kernel<BWD_DW1>, 2 * G, 256);
  }
  return e;
}

}  // namespace moe
