// The persistent expert-GEMM kernel instantiated for 8-bit integer activations and weights
// (one fp32 scale per row of either).
#include "gemm_device.h"

namespace moe {

hipError_t launch_gemm_int8(const GemmParams& P, int G, hipStream_t s) {
  hipLaunchKernelGGL(moe_gemm_kernel<OT_I8>, dim3(G), dim3(gemm_threads(true)), 0, s, P);
  return hipGetLastError();
}

}  // namespace moe
