// The persistent expert-GEMM kernel instantiated for MXFP4 activations and
// MXFP4 weights (E2M1 codes with E8M0 block scales on both sides).
#include "gemm_device.h"

namespace moe {

hipError_t launch_gemm_w4a4(const GemmParams& P, int G, hipStream_t s) {
  hipLaunchKernelGGL(moe_gemm_kernel<OT_W4A4>, dim3(G), dim3(gemm_threads(true)), 0, s, P);
  return hipGetLastError();
}

}  // namespace moe
