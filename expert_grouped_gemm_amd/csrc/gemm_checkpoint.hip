// The persistent expert-GEMM kernel instantiated for bf16 operands, whose Linear-1
// also leaves its SwiGLU inputs in MXINT8 for the backward pass.
#include "gemm_device.h"

namespace moe {

hipError_t launch_gemm_checkpoint(const GemmParams& P, int G, hipStream_t s) {
  hipLaunchKernelGGL(moe_gemm_kernel<OT_CKPT>, dim3(G), dim3(gemm_threads(false)), 0, s, P);
  return hipGetLastError();
}

}  // namespace moe
