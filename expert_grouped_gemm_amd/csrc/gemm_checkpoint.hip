// The persistent expert-GEMM kernel instantiated for bf16 operands, whose Linear-1
// also leaves its SwiGLU inputs in MXINT8 for the backward pass: the accumulators
// hold whole blocks of 32 columns of a row, so that the codes are made where the
// sums are. H is rounded to bf16 for Linear-2's MFMAs, as in moe_expert_forward: the
// outputs are off by 2.34e-3 of their norm, where rounding the exact ones costs 1.66e-3
// (H in two bf16 terms would double Linear-2). Linear-1 of 4096 rows of 32 experts, d =
// 7168, f = 2048: 390 us for 2.0 GB, 5.1 TB/s, bound by HBM; of 16384 rows of 8, d =
// 4096, f = 14336: 3717 us, 1.04 PFLOP/s, bound by the MFMA units.
#include "gemm_device.h"

namespace moe {

hipError_t launch_gemm_checkpoint(const GemmParams& P, int G, hipStream_t s) {
  hipLaunchKernelGGL(moe_gemm_kernel<OT_CKPT>, dim3(G), dim3(gemm_threads(false)), 0, s, P);
  return hipGetLastError();
}

}  // namespace moe
