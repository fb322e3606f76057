// The persistent expert-GEMM kernel instantiated for 8-bit integer activations and
// weights (one fp32 scale per row of either). The ring, tiles and schedule are the
// bf16 kernel's with half the bytes per value: a stage of 128 bytes per row holds
// 128 values of K, and v_mfma_i32_32x32x32_i8 takes a 16-byte chunk per lane as the
// bf16 MFMA does. The scales stay out of the K loop (sums of whole numbers are
// exact), so that a stage is rows alone. Linear-1 of 4096 tokens on 32 of 256
// experts, d = 7168, f = 2048: 187 us for 986 MB, 5.3 TB/s. Of 16384 rows, d = 4096, f
// = 14336: Linear-1 1958 us, 1.97 POP/s, Linear-2 970-980 (the fastest launch 900),
// 1.97, bound by the MFMA units and the tiles' stores (470 MB of H, 268 of slots).
#include "gemm_device.h"

namespace moe {

hipError_t launch_gemm_int8(const GemmParams& P, int G, hipStream_t s) {
  hipLaunchKernelGGL(moe_gemm_kernel<OT_I8>, dim3(G), dim3(gemm_threads(true)), 0, s, P);
  return hipGetLastError();
}

}  // namespace moe
