// The gradient of the experts' SwiGLU products from an 8-bit checkpoint
// (moe_expert_backward_checkpoint; see expert_backward_device.h).
#include "expert_backward_device.h"

namespace moe {
namespace {

// The rows of a checkpoint: the token rows in expert order, their MXINT8 codes
// as the bf16 values they stand for (exact), and with DO the output gradients as
// in order_rows_kernel. 8 values per lane.
template <bool DO>
__global__ __launch_bounds__(256) void expand_rows_kernel(BwdParams P) {
  if (P.meta[META_ARG_ERR] & ARG_ERR_PLAN) return;
  const int first = P.offsets[0], last = P.offsets[P.El], vec = P.d >> 3;
  const int64_t n = (int64_t)(last - first) * vec;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
    const int r = first + (int)(i / vec), c = (int)(i % vec);
    const size_t at = (size_t)r * vec + c, from = (size_t)(P.row_src ? P.row_src[r] / P.k : r) * vec + c;
    float v[8];
    mxint8_values8(reinterpret_cast<const uint2*>(P.X)[from], mxint8_step(P.Xs[from >> 2]), v);
    reinterpret_cast<uint4*>(P.Xp)[at] =
        make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
    if constexpr (DO)
      reinterpret_cast<uint4*>(P.dOp)[at] = reinterpret_cast<const uint4*>(P.dO)[(size_t)P.row_dst[r] * vec + c];
  }
}

}  // namespace

// From a checkpoint the gate and up product falls away: DACT reads its codes.
// MXINT8 tokens are expanded once, into expert order, for DW1 (its K-strided
// operand is fed to the bf16 MFMA; the values are exact in bf16).
hipError_t launch_expert_backward_checkpoint(const moe_problem_t& p, const Layout& L, char* ws, const void* X,
                                             const uint8_t* X_scale, const int32_t* row_src, const int32_t* offsets,
                                             const int32_t* row_dst, const int8_t* gu, const uint8_t* gu_scale,
                                             const void* W1, const void* W2, const void* dO, void* dxs, void* dW1,
                                             void* dW2, hipStream_t s) {
  const int G = gemm_grid(p);
  if (G <= 0) return hipErrorInvalidDevice;
  const bool long_rows = long_experts(p);
  hipError_t e = launch_plan_rows(p, L, ws, offsets, row_src, row_dst, ARG_ERR_DISPATCH_CAP | ARG_ERR_LINEAR1, 0, s);
  BwdParams P = backward_params(p, L, checkpoint_layout(p, L), ws, X, row_src, offsets, row_dst, W1, W2, dO, dxs, dW1,
                                dW2);
  P.Xs = X_scale;
  P.gu8 = gu;
  P.gus = gu_scale;
  auto go = [&](auto kern, int grid, int threads) {
    if (e != hipSuccess) return;
    hipLaunchKernelGGL(kern, dim3(grid), dim3(threads), 0, s, P);
    e = hipGetLastError();
  };
  go(expert_backward_kernel<BWD_DACT8>, G, kBwdThreads);
  if (e == hipSuccess) e = launch_backward_dx(P, G, s);
  if (X_scale) {
    if (long_rows) go(expand_rows_kernel<true>, 4096, 256);
    else go(expand_rows_kernel<false>, 4096, 256);
    P.X = reinterpret_cast<const uint8_t*>(P.Xp);  // the rows now stand in expert order
    P.row_src = nullptr;
  } else if (long_rows && e == hipSuccess) {
    e = launch_order_rows(P, s);
  }
  if (e == hipSuccess) e = launch_weight_gradients(P, long_rows, G, s);
  return e;
}

}  // namespace moe
