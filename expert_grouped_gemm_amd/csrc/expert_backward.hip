// The gradient of the experts' SwiGLU products (moe_expert_backward): the
// products over row bands, and the launch sequence. The kernels are in
// expert_backward_device.h, the weight gradients' launches in
// expert_backward_weights.hip.
#include "expert_backward_device.h"

namespace moe {
namespace {

// Copies of the token rows (with row_src) and of the output gradients in expert
// order, for the weight gradients of long experts: the call of 16384 rows, d =
// 4096, f = 14336 takes 15.2 ms with the copies (84 us of it) and 16.3 with the
// rows looked up in every stage. 16 bytes per lane.
__global__ __launch_bounds__(256) void order_rows_kernel(BwdParams P) {
  if (P.meta[META_ARG_ERR] & ARG_ERR_PLAN) return;
  const int first = P.offsets[0], last = P.offsets[P.El], vec = P.d >> 3;
  const int64_t n = (int64_t)(last - first) * vec;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
    const int r = first + (int)(i / vec), c = (int)(i % vec);
    const size_t at = (size_t)r * vec + c;
    if (P.row_src)
      reinterpret_cast<uint4*>(P.Xp)[at] =
          reinterpret_cast<const uint4*>(P.X)[(size_t)(P.row_src[r] / P.k) * vec + c];
    reinterpret_cast<uint4*>(P.dOp)[at] = reinterpret_cast<const uint4*>(P.dO)[(size_t)P.row_dst[r] * vec + c];
  }
}

template <int OP>
hipError_t launch_bands(const BwdParams& P, int G, hipStream_t s) {
  hipLaunchKernelGGL(expert_backward_kernel<OP>, dim3(G), dim3(kBwdThreads), 0, s, P);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_backward_dx(const BwdParams& P, int G, hipStream_t s) { return launch_bands<BWD_DX>(P, G, s); }

hipError_t launch_order_rows(const BwdParams& P, hipStream_t s) {
  hipLaunchKernelGGL(order_rows_kernel, dim3(4096), dim3(256), 0, s, P);
  return hipGetLastError();
}

BackwardLayout backward_layout(const moe_problem_t& p, const Layout& L) {
  BackwardLayout B;
  size_t o = align_up(L.pub.total, 256);
  auto take = [&](size_t bytes) { size_t at = o; o = align_up(o + bytes, 256); return at; };
  B.gu = take((size_t)L.cap * 2 * p.f * 4);
  B.act = take((size_t)L.cap * p.f * 2);
  B.dh = take((size_t)L.cap * 2 * p.f * 2);
  const size_t rows = long_experts(p) ? (size_t)L.cap * p.d * 2 : 0;
  B.x_rows = take(rows);
  B.do_rows = take(rows);
  B.total = o;
  return B;
}

BackwardLayout checkpoint_layout(const moe_problem_t& p, const Layout& L) {
  BackwardLayout B;
  size_t o = align_up(L.pub.total, 256);
  auto take = [&](size_t bytes) { size_t at = o; o = align_up(o + bytes, 256); return at; };
  B.gu = take(0);
  B.act = take((size_t)L.cap * p.f * 2);
  B.dh = take((size_t)L.cap * 2 * p.f * 2);
  B.x_rows = take((size_t)L.cap * p.d * 2);
  B.do_rows = take(long_experts(p) ? (size_t)L.cap * p.d * 2 : 0);
  B.total = o;
  return B;
}

BwdParams backward_params(const moe_problem_t& p, const Layout& L, const BackwardLayout& B, char* ws, const void* X,
                          const int32_t* row_src, const int32_t* offsets, const int32_t* row_dst, const void* W1,
                          const void* W2, const void* dO, void* dxs, void* dW1, void* dW2) {
  auto I = [&](size_t off) { return reinterpret_cast<const int32_t*>(ws + off); };
  BwdParams P{};
  P.X = static_cast<const uint8_t*>(X);
  P.dO = static_cast<const uint8_t*>(dO);
  P.W1 = static_cast<const uint8_t*>(W1);
  P.W2 = static_cast<const uint8_t*>(W2);
  P.GU = reinterpret_cast<float*>(ws + B.gu);
  P.act = reinterpret_cast<uint16_t*>(ws + B.act);
  P.dH = reinterpret_cast<uint16_t*>(ws + B.dh);
  P.dxs = static_cast<uint16_t*>(dxs);
  P.dW1 = static_cast<uint16_t*>(dW1);
  P.dW2 = static_cast<uint16_t*>(dW2);
  P.Xp = reinterpret_cast<uint16_t*>(ws + B.x_rows);
  P.dOp = reinterpret_cast<uint16_t*>(ws + B.do_rows);
  P.row_src = row_src;
  P.row_dst = row_dst;
  P.offsets = offsets;
  P.band_expert = I(L.band_expert);
  P.band_row0 = I(L.band_row0);
  P.band_rows = I(L.band_rows);
  P.meta = I(L.pub.meta);
  P.k = p.k;
  P.d = p.d;
  P.f = p.f;
  P.El = L.E_l;
  P.group_m = 4;  // as in the forward (2: GU and DW1 of long experts 4% slower; 8: DW2 2%)
  return P;
}

hipError_t launch_expert_backward(const moe_problem_t& p, const Layout& L, char* ws, const void* X,
                                  const int32_t* row_src, const int32_t* offsets, const int32_t* row_dst,
                                  const void* W1, const void* W2, const void* dO, void* dxs, void* dW1, void* dW2,
                                  hipStream_t s) {
  const int G = gemm_grid(p);
  if (G <= 0) return hipErrorInvalidDevice;
  hipError_t e = launch_plan_rows(p, L, ws, offsets, row_src, row_dst, ARG_ERR_DISPATCH_CAP | ARG_ERR_LINEAR1, 0, s);
  const BwdParams P = backward_params(p, L, backward_layout(p, L), ws, X, row_src, offsets, row_dst, W1, W2, dO, dxs,
                                      dW1, dW2);
  if (e == hipSuccess) e = launch_bands<BWD_GU>(P, G, s);
  if (e == hipSuccess) e = launch_bands<BWD_DACT>(P, G, s);
  if (e == hipSuccess) e = launch_backward_dx(P, G, s);
  if (e == hipSuccess && long_experts(p)) e = launch_order_rows(P, s);
  if (e == hipSuccess) e = launch_weight_gradients(P, long_experts(p), G, s);
  return e;
}

}  // namespace moe
