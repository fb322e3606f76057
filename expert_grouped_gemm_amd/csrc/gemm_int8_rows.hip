// The experts' Linears on 8-bit integers for experts of few rows (decoding
// steps) and for little weight: the weights' bytes, or the latency of a long K, are
// all that counts, and the persistent GEMM's tiles of 128 or 256 weight rows are
// too few and too coarse to spread over the CUs.
//
// A unit is 32 weight rows of one expert (Linear-1: 16 gate rows and the 16 up
// rows of the same SwiGLU columns) over all of K. Its workgroup's four
// wavefronts take the 128-byte slices of K in turn: each streams its own through
// its own ring in the LDS, without a barrier, and sums its share on
// v_mfma_i32_32x32x32_i8 (weights as the A operand: a lane holds one token row
// and 16 weight rows). The shares are whole numbers, so that they join in the
// LDS to the same sums in any order, the ones the persistent GEMM makes.
//
// One launch: every workgroup reads the offsets and checks the row indices for
// itself (2048 at most, 16 of each of 128 tokens, from the L2), to the same
// verdict, and the first one leaves the report in the workspace.
//
// Bound by HBM and the last-level cache: one token, two experts, d = 4096, f =
// 14336, Linear-1 46 us for 235 MB, 5.1 TB/s; 64 tokens on 32 of 256 experts, d =
// 7168, f = 2048, Linear-2 70 us for 411 MB, 5.9. (Against the persistent GEMM:
// few_rows in gemm.hip.)
#include <type_traits>

#include "gemm_device.h"

namespace moe {
namespace {

constexpr int kRowsWaves = 4;                     // wavefronts of a workgroup, two workgroups per CU
constexpr int kRowsLds = 20 * 1024;               // LDS of a wavefront: its ring, later its share of the sums
constexpr int kRowsBlock = 32;                    // token rows of a pass

// AR: KiB of token rows in a slice (8 rows each); the weights take 4.
__host__ __device__ constexpr int rows_ring(int AR) { return kRowsLds / ((4 + AR) * 1024); }

// Rows [row0, row0 + cnt) of expert e against unit n, cnt <= 8 AR.
template <bool L1, int AR, bool NT>
__device__ __forceinline__ void rows_pass(const GemmParams& P, int e, int n, int row0, int cnt, lds_t* lds) {
  constexpr int D = rows_ring(AR), LD = 4 + AR, SB = LD * 1024;
  const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int lr = lane & 31, hi = lane >> 5;
  const int K = L1 ? P.d : P.f, N = L1 ? 2 * P.f : P.d;
  const uint8_t* W = (L1 ? P.W1 : P.W2) + (size_t)e * N * K;
  const uint8_t* A = L1 ? P.X : P.H;
  lds_t* ring = lds + w * kRowsLds;
  // where this lane's 16 bytes of each load instruction are, K apart: weight
  // rows in order (Linear-1: 16 gate rows, 16 up rows), token rows
  const int sub = lane >> 3;
  uint32_t woff[4], aoff[AR];
  const uint8_t* wbase[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int r = j * 8;
    wbase[j] = W + (size_t)(L1 ? (r < 16 ? n * 16 + r : P.f + n * 16 + r - 16) : n * 32 + r) * K;
    woff[j] = (uint32_t)sub * K + (((lane & 7) ^ chunk_swizzle<128>(r + sub)) << 4);
  }
#pragma unroll
  for (int j = 0; j < AR; ++j) {
    const int r = j * 8 + sub, at = row0 + min(r, cnt - 1);
    aoff[j] = (uint32_t)(L1 && P.a_src ? P.a_src[at] / P.a_k : at) * (uint32_t)K +
              (((lane & 7) ^ chunk_swizzle<128>(r)) << 4);
  }
  // the scales of the sums that this thread will join: token row lr, weight rows
  // 8 q + 4 hi .. + 3 with q = w (Linear-1: gate and up of q = w, w < 2)
  const bool joins = lr < cnt && (!L1 || w < 2);
  const int arow = row0 + min(lr, cnt - 1);
  const float sx = P.Ar[L1 && P.a_src ? P.a_src[arow] / P.a_k : arow];
  const float* Ws = P.Wc + (size_t)e * N;
  const int col = L1 ? n * 16 + 8 * (w & 1) + 4 * hi : n * 32 + 8 * w + 4 * hi;
  const float4 s0 = *reinterpret_cast<const float4*>(Ws + col);
  float4 s1 = s0;
  if constexpr (L1) s1 = *reinterpret_cast<const float4*>(Ws + P.f + col);
  int dst = 0;
  if constexpr (!L1) dst = P.row_dst[arow];

  auto issue = [&](int s, int slot) {
    lds_t* st = ring + slot * SB;
    const uint32_t k = (uint32_t)s * 128;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      __builtin_amdgcn_global_load_lds(wbase[j] + (woff[j] + k), st + j * 1024, 16, 0, NT ? kCpolNT : 0);
#pragma unroll
    for (int j = 0; j < AR; ++j) __builtin_amdgcn_global_load_lds(A + (aoff[j] + k), st + 4096 + j * 1024, 16, 0, 0);
  };
  const int KT = K / 128;
  f32x16 acc = {};
#pragma unroll
  for (int i = 0; i < D; ++i)
    if (w + i * kRowsWaves < KT) issue(w + i * kRowsWaves, i);
  int slot = 0;
  for (int s = w; s < KT; s += kRowsWaves) {
    // the slices after this one that are in flight
    const int after = min((KT - 1 - s) / kRowsWaves, D - 1);
    if (D > 3 && after >= 3) wait_vmcnt<3 * LD>();
    else if (D > 2 && after >= 2) wait_vmcnt<2 * LD>();
    else if (after >= 1) wait_vmcnt<LD>();
    else wait_vmcnt<0>();
    asm volatile("" ::: "memory");
    const lds_t* st = ring + slot * SB;
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      const bf16x8 b = *(const lds_bf16x8*)(st + lds_off<128>(lr, ks * 2 + hi));
      const bf16x8 a = *(const lds_bf16x8*)(st + 4096 + lds_off<128>(min(lr, 8 * AR - 1), ks * 2 + hi));
      acc = mfma_chunk<OT_I8>(b, a, acc);
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the slot has been read
    if (s + D * kRowsWaves < KT) issue(s + D * kRowsWaves, slot);
    slot = slot + 1 == D ? 0 : slot + 1;
  }
  // the four shares, joined
#pragma unroll
  for (int q = 0; q < 4; ++q)
    *(lds_f32x4*)(ring + q * 1024 + lane * 16) = f32x4{acc[4 * q], acc[4 * q + 1], acc[4 * q + 2], acc[4 * q + 3]};
  __syncthreads();
  auto total = [&](int q, const float4& s, float (&v)[4]) {
    i32x4 t = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < kRowsWaves; ++i) t += *(const lds_i32x4*)(lds + i * kRowsLds + q * 1024 + lane * 16);
    v[0] = (float)t[0] * sx * s.x;
    v[1] = (float)t[1] * sx * s.y;
    v[2] = (float)t[2] * sx * s.z;
    v[3] = (float)t[3] * sx * s.w;
  };
  if (joins) {
    float v[4];
    total(w, s0, v);
    if constexpr (L1) {
      float u[4];
      total(w + 2, s1, u);
      const uint32_t lo = (uint32_t)f32_to_bf16_rne(silu_mul(v[0], u[0])) | ((uint32_t)f32_to_bf16_rne(silu_mul(v[1], u[1])) << 16);
      const uint32_t up = (uint32_t)f32_to_bf16_rne(silu_mul(v[2], u[2])) | ((uint32_t)f32_to_bf16_rne(silu_mul(v[3], u[3])) << 16);
      *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(P.H) + (size_t)arow * P.f + col) = make_uint2(lo, up);
    } else if (P.c_bf16) {
      const uint32_t lo = (uint32_t)f32_to_bf16_rne(v[0]) | ((uint32_t)f32_to_bf16_rne(v[1]) << 16);
      const uint32_t up = (uint32_t)f32_to_bf16_rne(v[2]) | ((uint32_t)f32_to_bf16_rne(v[3]) << 16);
      *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(P.C) + (size_t)dst * P.d + col) = make_uint2(lo, up);
    } else {
      *reinterpret_cast<float4*>(reinterpret_cast<float*>(P.C) + (size_t)dst * P.d + col) = make_float4(v[0], v[1], v[2], v[3]);
    }
  }
  __syncthreads();  // the shares have been read
}

template <bool L1, bool NT>
__device__ __forceinline__ void rows_unit(const GemmParams& P, int e, int n, int row0, int rows, lds_t* lds) {
  for (int first = 0; first < rows; first += kRowsBlock) {
    const int cnt = min(kRowsBlock, rows - first);
    if (cnt <= 8) rows_pass<L1, 1, NT>(P, e, n, row0 + first, cnt, lds);
    else if (cnt <= 16) rows_pass<L1, 2, NT>(P, e, n, row0 + first, cnt, lds);
    else rows_pass<L1, 4, NT>(P, e, n, row0 + first, cnt, lds);
  }
}

// The checks of plan_rows_kernel, and the experts that have rows: bit i of
// has[j] is expert 64 j + i (wavefront-uniform). False where a check fails.
__device__ __forceinline__ bool plan_few_rows(const RowsPlan& R, const GemmParams& P, uint64_t (&has)[16], lds_t* lds) {
  const int tid = threadIdx.x, lane = tid & 63;
  lds_i32* err = (lds_i32*)lds;
  if (tid == 0) *err = 0;
  const int first = R.offsets[0], last = R.offsets[R.El];
  int bits = first < 0 || last > P.cap ? ARG_ERR_OFFSETS : 0, bands = 0;
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    const int e = j * 64 + lane;
    // compared, not subtracted: two offsets far apart differ by more than 32 bits hold
    const int lo = e < R.El ? R.offsets[e] : 0, hi = e < R.El ? R.offsets[e + 1] : 0;
    if (hi < lo) bits |= ARG_ERR_OFFSETS;
    has[j] = __ballot(hi > lo);
    if (hi > lo) bands += (int)(((int64_t)hi - lo + kBM - 1) / kBM);
  }
  const int r_end = min(P.cap, last);
  auto check = [&](int r0, auto n) {  // N of either array per thread in flight
    constexpr int N = decltype(n)::value;
    int src[N], dst[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int r = min(r0 + i * kRowsWaves * 64 + tid, r_end - 1);
      src[i] = P.a_src ? P.a_src[r] : 0;
      dst[i] = P.row_dst ? P.row_dst[r] : 0;
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (src[i] < 0 || src[i] >= R.src_end) bits |= ARG_ERR_ROW_SRC;
      if ((unsigned)dst[i] >= (unsigned)P.cap) bits |= ARG_ERR_ROW_DST;
    }
    return r0 + N * kRowsWaves * 64;
  };
  for (int r = max(0, first); r < r_end;)
    r = r_end - r > kRowsWaves * 64 ? check(r, std::integral_constant<int, 8>{})
                                    : check(r, std::integral_constant<int, 1>{});
  __syncthreads();
  if (bits) __hip_atomic_fetch_or((__attribute__((address_space(3))) int*)err, bits, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
  __syncthreads();
  const int all = *err;
  __syncthreads();  // the ring may be filled
  if (blockIdx.x == 0 && tid < 64) {
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) bands += __shfl_xor(bands, off, 64);
    if (tid == 0) {
      int32_t* meta = P.meta;
      const bool written = meta[META_TAG] == kMetaTag;
      const int wait_err = written ? meta[META_ERR] : 0, kept = written ? meta[META_ARG_ERR] & R.keep : 0;
      meta[META_ERR] = wait_err;
      meta[META_TRACE_N] = 0;
      meta[META_ARG_ERR] = kept | all | (all ? R.mark : 0);
      meta[META_TAG] = kMetaTag;
      meta[META_P] = all ? 0 : bands;
      meta[META_A] = all ? 0 : last;
    }
  }
  return all == 0;
}

template <bool L1>
__global__ __launch_bounds__(kRowsWaves * 64, 2) void int8_rows_kernel(GemmParams P, RowsPlan R) {
  __shared__ __attribute__((aligned(1024))) uint8_t smem[kRowsWaves * kRowsLds];
  lds_t* lds = (lds_t*)smem;
  const int G = gridDim.x, b = blockIdx.x, lane = threadIdx.x & 63;
  const int lid = G % 8 == 0 ? (b % 8) * (G / 8) + b / 8 : b;
  uint64_t has[16];
  if (!plan_few_rows(R, P, has, lds)) return;
  int experts = 0;
#pragma unroll
  for (int j = 0; j < 16; ++j) experts += __popcll(has[j]);
  const int units = L1 ? P.f / 16 : P.d / 32;
  const int64_t total = (int64_t)experts * units;
  for (int64_t i = lid; i < total; i += G) {
    int left = (int)(i / units);
    const int n = (int)(i - (int64_t)left * units);
    // the expert that `left` others with rows come before
    uint64_t word = 0;
    int base = -1;
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const int c = __popcll(has[j]);
      if (base < 0 && left < c) {
        word = has[j];
        base = j * 64;
      } else if (base < 0) {
        left -= c;
      }
    }
    const bool mine = (word >> lane & 1) && __popcll(word & ((1ull << lane) - 1)) == left;
    const int e = __builtin_amdgcn_readfirstlane(base + __builtin_ctzll(__ballot(mine)));
    const int row0 = R.offsets[e], rows = R.offsets[e + 1] - row0;
    // weights that one pass reads are read once (see streams_once)
    if (rows <= kRowsBlock) rows_unit<L1, true>(P, e, n, row0, rows, lds);
    else rows_unit<L1, false>(P, e, n, row0, rows, lds);
  }
}

}  // namespace

hipError_t launch_int8_rows(const GemmParams& P, const RowsPlan& R, int G, hipStream_t s) {
  if (P.mode == MODE_SEP_L1)
    hipLaunchKernelGGL(int8_rows_kernel<true>, dim3(2 * G), dim3(kRowsWaves * 64), 0, s, P, R);
  else hipLaunchKernelGGL(int8_rows_kernel<false>, dim3(2 * G), dim3(kRowsWaves * 64), 0, s, P, R);
  return hipGetLastError();
}

}  // namespace moe
