// Gradient of the experts' SwiGLU products (moe_expert_backward).
//
// Per local expert e and its rows r (x the token, do the gradient of the
// expert's output), with [g u] = W1 x recomputed and s = sigmoid(g):
//   a  = g s u                         (bf16: Linear-2's operand in the forward)
//   da = W2^T do
//   dg = da u s (1 + g (1 - s)),  du = da g s,  dh = bf16([dg du])
//   dx = W1^T dh,   dW2 = sum_r do a^T,   dW1 = sum_r dh x^T
// 16 A d f operations on A rows, as five grouped products on bf16 MFMA:
//   GU    g, u (fp32)        rows x W1 rows          both contiguous along K = d
//   DACT  da -> dh, a        rows x W2 columns       W2 strided along K = d
//   DX    dx                 rows x W1 columns       W1 strided along K = 2f
//   DW2   dW2[e] = do^T a    both strided along K = the expert's rows
//   DW1   dW1[e] = dh^T x    both strided along K
// a and dh are rounded to bf16, the operand type of the products they enter
// (a as in the forward); every sum is fp32, dx and the weight gradients are
// rounded once. Every output element is one workgroup's sum in one K order:
// no atomics, the same result on every call.
//
// An operand contiguous along K (KC) lies in the LDS as rows of 64 K values
// and is read 16 bytes per lane; one strided along K (KS) lies as 64 rows of K
// with the tile's 256 columns each and is read by the transposing LDS read
// (ds_read_b64_tr_b16: 16 lanes take 4 K rows x 16 columns, lane i ends with
// the 4 K values of column i), so no operand is ever transposed in memory.
#include "gemm_device.h"

namespace moe {
namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

enum BwdOp { BWD_GU = 0, BWD_DACT = 1, BWD_DX = 2, BWD_DW2 = 3, BWD_DW1 = 4 };
__host__ __device__ constexpr bool p_strided(int OP) { return OP != BWD_GU; }
__host__ __device__ constexpr bool q_strided(int OP) { return OP >= BWD_DW2; }

constexpr int kBK = 64;                      // K values per stage
constexpr int kTP = 256;                     // columns (P side) of a tile
constexpr int kBwdThreads = 512;             // 8 wavefronts: 2 (Q) x 4 (P)
constexpr int kStageP = kTP * kBK * 2;       // bytes of the P operand in a stage
constexpr int kStageQ = kBM * kBK * 2;

struct BwdParams {
  const uint8_t* X;          // token rows [T, d] (through row_src) or expert-ordered rows
  const uint8_t* dO;         // [cap, d], row r at slot row_dst[r]
  const uint8_t* W1;         // [E_l, 2f, d]
  const uint8_t* W2;         // [E_l, d, f]
  float* GU;                 // [cap, 2f]
  uint16_t* act;             // [cap, f]
  uint16_t* dH;              // [cap, 2f]
  uint16_t* dxs;             // [cap, d] by slot
  uint16_t* dW1;
  uint16_t* dW2;
  const int32_t* row_src;    // or null
  const int32_t* row_dst;
  const int32_t* offsets;
  const int32_t* band_expert;
  const int32_t* band_row0;
  const int32_t* band_rows;
  const int32_t* meta;
  int k, d, f, El, group_m;
};

// One operand of a tile. KC: `valid` rows (the non-K dimension) of pitch
// bytes; KS: `valid` K rows, of which the tile takes the columns from base on
// (`chunks` 16-byte chunks of them exist, 16 or 32). idx: row r is row
// idx[r] / div of base.
struct Side {
  const uint8_t* base;
  uint32_t pitch;
  int valid;
  int chunks;
  const int32_t* idx;
  int div;
};

__device__ __forceinline__ int side_row(const Side& s, int r) {
  r = min(r, s.valid - 1);
  return s.idx ? s.idx[r] / s.div : r;
}

// Column-chunk swizzle of a KS stage: the four K rows a transposing read takes
// go to the four 64-byte quarters of a bank line.
__device__ __forceinline__ int ks_swizzle(int kk) { return (kk & 3) << 2; }

// Stage kt of one side into st: ROWS rows of 128 bytes (KC), or 64 K rows of
// 512 bytes (KS). Rows past the valid ones re-read the last.
template <bool KS, int ROWS>
__device__ __forceinline__ void issue_side(const Side& s, int kt, lds_t* st, int w, int lane) {
  if constexpr (KS) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int i = j * 8 + w, kk = 2 * i + (lane >> 5);
      const int chunk = ((lane & 31) ^ ks_swizzle(kk)) & (s.chunks - 1);
      const uint8_t* g = s.base + (size_t)side_row(s, kt * kBK + kk) * s.pitch + (chunk << 4);
      __builtin_amdgcn_global_load_lds(g, st + i * 1024, 16, 0, 0);
    }
  } else {
#pragma unroll
    for (int j = 0; j < ROWS / 64; ++j) {
      const int i = j * 8 + w, r = i * 8 + (lane >> 3);
      const int chunk = (lane & 7) ^ chunk_swizzle<128>(r);
      const uint8_t* g = s.base + (size_t)side_row(s, r) * s.pitch + kt * 128 + (chunk << 4);
      __builtin_amdgcn_global_load_lds(g, st + i * 1024, 16, 0, 0);
    }
  }
}

// Fragment of the 16 K values of step ks and the 32 rows / columns of block
// blk: lane l holds row blk * 32 + l % 32, K values 8 (l / 32) .. + 7.
template <bool KS>
__device__ __forceinline__ bf16x8 fragment(const lds_t* st, int blk, int ks, int lane) {
  const int hi = lane >> 5;
  if constexpr (KS) {
    const int kk = ks * 16 + hi * 8 + ((lane & 15) >> 2);
    const int col = blk * 32 + (lane & 16) + (lane & 3) * 4;
    const lds_t* a = st + kk * 512 + (((col >> 3) ^ ks_swizzle(kk)) << 4) + (col & 4) * 2;
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)a);
    const s16x4 up = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(a + 4 * 512));
    return __builtin_bit_cast(bf16x8, s16x8{lo[0], lo[1], lo[2], lo[3], up[0], up[1], up[2], up[3]});
  } else {
    return *(const lds_bf16x8*)(st + lds_off<128>(blk * 32 + (lane & 31), ks * 2 + hi));
  }
}

__device__ __forceinline__ uint2 pack4(const float (&v)[4]) {
  return make_uint2((uint32_t)f32_to_bf16_rne(v[0]) | ((uint32_t)f32_to_bf16_rne(v[1]) << 16),
                    (uint32_t)f32_to_bf16_rne(v[2]) | ((uint32_t)f32_to_bf16_rne(v[3]) << 16));
}

// A tile: where its operands are and where its results go.
struct BwdTile {
  Side P, Q;
  int ktiles;
  int e;        // expert
  int row0;     // first row (GU, DACT, DX: of the band; DW: first output row)
  int rows;     // valid Q rows / output rows
  int col0;     // first output column
  int cols;     // valid output columns (128 or 256)
};

template <int OP>
__device__ __forceinline__ void store_tile(const BwdParams& P, const BwdTile& t, int m, int c, const float (&v)[4]) {
  const size_t row = (size_t)t.row0 + m;
  const int col = t.col0 + c;
  if constexpr (OP == BWD_GU) {
    *reinterpret_cast<float4*>(P.GU + row * (2 * (size_t)P.f) + col) = make_float4(v[0], v[1], v[2], v[3]);
  } else if constexpr (OP == BWD_DACT) {
    const float* gu = P.GU + row * (2 * (size_t)P.f) + col;
    const float4 g4 = *reinterpret_cast<const float4*>(gu), u4 = *reinterpret_cast<const float4*>(gu + P.f);
    const float g[4] = {g4.x, g4.y, g4.z, g4.w}, u[4] = {u4.x, u4.y, u4.z, u4.w};
    float a[4], dg[4], du[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float s = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(g[i] * -1.4426950408889634f));
      const float gs = g[i] * s;
      a[i] = gs * u[i];
      du[i] = v[i] * gs;
      dg[i] = v[i] * u[i] * (s + gs * (1.0f - s));
    }
    *reinterpret_cast<uint2*>(P.act + row * P.f + col) = pack4(a);
    uint16_t* dh = P.dH + row * (2 * (size_t)P.f) + col;
    *reinterpret_cast<uint2*>(dh) = pack4(dg);
    *reinterpret_cast<uint2*>(dh + P.f) = pack4(du);
  } else if constexpr (OP == BWD_DX) {
    *reinterpret_cast<uint2*>(P.dxs + (size_t)P.row_dst[row] * P.d + col) = pack4(v);
  } else if constexpr (OP == BWD_DW2) {
    *reinterpret_cast<uint2*>(P.dW2 + ((size_t)t.e * P.d + row) * P.f + col) = pack4(v);
  } else {
    *reinterpret_cast<uint2*>(P.dW1 + ((size_t)t.e * 2 * P.f + row) * P.d + col) = pack4(v);
  }
}

// QB: 32-row blocks of the Q side (4 or 8). Each wavefront owns QB / 2 of
// them and 2 of the 8 column blocks.
template <int OP, int QB>
__device__ __forceinline__ void run_bwd_tile(const BwdParams& P, const BwdTile& t, lds_t* lds) {
  constexpr bool PS = p_strided(OP), QS = q_strided(OP);
  constexpr int NM = QB / 2, LD = 4 + (QS ? 4 : QB / 2);
  constexpr int SB = kStageP + kStageQ;
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, wq = w & 1, wp = w >> 1;
  f32x16 acc[NM][2];
#pragma unroll
  for (int a = 0; a < NM; ++a)
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[a][b][i] = 0.0f;

  auto issue = [&](int kt) {
    lds_t* st = lds + (kt & 1) * SB;
    issue_side<PS, kTP>(t.P, kt, st, w, lane);
    issue_side<QS, QB * 32>(t.Q, kt, st + kStageP, w, lane);
  };
  if (t.ktiles > 0) issue(0);
  for (int kt = 0; kt < t.ktiles; ++kt) {
    if (kt + 1 < t.ktiles) {
      issue(kt + 1);
      wait_vmcnt<LD>();
    } else {
      wait_vmcnt<0>();
    }
    lds_barrier();
    lds_t* st = lds + (kt & 1) * SB;
    if constexpr (QS) {
      // K rows past the expert's last: zero on both sides
      const int left = t.P.valid - kt * kBK;
      if (left < kBK) {
        for (int i = left * 32 + (int)threadIdx.x; i < kBK * 32; i += kBwdThreads) {
          *(lds_i32x4*)(st + i * 16) = i32x4{0, 0, 0, 0};
          *(lds_i32x4*)(st + kStageP + i * 16) = i32x4{0, 0, 0, 0};
        }
        lds_barrier();
      }
    }
#pragma unroll
    for (int ks = 0; ks < kBK / 16; ++ks) {
      bf16x8 fp[2], fq[NM];
#pragma unroll
      for (int b = 0; b < 2; ++b) fp[b] = fragment<PS>(st, wp + 4 * b, ks, lane);
#pragma unroll
      for (int a = 0; a < NM; ++a) fq[a] = fragment<QS>(st + kStageP, wq + 2 * a, ks, lane);
#pragma unroll
      for (int a = 0; a < NM; ++a)
#pragma unroll
        for (int b = 0; b < 2; ++b)
          acc[a][b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fp[b], fq[a], acc[a][b], 0, 0, 0);
    }
    lds_barrier();  // the stage may be refilled
  }
  // lane l holds Q row l % 32 of each block and, in elements 4q .. 4q + 3, the
  // columns 8q + 4 (l / 32) + 0..3
#pragma unroll
  for (int a = 0; a < NM; ++a) {
    const int m = (wq + 2 * a) * 32 + (lane & 31);
    if (m >= t.rows) continue;
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      const int c0 = (wp + 4 * b) * 32;
      if (c0 >= t.cols) continue;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float v[4] = {acc[a][b][4 * q], acc[a][b][4 * q + 1], acc[a][b][4 * q + 2], acc[a][b][4 * q + 3]};
        store_tile<OP>(P, t, m, c0 + 8 * q + 4 * (lane >> 5), v);
      }
    }
  }
}

// Tile (p, n) of GU, DACT or DX: row band p, column tile n.
template <int OP>
__device__ __forceinline__ BwdTile band_tile(const BwdParams& P, int p, int n) {
  BwdTile t;
  t.e = P.band_expert[p] & kBandExpertMask;
  t.row0 = P.band_row0[p];
  t.rows = P.band_rows[p];
  t.col0 = n * kTP;
  const uint32_t db = (uint32_t)P.d * 2, fb = (uint32_t)P.f * 2;
  const uint8_t* w1 = P.W1 + (size_t)t.e * (2 * (size_t)P.f) * db;
  const uint8_t* w2 = P.W2 + (size_t)t.e * (size_t)P.d * fb;
  if constexpr (OP == BWD_GU) {
    t.cols = min(kTP, 2 * P.f - t.col0);
    t.ktiles = P.d / kBK;
    t.P = Side{w1 + (size_t)t.col0 * db, db, t.cols, 0, nullptr, 1};
    t.Q = P.row_src ? Side{P.X, db, t.rows, 0, P.row_src + t.row0, P.k}
                    : Side{P.X + (size_t)t.row0 * db, db, t.rows, 0, nullptr, 1};
  } else if constexpr (OP == BWD_DACT) {
    t.cols = min(kTP, P.f - t.col0);
    t.ktiles = P.d / kBK;
    t.P = Side{w2 + (size_t)t.col0 * 2, fb, P.d, t.cols / 8, nullptr, 1};
    t.Q = Side{P.dO, db, t.rows, 0, P.row_dst + t.row0, 1};
  } else {
    t.cols = min(kTP, P.d - t.col0);
    t.ktiles = 2 * P.f / kBK;
    t.P = Side{w1 + (size_t)t.col0 * 2, db, 2 * P.f, t.cols / 8, nullptr, 1};
    t.Q = Side{reinterpret_cast<const uint8_t*>(P.dH) + (size_t)t.row0 * (2 * fb), 2 * fb, t.rows, 0, nullptr, 1};
  }
  return t;
}

// Tile (m, n) of an expert's weight gradient.
template <int OP>
__device__ __forceinline__ BwdTile weight_tile(const BwdParams& P, int e, int m, int n) {
  BwdTile t;
  t.e = e;
  const int r0 = P.offsets[e], cnt = P.offsets[e + 1] - r0;
  const int M = OP == BWD_DW2 ? P.d : 2 * P.f, N = OP == BWD_DW2 ? P.f : P.d;
  t.row0 = m * kBM;
  t.rows = min(kBM, M - t.row0);
  t.col0 = n * kTP;
  t.cols = min(kTP, N - t.col0);
  t.ktiles = (cnt + kBK - 1) / kBK;
  const uint32_t db = (uint32_t)P.d * 2, fb = (uint32_t)P.f * 2;
  if constexpr (OP == BWD_DW2) {
    t.P = Side{reinterpret_cast<const uint8_t*>(P.act) + (size_t)r0 * fb + (size_t)t.col0 * 2, fb, cnt, t.cols / 8,
               nullptr, 1};
    t.Q = Side{P.dO + (size_t)t.row0 * 2, db, cnt, t.rows / 8, P.row_dst + r0, 1};
  } else {
    t.P = P.row_src ? Side{P.X + (size_t)t.col0 * 2, db, cnt, t.cols / 8, P.row_src + r0, P.k}
                    : Side{P.X + (size_t)r0 * db + (size_t)t.col0 * 2, db, cnt, t.cols / 8, nullptr, 1};
    t.Q = Side{reinterpret_cast<const uint8_t*>(P.dH) + (size_t)r0 * (2 * fb) + (size_t)t.row0 * 2, 2 * fb, cnt,
               t.rows / 8, nullptr, 1};
  }
  return t;
}

template <int OP>
__global__ __launch_bounds__(kBwdThreads, 1) void expert_backward_kernel(BwdParams P) {
  __shared__ __attribute__((aligned(1024))) uint8_t smem[2 * (kStageP + kStageQ)];
  lds_t* lds = (lds_t*)smem;
  const int G = gridDim.x, b = blockIdx.x;
  const int lid = (G % 8 == 0) ? (b % 8) * (G / 8) + b / 8 : b;  // consecutive ids on one XCD
  // rejected row indices or offsets: nothing is computed
  if (P.meta[META_ARG_ERR] & ARG_ERR_ALL) return;
  if constexpr (OP <= BWD_DX) {
    const int nb = P.meta[META_P];
    const int width = OP == BWD_GU ? 2 * P.f : OP == BWD_DACT ? P.f : P.d;
    const int N = (width + kTP - 1) / kTP;
    for (int i = lid; i < nb * N; i += G) {
      int p, n;
      raster(i, nb, N, P.group_m, p, n);
      const BwdTile t = band_tile<OP>(P, p, n);
      if (t.rows <= 128) run_bwd_tile<OP, 4>(P, t, lds);
      else run_bwd_tile<OP, 8>(P, t, lds);
    }
  } else {
    const int M = ((OP == BWD_DW2 ? P.d : 2 * P.f) + kBM - 1) / kBM;
    const int N = ((OP == BWD_DW2 ? P.f : P.d) + kTP - 1) / kTP;
    for (int64_t i = lid; i < (int64_t)P.El * M * N; i += G) {
      const int e = (int)(i / (M * N));
      int m, n;
      raster((int)(i - (int64_t)e * M * N), M, N, P.group_m, m, n);
      run_bwd_tile<OP, 8>(P, weight_tile<OP>(P, e, m, n), lds);
    }
  }
}

}  // namespace

BackwardLayout backward_layout(const moe_problem_t& p, const Layout& L) {
  BackwardLayout B;
  size_t o = align_up(L.pub.total, 256);
  auto take = [&](size_t bytes) { size_t at = o; o = align_up(o + bytes, 256); return at; };
  B.gu = take((size_t)L.cap * 2 * p.f * 4);
  B.act = take((size_t)L.cap * p.f * 2);
  B.dh = take((size_t)L.cap * 2 * p.f * 2);
  B.total = o;
  return B;
}

hipError_t launch_expert_backward(const moe_problem_t& p, const Layout& L, char* ws, const void* X,
                                  const int32_t* row_src, const int32_t* offsets, const int32_t* row_dst,
                                  const void* W1, const void* W2, const void* dO, void* dxs, void* dW1, void* dW2,
                                  hipStream_t s) {
  const int G = gemm_grid(p);
  if (G <= 0) return hipErrorInvalidDevice;
  hipError_t e = launch_plan_rows(p, L, ws, offsets, row_src, row_dst, s);
  if (e != hipSuccess) return e;
  const BackwardLayout B = backward_layout(p, L);
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
  P.group_m = 4;
  auto go = [&](auto kern) {
    if (e != hipSuccess) return;
    hipLaunchKernelGGL(kern, dim3(G), dim3(kBwdThreads), 0, s, P);
    e = hipGetLastError();
  };
  go(expert_backward_kernel<BWD_GU>);
  go(expert_backward_kernel<BWD_DACT>);
  go(expert_backward_kernel<BWD_DX>);
  go(expert_backward_kernel<BWD_DW2>);
  go(expert_backward_kernel<BWD_DW1>);
  return e;
}

}  // namespace moe
