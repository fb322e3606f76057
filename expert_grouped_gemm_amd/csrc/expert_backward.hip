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
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
typedef __attribute__((address_space(3))) u32x2 lds_u32x2;

enum BwdOp { BWD_GU = 0, BWD_DACT = 1, BWD_DX = 2, BWD_DW2 = 3, BWD_DW1 = 4 };
__host__ __device__ constexpr bool p_strided(int OP) { return OP != BWD_GU; }
__host__ __device__ constexpr bool q_strided(int OP) { return OP >= BWD_DW2; }

constexpr int kBK = 64;                      // K values per stage
constexpr int kTP = 256;                     // columns (P side) of a tile
constexpr int kBwdThreads = 512;             // 8 wavefronts: 2 (Q) x 4 (P)
constexpr int kLoaders = 4;                  // the last 4 (one per SIMD) issue the ring's loads
constexpr int kStageP = kTP * kBK * 2;       // bytes of the P operand in a stage

// QB: 32-row blocks of the Q side of a tile. A band of up to 256 rows takes
// the smallest of 2, 4, 5, 6 and 8 that holds it: absent blocks cost no loads
// and no MFMAs, and a smaller stage makes a deeper ring (4, 3, 3, 2 and 2
// stages). Measured on the share (counts of 128 on the average, half of them
// above): with 4 and 8 only, GU 501, DACT 267 and DX 542 us.
__host__ __device__ constexpr int stage_q(int QB) { return QB * 32 * kBK * 2; }
__host__ __device__ constexpr int bwd_ring(int QB) { return kGemmLds / (kStageP + stage_q(QB)); }

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

// Column-chunk swizzle of a KS stage: the four K rows a transposing read takes
// go to the four 64-byte quarters of a bank line.
__device__ __forceinline__ int ks_swizzle(int kk) { return (kk & 3) << 2; }

// The ring's loads of one side, as one loader wavefront issues them: NI
// instructions of 1 KiB per stage. An instruction takes 8 rows of 128 bytes
// (KC) or 2 K rows of 512 (KS); loader lw of 4 takes instructions 4 j + lw, so
// its lanes' rows advance by a uniform step from one to the next (and the
// swizzle, which depends on the row modulo 16 or 4, not at all): the address is
// a uniform base plus one 32-bit lane offset.
template <bool KS, int NI>
struct Loads {
  const uint8_t* base;
  uint32_t pitch, lane_off;
  const int32_t* idx;
  int div, valid;
  uint32_t row_off[KS ? 1 : NI];  // KC with rows of their own places
  bool direct;
  int next;                       // KS through idx: this lane's K row of the next stage to issue

  __device__ __forceinline__ void init(const Side& s, int lw, int lane, bool plain_rows) {
    base = s.base;
    pitch = s.pitch;
    idx = s.idx;
    div = s.div;
    valid = s.valid;
    direct = plain_rows;
    if constexpr (KS) {
      const int kk = 2 * lw + (lane >> 5);
      lane_off = (((lane & 31) ^ ks_swizzle(kk)) & (s.chunks - 1)) << 4;
      direct = idx == nullptr;
      next = idx && valid > 0 ? idx[min(lane, valid - 1)] / div : 0;
    } else {
      const int r = lw * 8 + (lane >> 3);
      const uint32_t chunk = ((lane & 7) ^ chunk_swizzle<128>(r)) << 4;
      lane_off = direct ? r * pitch + chunk : chunk;
      if (!direct) {
#pragma unroll
        for (int j = 0; j < NI; ++j) {
          const int row = min(j * 32 + r, valid - 1);
          row_off[j] = (uint32_t)(idx ? idx[row] / div : row) * pitch;
        }
      }
    }
  }

  // NT: with the non-temporal hint
  template <bool NT>
  __device__ __forceinline__ void issue(int kt, lds_t* st, int lw, int lane) {
    if constexpr (KS) {
      const int left = valid - kt * kBK;
      if (direct && left >= kBK) {
        const uint8_t* b0 = base + (size_t)kt * kBK * pitch;
        const uint32_t off = (uint32_t)(2 * lw + (lane >> 5)) * pitch + lane_off;
#pragma unroll
        for (int j = 0; j < NI; ++j)
          __builtin_amdgcn_global_load_lds(b0 + (size_t)j * 8 * pitch + off, st + (4 * j + lw) * 1024, 16, 0, NT ? kCpolNT : 0);
      } else {
        // K row kk of the stage is row `rows` of lane kk: through idx (fetched
        // when the stage before was issued), or, in a last, partial stage,
        // rows past the end re-reading the last (they are zeroed in the LDS)
        const int rows = direct ? kt * kBK + min(lane, left - 1) : next;
        if (!direct) next = idx[min((kt + 1) * kBK + lane, valid - 1)] / div;
#pragma unroll
        for (int j = 0; j < NI; ++j) {
          const int r0 = __builtin_amdgcn_readlane(rows, 8 * j + 2 * lw);
          const int r1 = __builtin_amdgcn_readlane(rows, 8 * j + 2 * lw + 1);
          const uint8_t* g = base + (size_t)(lane < 32 ? r0 : r1) * pitch + lane_off;
          __builtin_amdgcn_global_load_lds(g, st + (4 * j + lw) * 1024, 16, 0, NT ? kCpolNT : 0);
        }
      }
    } else {
      const uint8_t* b0 = base + (size_t)kt * 128;
#pragma unroll
      for (int j = 0; j < NI; ++j) {
        // columns that do not exist (a 128-wide tile) re-read the first ones
        const uint8_t* bj = direct ? b0 + (size_t)(j * 32 < valid ? j : j - NI / 2) * 32 * pitch : b0;
        const uint32_t off = direct ? lane_off : row_off[j] + lane_off;
        __builtin_amdgcn_global_load_lds(bj + off, st + (4 * j + lw) * 1024, 16, 0, NT ? kCpolNT : 0);
      }
    }
  }
};

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

__device__ __forceinline__ uint32_t pack2(float a, float b) {
  return (uint32_t)f32_to_bf16_rne(a) | ((uint32_t)f32_to_bf16_rne(b) << 16);
}

// A tile: where its operands are and where its results go.
struct BwdTile {
  Side P, Q;
  int ktiles;
  int krot;     // stage kt holds K slice (kt + krot) mod ktiles
  int e;        // expert
  int row0;     // first row (GU, DACT, DX: of the band; DW: first output row)
  int rows;     // valid Q rows / output rows
  int col0;     // first output column
  int cols;     // valid output columns (128 or 256)
};

// The results of one 32-row block of a wavefront (its 64 columns), through the
// wavefront's own 8 KiB of the free ring: a lane of the accumulator holds 4
// consecutive columns of a row, whose direct store would write 8 or 16 bytes
// into each of 32 rows; read back, every store writes whole 128-byte lines of
// few rows. m0: the block's first row; dst: this lane's output row of block
// row lane % 32 (DX: its slot).
template <int OP>
__device__ __forceinline__ void store_block(const BwdParams& P, const BwdTile& t, lds_t* wl, const f32x16 (&acc)[2],
                                            int m0, int c0, int dst, int lane) {
  const int lr = lane & 31, hi = lane >> 5;
  if constexpr (OP == BWD_GU || OP == BWD_DACT) {
    // 32 rows of 256 bytes (fp32), 16-byte chunks swizzled by row
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *(lds_f32x4*)(wl + lr * 256 + (((b * 8 + 2 * q + hi) ^ (lr & 15)) << 4)) =
            f32x4{acc[b][4 * q], acc[b][4 * q + 1], acc[b][4 * q + 2], acc[b][4 * q + 3]};
    wave_lds_sync();
    const int c = lane & 15;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int r = j * 4 + (lane >> 4);
      const f32x4 v = *(const lds_f32x4*)(wl + r * 256 + ((c ^ (r & 15)) << 4));
      if (m0 + r >= t.rows) continue;
      const size_t row = (size_t)t.row0 + m0 + r;
      const int col = t.col0 + c0 + c * 4;
      if constexpr (OP == BWD_GU) {
        *reinterpret_cast<float4*>(P.GU + row * (2 * (size_t)P.f) + col) = make_float4(v[0], v[1], v[2], v[3]);
      } else {
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
        *reinterpret_cast<uint2*>(P.act + row * P.f + col) = make_uint2(pack2(a[0], a[1]), pack2(a[2], a[3]));
        uint16_t* dh = P.dH + row * (2 * (size_t)P.f) + col;
        *reinterpret_cast<uint2*>(dh) = make_uint2(pack2(dg[0], dg[1]), pack2(dg[2], dg[3]));
        *reinterpret_cast<uint2*>(dh + P.f) = make_uint2(pack2(du[0], du[1]), pack2(du[2], du[3]));
      }
    }
  } else {
    // 32 rows of 128 bytes (bf16)
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *(lds_u32x2*)(wl + lr * 128 + (((b * 4 + q) ^ (lr & 7)) << 4) + hi * 8) =
            u32x2{pack2(acc[b][4 * q], acc[b][4 * q + 1]), pack2(acc[b][4 * q + 2], acc[b][4 * q + 3])};
    wave_lds_sync();
    const int c = lane & 7;
    const size_t ld = OP == BWD_DW2 ? P.f : P.d;
    uint16_t* out = OP == BWD_DX    ? P.dxs
                    : OP == BWD_DW2 ? P.dW2 + (size_t)t.e * P.d * P.f
                                    : P.dW1 + (size_t)t.e * 2 * P.f * P.d;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int r = j * 8 + (lane >> 3);
      const i32x4 v = *(const lds_i32x4*)(wl + r * 128 + ((c ^ (r & 7)) << 4));
      const size_t row = OP == BWD_DX ? (size_t)__shfl(dst, r, 64) : (size_t)t.row0 + m0 + r;
      i32x4* at = reinterpret_cast<i32x4*>(out + row * ld + t.col0 + c0 + c * 8);
      // the weight gradients are not read again here: past the caches. (DX's
      // rows are, by the dispatch's gradient.) Measured: DW1 of the share 832
      // -> 768 us, of 16384 rows 4640 -> 4300; DX with the hint 3% slower.
      if (m0 + r < t.rows) {
        if constexpr (OP == BWD_DX) *at = v;
        else __builtin_nontemporal_store(v, at);
      }
    }
  }
  wave_lds_sync();
}

// One stage: MFMAs of a wavefront that owns NM Q blocks wq, wq + 2, ... and the
// two P blocks from 2 wp on. The fragments of step ks + 1 are read before the
// MFMAs of step ks.
template <bool PS, bool QS, int NM, class Issue>
__device__ __forceinline__ void bwd_stage(const lds_t* st, int wq, int wp, int lane, f32x16 (&acc)[NM][2],
                                          const Issue& issue) {
  bf16x8 fp[2][2], fq[2][NM];
  auto read = [&](int ks, int buf) {
#pragma unroll
    for (int b = 0; b < 2; ++b) fp[buf][b] = fragment<PS>(st, 2 * wp + b, ks, lane);
#pragma unroll
    for (int a = 0; a < NM; ++a) fq[buf][a] = fragment<QS>(st + kStageP, wq + 2 * a, ks, lane);
  };
  read(0, 0);
#pragma unroll
  for (int ks = 0; ks < kBK / 16; ++ks) {
    if (ks + 1 < kBK / 16) read(ks + 1, (ks + 1) & 1);
    if (ks == 0) issue();
#pragma unroll
    for (int a = 0; a < NM; ++a)
#pragma unroll
      for (int b = 0; b < 2; ++b)
        acc[a][b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fp[ks & 1][b], fq[ks & 1][a], acc[a][b], 0, 0, 0);
  }
}

// One tile. A ring of bwd_ring(QB) stages in the LDS, one barrier per stage:
// it shows the stage complete (each loader has waited for its own loads) and
// every wavefront done with the slot the loaders refill next.
template <int OP, int QB, bool LOADER, int WQ, bool NT>
__device__ __forceinline__ void bwd_tile_body(const BwdParams& P, const BwdTile& t, lds_t* lds) {
  constexpr bool PS = p_strided(OP), QS = q_strided(OP);
  constexpr int NM = (QB + 1 - WQ) / 2, NIQ = QS ? 8 : QB, LD = 8 + NIQ;
  constexpr int S = bwd_ring(QB), SB = kStageP + stage_q(QB);
  static_assert(!QS || QB == 8, "a strided Q side has 256 columns");
  int tid = threadIdx.x;
  asm volatile("" : "+v"(tid));
  const int lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6), wp = w >> 1, lw = w - 4;
  f32x16 acc[NM][2];
#pragma unroll
  for (int a = 0; a < NM; ++a)
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[a][b][i] = 0.0f;

  const int KT = t.ktiles;
  Loads<PS, 8> lp;
  Loads<QS, NIQ> lq;
  auto issue = [&](int stage, int slot) {
    int kt = stage;
    if constexpr (!QS) kt = stage + t.krot >= KT ? stage + t.krot - KT : stage + t.krot;
    lp.template issue<NT>(kt, lds + slot * SB, lw, lane);
    lq.template issue<false>(kt, lds + slot * SB + kStageP, lw, lane);
  };
  if constexpr (LOADER) {
    lp.init(t.P, lw, lane, true);
    lq.init(t.Q, lw, lane, false);
#pragma unroll
    for (int s = 0; s < S - 1; ++s)
      if (s < KT) issue(s, s);
  }
  int rd = 0, wr = S - 1;
  for (int kt = 0; kt < KT; ++kt) {
    if constexpr (LOADER) {
      // the stages after kt that are in flight: S - 2, near the end fewer
      const int after = KT - 1 - kt;
      if (after >= S - 2) wait_vmcnt<(S - 2) * LD>();
      else if (S > 3 && after == 1) wait_vmcnt<LD>();
      else wait_vmcnt<0>();
    }
    lds_barrier();
    lds_t* st = lds + rd * SB;
    if constexpr (QS) {
      // K rows past the expert's last: zero on both sides
      const int left = t.P.valid - kt * kBK;
      if (left < kBK) {
        for (int i = left * 32 + tid; i < kBK * 32; i += kBwdThreads) {
          *(lds_i32x4*)(st + i * 16) = i32x4{0, 0, 0, 0};
          *(lds_i32x4*)(st + kStageP + i * 16) = i32x4{0, 0, 0, 0};
        }
        lds_barrier();
      }
    }
    bwd_stage<PS, QS, NM>(st, WQ, wp, lane, acc, [&]() {
      if constexpr (LOADER) {
        if (kt + S - 1 < KT) issue(kt + S - 1, wr);
      }
    });
    rd = rd + 1 == S ? 0 : rd + 1;
    wr = wr + 1 == S ? 0 : wr + 1;
  }
  lds_barrier();  // the ring is free
  int dst[NM];
  if constexpr (OP == BWD_DX) {
#pragma unroll
    for (int a = 0; a < NM; ++a) {
      const int m = (WQ + 2 * a) * 32 + (lane & 31);
      dst[a] = m < t.rows ? P.row_dst[t.row0 + m] : 0;
    }
  }
  if (wp * 64 < t.cols) {
#pragma unroll
    for (int a = 0; a < NM; ++a) {
      const int m0 = (WQ + 2 * a) * 32;
      if (m0 < t.rows) store_block<OP>(P, t, lds + w * 8192, acc[a], m0, wp * 64, OP == BWD_DX ? dst[a] : 0, lane);
    }
  }
  lds_barrier();  // ... for the next tile's loads
}

// A wavefront's role: loader or not, and its row of the 2 x 4 wavefront grid.
template <int OP, int QB, bool NT>
__device__ __forceinline__ void run_bwd_tile(const BwdParams& P, const BwdTile& t, lds_t* lds) {
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (w >= 8 - kLoaders) {
    if (w & 1) bwd_tile_body<OP, QB, true, 1, NT>(P, t, lds);
    else bwd_tile_body<OP, QB, true, 0, NT>(P, t, lds);
  } else {
    if (w & 1) bwd_tile_body<OP, QB, false, 1, NT>(P, t, lds);
    else bwd_tile_body<OP, QB, false, 0, NT>(P, t, lds);
  }
}

template <int OP, bool NT>
__device__ __forceinline__ void run_band_tile(const BwdParams& P, const BwdTile& t, lds_t* lds) {
  if (t.rows <= 64) run_bwd_tile<OP, 2, NT>(P, t, lds);
  else if (t.rows <= 128) run_bwd_tile<OP, 4, NT>(P, t, lds);
  else if (t.rows <= 160) run_bwd_tile<OP, 5, NT>(P, t, lds);
  else if (t.rows <= 192) run_bwd_tile<OP, 6, NT>(P, t, lds);
  else run_bwd_tile<OP, 8, NT>(P, t, lds);
}

// Tile (p, n) of GU, DACT or DX: row band p, column tile n.
template <int OP>
__device__ __forceinline__ BwdTile band_tile(const BwdParams& P, int p, int n) {
  BwdTile t;
  t.e = P.band_expert[p] & kBandExpertMask;
  // bands of different experts run together: DACT starts their K slices apart,
  // or all of them stream the same HBM channels (see kKRot; the share's DACT
  // 266 -> 251 us, nothing to gain for GU and DX)
  const bool once = (P.band_expert[p] & kBandSingle) != 0;
  t.row0 = P.band_row0[p];
  t.rows = P.band_rows[p];
  t.col0 = n * kTP;
  const uint32_t db = (uint32_t)P.d * 2, fb = (uint32_t)P.f * 2;
  const uint8_t* w1 = P.W1 + (size_t)t.e * (2 * (size_t)P.f) * db;
  const uint8_t* w2 = P.W2 + (size_t)t.e * (size_t)P.d * fb;
  if constexpr (OP == BWD_GU) {
    t.cols = min(kTP, 2 * P.f - t.col0);
    t.ktiles = P.d / kBK;
    t.krot = 0;
    t.P = Side{w1 + (size_t)t.col0 * db, db, t.cols, 0, nullptr, 1};
    t.Q = P.row_src ? Side{P.X, db, t.rows, 0, P.row_src + t.row0, P.k}
                    : Side{P.X + (size_t)t.row0 * db, db, t.rows, 0, nullptr, 1};
  } else if constexpr (OP == BWD_DACT) {
    t.cols = min(kTP, P.f - t.col0);
    t.ktiles = P.d / kBK;
    t.krot = once ? t.e * kKRot % t.ktiles : 0;
    t.P = Side{w2 + (size_t)t.col0 * 2, fb, P.d, t.cols / 8, nullptr, 1};
    t.Q = Side{P.dO, db, t.rows, 0, P.row_dst + t.row0, 1};
  } else {
    t.cols = min(kTP, P.d - t.col0);
    t.ktiles = 2 * P.f / kBK;
    t.krot = 0;
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
  __shared__ __attribute__((aligned(1024))) uint8_t smem[kGemmLds];
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
      // weights of an expert with one band are read once per launch (see
      // streams_once)
      if (P.band_expert[p] & kBandSingle) run_band_tile<OP, true>(P, t, lds);
      else run_band_tile<OP, false>(P, t, lds);
    }
  } else {
    const int M = ((OP == BWD_DW2 ? P.d : 2 * P.f) + kBM - 1) / kBM;
    const int N = ((OP == BWD_DW2 ? P.f : P.d) + kTP - 1) / kTP;
    for (int64_t i = lid; i < (int64_t)P.El * M * N; i += G) {
      const int e = (int)(i / (M * N));
      int m, n;
      raster((int)(i - (int64_t)e * M * N), M, N, P.group_m, m, n);
      run_bwd_tile<OP, 8, false>(P, weight_tile<OP>(P, e, m, n), lds);
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
