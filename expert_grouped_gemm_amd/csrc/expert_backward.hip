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
//
// Measured (us; rates in TFLOP/s or TB/s of the bytes the product cannot do
// without). The share (4096 rows of 32 experts, d = 7168, f = 2048), bound by HBM
// but for the weight gradients, whose tiles of two to five stages are half setup
// and stores: GU 356 (5.3 TB/s), DACT 183 (5.1), DX 386 (4.9), DW2 291 (3.2), DW1 590
// (3.2). 16384 rows of 8 experts, d = 4096, f = 14336, bound by the MFMA units, busy
// 59% of the time at the clock the chip holds under them, and the loads and LDS
// reads that do not overlap with them: GU 3564 (1080), DACT 2282 (843, with the
// epilogue's 3.3 GB), DX 3408 (1129), DW2 1906 (1009), DW1 3751 (1026).
// These last two (WAVES = 8) spill 16 registers, output row numbers of their
// epilogue that one loader role reloads between its stores; no accumulator and
// nothing of a K loop is spilled, and no other kernel here spills any.
// Not kept: a ring of 32-wide K stages with the loads spread over the MFMAs and
// fragments read across the barrier (20% slower) and every wavefront loading
// (6%), both while the loads still went through the builtin (see dma16); the
// next weight-gradient tile's loads issued before the stores of the last, and
// DACT's gate and up values all fetched ahead of its stores (registers spilled).
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
constexpr int kBwdThreads = 512;             // 8 wavefronts: 2 (Q) x 4 (P)
constexpr int kLoaders = 4;                  // the last 4 (one per SIMD) issue the ring's loads

// A tile has PB 32-column blocks (8, or 4 in the last, partly idle round of the
// persistent grid: twice as many tiles of half the width) and QB 32-row blocks.
// A band of up to 256 rows takes the smallest of 2, 4, 5, 6 and 8 that holds
// it: absent blocks cost no loads and no MFMAs, and a smaller stage makes a
// deeper ring. Measured on the share (counts of 128 on the average, half of them
// above): with 4 and 8 only, GU 501, DACT 267 and DX 542 us; with all, 409, 266
// and 515.
__host__ __device__ constexpr int stage_bytes_of(int blocks) { return blocks * 32 * kBK * 2; }
__host__ __device__ constexpr int bwd_ring(int PB, int QB) {
  const int s = kGemmLds / stage_bytes_of(PB + QB);
  return s > 6 ? 6 : s;
}

// Rows per expert up to which weight_backward_short_kernel runs. Whole calls
// with it / with the other kernel and its copies, us:
//   rows per expert              128          256          512         1024          2048
//   32 experts, d 7168, f 2048   1812 / 1932  3340 / 3335  5257 / 5090  9179 / 8623  17264 / 15646
//   8 of 4096, 14336                          3444 / 3401  5458 / 5182  9294 / 8576  17291 / 15308
//   16 of 2048, 1024              183 / 203    279 / 295    453 / 458    767 / 763    1402 / 1359
// They cross between 256 and 640 rows; at 512 the two differ by at most 5%. The
// rows are the router's mean, T k / E_global, as the host does not see the call's
// offsets: a share that holds the favoured experts may take the short kernel for
// long ones (4 of 64 experts, a Zipf router, 8192 tokens: 2119 / 1923).
constexpr int kShortRows = 512;

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
  uint16_t* Xp;              // long experts: the token rows and the output gradients in expert order
  uint16_t* dOp;             // [cap, d] each
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

// One direct global -> LDS load of 16 bytes per lane: lane l's bytes at base +
// off land at st + 16 l. Written out because the compiler, which cannot tell
// the transposing LDS reads that follow from the bytes still under way, waits
// for every load it issued through the builtin before the next such read:
// the loaders then stood still in every stage until the next stage's data had
// come, and the ring overlapped nothing. The load has no register result; its
// completion is waited for in wait_vmcnt() before the barrier that publishes
// the stage. The wait states between are the instruction's own to keep: one
// after the write of M0, and five after a vector instruction (readfirstlane)
// that wrote the scalar base.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"  // M0 is reserved, and named as overwritten
template <bool NT>
__device__ __forceinline__ void dma16(const uint8_t* base, uint32_t off, lds_t* st) {
  const uint64_t b = reinterpret_cast<uint64_t>(base);  // a uniform value, as the instruction's scalar base
  const uint64_t sb = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)b) |
                      ((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(b >> 32)) << 32);
  const uint32_t m0 = __builtin_amdgcn_readfirstlane((int)(uint32_t)(uintptr_t)st);
  if constexpr (NT)
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tglobal_load_lds_dwordx4 %1, %2 nt" ::"s"(m0), "v"(off), "s"(sb)
                 : "memory", "m0");
  else
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(m0), "v"(off), "s"(sb)
                 : "memory", "m0");
}
#pragma clang diagnostic pop

// The ring's loads of one side, as one loader wavefront issues them: NI
// instructions of 1 KiB per stage. An instruction takes 8 rows of 128 bytes
// (KC), 2 K rows of 512 bytes or 4 of 256 (KS); loader lw of 4 takes
// instructions 4 j + lw, so its lanes' rows advance by a uniform step from one
// to the next, and the swizzle, which depends on the row modulo 16 or 4, stays:
// an address is a uniform base plus one 32-bit lane offset.

// A weight matrix: every row exists, at its own place. Of a KS tile of 256
// columns only 128 may exist: the others re-read those (the rows of a KC tile
// all exist: 2f is a multiple of 256). NT: with the non-temporal hint.
template <bool KS, int BLOCKS, bool NT>
struct WeightLoads {
  static constexpr int NI = BLOCKS;                       // BLOCKS * 4 KiB over 4 loaders
  static constexpr int CPR = KS ? BLOCKS * 4 : 8;         // 16-byte chunks per LDS row
  static constexpr int RPI = 64 / CPR;                    // rows per instruction
  const uint8_t* base;
  uint32_t pitch, lane_off;

  __device__ __forceinline__ void init(const Side& s, int lw, int lane) {
    base = s.base;
    pitch = s.pitch;
    const int r = lw * RPI + lane / CPR, c = lane % CPR;
    if constexpr (KS) lane_off = r * pitch + (((c ^ ks_swizzle(r)) & (s.chunks - 1)) << 4);
    else lane_off = r * pitch + ((c ^ chunk_swizzle<128>(r)) << 4);
  }
  __device__ __forceinline__ void issue(int kt, lds_t* st, int lw, int) {
    const uint8_t* b0 = base + (KS ? (size_t)kt * kBK * pitch : (size_t)kt * (kBK * 2));
#pragma unroll
    for (int j = 0; j < NI; ++j)
      dma16<NT>(b0 + (size_t)(j * 4 * RPI) * pitch, lane_off, st + (4 * j + lw) * 1024);
  }
};

// Rows of a band (KC), perhaps through idx, the last one repeated.
template <int BLOCKS>
struct BandLoads {
  static constexpr int NI = BLOCKS;
  const uint8_t* base;
  uint32_t off[NI];

  __device__ __forceinline__ void init(const Side& s, int lw, int lane) {
    base = s.base;
    const int r = lw * 8 + (lane >> 3);
#pragma unroll
    for (int j = 0; j < NI; ++j) {
      const int row = min(j * 32 + r, s.valid - 1);
      off[j] = (uint32_t)(s.idx ? s.idx[row] / s.div : row) * s.pitch + (((lane & 7) ^ chunk_swizzle<128>(r)) << 4);
    }
  }
  __device__ __forceinline__ void issue(int kt, lds_t* st, int lw, int) {
    const uint8_t* b0 = base + (size_t)kt * (kBK * 2);
#pragma unroll
    for (int j = 0; j < NI; ++j) dma16<false>(b0, off[j], st + (4 * j + lw) * 1024);
  }
};

// An expert's rows as K (KS), BK of them a stage, perhaps through idx. Lane kk
// holds the offset of K row kk of a stage for all lanes; rows past the last
// re-read it (the stage's LDS rows are zeroed). Offsets through idx fit 32 bits
// (the problem limits keep T * d and cap * d below 2^31 elements) and are
// fetched ahead: those of a tile's first S stages together, a later stage's
// when the stage before it is issued. Without idx they count from the stage's
// first row.
// IDX: the rows may be looked up (otherwise they stand in expert order).
template <int BLOCKS, int BK, int S, bool IDX>
struct RowLoads {
  static constexpr int CPR = BLOCKS * 4, RPI = 64 / CPR, NI = BK * BLOCKS / 64;
  const uint8_t* base;
  uint32_t pitch, lane_off, ahead[S];
  const int32_t* idx;
  int div, valid;

  __device__ __forceinline__ uint32_t look_up(int kt, int lane) const {
    return (uint32_t)(idx[min(kt * BK + (lane & (BK - 1)), valid - 1)] / div) * pitch;
  }
  __device__ __forceinline__ void init(const Side& s, int lw, int lane) {
    base = s.base;
    pitch = s.pitch;
    idx = IDX ? s.idx : nullptr;
    div = s.div;
    valid = s.valid;
    const int kk = lw * RPI + lane / CPR;
    lane_off = (((lane % CPR) ^ ks_swizzle(kk)) & (s.chunks - 1)) << 4;
    if (idx && valid > 0) {
#pragma unroll
      for (int i = 0; i < S; ++i) ahead[i] = look_up(i, lane);
    }
  }
  __device__ __forceinline__ void issue_rows(int kt, uint32_t rows, lds_t* st, int lw, int lane) {
    const int kk = lw * RPI + lane / CPR, left = valid - kt * BK;
    const uint8_t* b0 = idx ? base : base + (size_t)kt * BK * pitch;
    if (!idx && left >= BK) {
      const uint32_t off = kk * pitch + lane_off;
#pragma unroll
      for (int j = 0; j < NI; ++j)
        dma16<false>(b0 + (size_t)(4 * j * RPI) * pitch, off, st + (4 * j + lw) * 1024);
      return;
    }
    if (!idx) rows = min(lane & (BK - 1), left - 1) * pitch;
#pragma unroll
    for (int j = 0; j < NI; ++j)
      dma16<false>(b0, (uint32_t)__shfl((int)rows, 4 * j * RPI + kk, 64) + lane_off, st + (4 * j + lw) * 1024);
  }
  // stage kt < S, of the tile's first ones
  __device__ __forceinline__ void issue_first(int kt, lds_t* st, int lw, int lane) {
    issue_rows(kt, ahead[kt], st, lw, lane);
    if (kt == S - 1 && idx) ahead[0] = look_up(S, lane);
  }
  // a later stage
  __device__ __forceinline__ void issue(int kt, lds_t* st, int lw, int lane) {
    const uint32_t rows = ahead[0];
    if (idx && (kt + 1) * BK < valid) ahead[0] = look_up(kt + 1, lane);
    issue_rows(kt, rows, st, lw, lane);
  }
};

// Fragment of the 16 K values of step ks and the 32 rows / columns of block
// blk: lane l holds row blk * 32 + l % 32, K values 8 (l / 32) .. + 7. BLOCKS:
// the side's blocks (KS: its LDS rows hold 64 bytes of each).
template <bool KS, int BLOCKS>
__device__ __forceinline__ bf16x8 fragment(const lds_t* st, int blk, int ks, int lane) {
  const int hi = lane >> 5;
  if constexpr (KS) {
    const int kk = ks * 16 + hi * 8 + ((lane & 15) >> 2);
    const int col = blk * 32 + (lane & 16) + (lane & 3) * 4;
    const lds_t* a = st + kk * (BLOCKS * 64) + (((col >> 3) ^ ks_swizzle(kk)) << 4) + (col & 4) * 2;
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)a);
    const s16x4 up = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(a + 4 * BLOCKS * 64));
    return __builtin_bit_cast(bf16x8, s16x8{lo[0], lo[1], lo[2], lo[3], up[0], up[1], up[2], up[3]});
  } else {
    return *(const lds_bf16x8*)(st + lds_off<128>(blk * 32 + (lane & 31), ks * 2 + hi));
  }
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

// The results of one 32-row block of a wavefront (its NB * 32 columns), through
// the wavefront's own LDS: a lane of the accumulator holds 4 consecutive columns
// of a row, whose direct store would write 8 or 16 bytes into each of 32 rows;
// read back, every store writes whole 128-byte lines of few rows (64 bytes with
// NB = 1). m0: the block's first row; dst: this lane's output row of block row
// lane % 32 (DX: its slot).
template <int OP, int NB>
__device__ __forceinline__ void store_block(const BwdParams& P, const BwdTile& t, lds_t* wl, const f32x16 (&acc)[NB],
                                            int m0, int c0, int dst, int lane) {
  const int lr = lane & 31, hi = lane >> 5;
  if constexpr (OP == BWD_GU || OP == BWD_DACT) {
    constexpr int C = 8 * NB;  // 16-byte chunks of a row (fp32), swizzled by row
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *(lds_f32x4*)(wl + lr * (C * 16) + (((b * 8 + 2 * q + hi) ^ (lr & (C - 1))) << 4)) =
            f32x4{acc[b][4 * q], acc[b][4 * q + 1], acc[b][4 * q + 2], acc[b][4 * q + 3]};
    wave_lds_sync();
    const int c = lane & (C - 1);
#pragma unroll
    for (int j = 0; j < C / 2; ++j) {
      const int r = j * (64 / C) + lane / C;
      const f32x4 v = *(const lds_f32x4*)(wl + r * (C * 16) + ((c ^ (r & (C - 1))) << 4));
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
        *reinterpret_cast<uint2*>(P.act + row * P.f + col) = make_uint2(pack_bf16(a[0], a[1]), pack_bf16(a[2], a[3]));
        uint16_t* dh = P.dH + row * (2 * (size_t)P.f) + col;
        *reinterpret_cast<uint2*>(dh) = make_uint2(pack_bf16(dg[0], dg[1]), pack_bf16(dg[2], dg[3]));
        *reinterpret_cast<uint2*>(dh + P.f) = make_uint2(pack_bf16(du[0], du[1]), pack_bf16(du[2], du[3]));
      }
    }
  } else {
    constexpr int C = 4 * NB;  // 16-byte chunks of a row (bf16)
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *(lds_u32x2*)(wl + lr * (C * 16) + (((b * 4 + q) ^ (lr & (C - 1))) << 4) + hi * 8) =
            u32x2{pack_bf16(acc[b][4 * q], acc[b][4 * q + 1]), pack_bf16(acc[b][4 * q + 2], acc[b][4 * q + 3])};
    wave_lds_sync();
    const int c = lane & (C - 1);
    const size_t ld = OP == BWD_DW2 ? P.f : P.d;
    uint16_t* out = OP == BWD_DX    ? P.dxs
                    : OP == BWD_DW2 ? P.dW2 + (size_t)t.e * P.d * P.f
                                    : P.dW1 + (size_t)t.e * 2 * P.f * P.d;
#pragma unroll
    for (int j = 0; j < C / 2; ++j) {
      const int r = j * (64 / C) + lane / C;
      const i32x4 v = *(const lds_i32x4*)(wl + r * (C * 16) + ((c ^ (r & (C - 1))) << 4));
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

// One stage: MFMAs of a wavefront that owns NM Q blocks wq, wq + QSTEP, ... and the
// P blocks from wp * PB / 4 on. The fragments of step ks + 1 are read before
// the MFMAs of step ks; issue() issues the loader's loads behind the first.
template <bool PS, bool QS, int PB, int QB, int NM, int BK = kBK, int QSTEP = 2, class Issue>
__device__ __forceinline__ void bwd_stage(const lds_t* st, int wq, int wp, int lane, f32x16 (&acc)[NM][PB / 4],
                                          const Issue& issue) {
  constexpr int NB = PB / 4;
  bf16x8 fp[2][NB], fq[2][NM];
  auto read = [&](int ks, int buf) {
#pragma unroll
    for (int b = 0; b < NB; ++b) fp[buf][b] = fragment<PS, PB>(st, NB * wp + b, ks, lane);
#pragma unroll
    for (int a = 0; a < NM; ++a) fq[buf][a] = fragment<QS, QB>(st + PB * 64 * BK, wq + QSTEP * a, ks, lane);
  };
  read(0, 0);
#pragma unroll
  for (int ks = 0; ks < BK / 16; ++ks) {
    if (ks + 1 < BK / 16) read(ks + 1, (ks + 1) & 1);
    if (ks == 0) issue();
#pragma unroll
    for (int a = 0; a < NM; ++a)
#pragma unroll
      for (int b = 0; b < NB; ++b)
        acc[a][b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fp[ks & 1][b], fq[ks & 1][a], acc[a][b], 0, 0, 0);
  }
}

template <int NM, int NB>
__device__ __forceinline__ void clear_acc(f32x16 (&acc)[NM][NB]) {
#pragma unroll
  for (int a = 0; a < NM; ++a)
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[a][b][i] = 0.0f;
}

// Wait until at most min(N, n) stages of LD loads are in flight.
template <int LD, int N>
__device__ __forceinline__ void wait_stages(int n) {
  if constexpr (N == 0) wait_vmcnt<0>();
  else if (n >= N) wait_vmcnt<N * LD>();
  else wait_stages<LD, N - 1>(n);
}

// A tile of GU, DACT or DX. A ring of bwd_ring() stages in the LDS, one barrier
// per stage: it shows the stage complete (each loader has waited for its own
// loads) and every wavefront done with the slot the loaders refill next.
template <int OP, int PB, int QB, bool LOADER, int WQ, bool NT>
__device__ __forceinline__ void band_tile_body(const BwdParams& P, const BwdTile& t, lds_t* lds) {
  constexpr bool PS = p_strided(OP);
  constexpr int NM = (QB + 1 - WQ) / 2, NB = PB / 4, LD = PB + QB;
  constexpr int S = bwd_ring(PB, QB), SB = stage_bytes_of(PB + QB);
  static_assert(S >= 2 && (S - 2) * LD < 64, "ring depth");
  int tid = threadIdx.x;
  asm volatile("" : "+v"(tid));
  const int lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6), wp = w >> 1, lw = w - 4;
  f32x16 acc[NM][NB];
  clear_acc(acc);

  const int KT = t.ktiles;
  WeightLoads<PS, PB, NT> lp;
  BandLoads<QB> lq;
  auto issue = [&](int stage, int slot) {
    const int kt = stage + t.krot >= KT ? stage + t.krot - KT : stage + t.krot;
    lp.issue(kt, lds + slot * SB, lw, lane);
    lq.issue(kt, lds + slot * SB + stage_bytes_of(PB), lw, lane);
  };
  if constexpr (LOADER) {
    lp.init(t.P, lw, lane);
    lq.init(t.Q, lw, lane);
#pragma unroll
    for (int s = 0; s < S - 1; ++s)
      if (s < KT) issue(s, s);
  }
  int rd = 0, wr = S - 1;
  for (int kt = 0; kt < KT; ++kt) {
    if constexpr (LOADER) wait_stages<LD, S - 2>(KT - 1 - kt);
    lds_barrier();
    bwd_stage<PS, false, PB, QB, NM>(lds + rd * SB, WQ, wp, lane, acc, [&]() {
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
  if (wp * (NB * 32) < t.cols) {
#pragma unroll
    for (int a = 0; a < NM; ++a) {
      const int m0 = (WQ + 2 * a) * 32;
      if (m0 < t.rows)
        store_block<OP, NB>(P, t, lds + w * 8192, acc[a], m0, wp * (NB * 32), OP == BWD_DX ? dst[a] : 0, lane);
    }
  }
  lds_barrier();  // ... for the next tile's loads
}

// A wavefront's role: loader or not, and its row of the 2 x 4 wavefront grid.
template <int OP, int PB, int QB, bool NT>
__device__ __forceinline__ void run_roles(const BwdParams& P, const BwdTile& t, lds_t* lds) {
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (w >= 8 - kLoaders) {
    if (w & 1) band_tile_body<OP, PB, QB, true, 1, NT>(P, t, lds);
    else band_tile_body<OP, PB, QB, true, 0, NT>(P, t, lds);
  } else {
    if (w & 1) band_tile_body<OP, PB, QB, false, 1, NT>(P, t, lds);
    else band_tile_body<OP, PB, QB, false, 0, NT>(P, t, lds);
  }
}

template <int OP, int PB, bool NT>
__device__ __forceinline__ void run_band_tile(const BwdParams& P, const BwdTile& t, lds_t* lds) {
  if (t.rows <= 64) run_roles<OP, PB, 2, NT>(P, t, lds);
  else if (t.rows <= 128) run_roles<OP, PB, 4, NT>(P, t, lds);
  else if (t.rows <= 160) run_roles<OP, PB, 5, NT>(P, t, lds);
  else if (t.rows <= 192) run_roles<OP, PB, 6, NT>(P, t, lds);
  else run_roles<OP, PB, 8, NT>(P, t, lds);
}

// Tile (p, n) of GU, DACT or DX: row band p, column tile n of `width` columns.
template <int OP>
__device__ __forceinline__ BwdTile band_tile(const BwdParams& P, int p, int n, int width) {
  BwdTile t;
  t.e = P.band_expert[p] & kBandExpertMask;
  // bands of different experts run together: DACT starts their K slices apart,
  // or all of them stream the same HBM channels (see kKRot; the share's DACT
  // 266 -> 251 us, nothing to gain for GU and DX)
  const bool once = (P.band_expert[p] & kBandSingle) != 0;
  t.row0 = P.band_row0[p];
  t.rows = P.band_rows[p];
  t.col0 = n * width;
  const uint32_t db = (uint32_t)P.d * 2, fb = (uint32_t)P.f * 2;
  const uint8_t* w1 = P.W1 + (size_t)t.e * (2 * (size_t)P.f) * db;
  const uint8_t* w2 = P.W2 + (size_t)t.e * (size_t)P.d * fb;
  if constexpr (OP == BWD_GU) {
    t.cols = min(width, 2 * P.f - t.col0);
    t.ktiles = P.d / kBK;
    t.krot = 0;
    t.P = Side{w1 + (size_t)t.col0 * db, db, t.cols, 0, nullptr, 1};
    t.Q = P.row_src ? Side{P.X, db, t.rows, 0, P.row_src + t.row0, P.k}
                    : Side{P.X + (size_t)t.row0 * db, db, t.rows, 0, nullptr, 1};
  } else if constexpr (OP == BWD_DACT) {
    t.cols = min(width, P.f - t.col0);
    t.ktiles = P.d / kBK;
    t.krot = once ? t.e * kKRot % t.ktiles : 0;
    t.P = Side{w2 + (size_t)t.col0 * 2, fb, P.d, t.cols / 8, nullptr, 1};
    t.Q = Side{P.dO, db, t.rows, 0, P.row_dst + t.row0, 1};
  } else {
    t.cols = min(width, P.d - t.col0);
    t.ktiles = 2 * P.f / kBK;
    t.krot = 0;
    t.P = Side{w1 + (size_t)t.col0 * 2, db, 2 * P.f, t.cols / 8, nullptr, 1};
    t.Q = Side{reinterpret_cast<const uint8_t*>(P.dH) + (size_t)t.row0 * (2 * fb), 2 * fb, t.rows, 0, nullptr, 1};
  }
  return t;
}

// Rows [first, first + count) of a band's tile.
__device__ __forceinline__ void take_rows(BwdTile& t, int first, int count) {
  t.rows = min(count, t.rows - first);
  t.row0 += first;
  t.Q.valid = t.rows;
  if (t.Q.idx) t.Q.idx += first;
  else t.Q.base += (size_t)first * t.Q.pitch;
}

// Tile (m, n) of an expert's weight gradient, TM rows high. IDX: the rows of X
// and dO are looked up; otherwise they are read from their ordered copies.
template <int OP, bool IDX>
__device__ __forceinline__ BwdTile weight_tile(const BwdParams& P, int e, int m, int n, int TM) {
  BwdTile t;
  t.e = e;
  const int r0 = P.offsets[e], cnt = P.offsets[e + 1] - r0;
  const int M = OP == BWD_DW2 ? P.d : 2 * P.f, N = OP == BWD_DW2 ? P.f : P.d;
  t.row0 = m * TM;
  t.rows = min(TM, M - t.row0);
  t.col0 = n * 256;
  t.cols = min(256, N - t.col0);
  const uint32_t db = (uint32_t)P.d * 2, fb = (uint32_t)P.f * 2;
  if constexpr (OP == BWD_DW2) {
    t.P = Side{reinterpret_cast<const uint8_t*>(P.act) + (size_t)r0 * fb + (size_t)t.col0 * 2, fb, cnt, t.cols / 8,
               nullptr, 1};
    t.Q = IDX ? Side{P.dO + (size_t)t.row0 * 2, db, cnt, t.rows / 8, P.row_dst + r0, 1}
              : Side{reinterpret_cast<const uint8_t*>(P.dOp) + (size_t)r0 * db + (size_t)t.row0 * 2, db, cnt,
                     t.rows / 8, nullptr, 1};
  } else {
    const uint8_t* rows = IDX || !P.row_src ? P.X : reinterpret_cast<const uint8_t*>(P.Xp);
    t.P = IDX && P.row_src ? Side{P.X + (size_t)t.col0 * 2, db, cnt, t.cols / 8, P.row_src + r0, P.k}
                           : Side{rows + (size_t)r0 * db + (size_t)t.col0 * 2, db, cnt, t.cols / 8, nullptr, 1};
    t.Q = Side{reinterpret_cast<const uint8_t*>(P.dH) + (size_t)r0 * (2 * fb) + (size_t)t.row0 * 2, 2 * fb, cnt,
               t.rows / 8, nullptr, 1};
  }
  return t;
}

// DW1 or DW2: a workgroup's tiles, one after the other.
// WAVES = 8: 256 x 256 tiles, a ring of two stages of 64 K rows, one workgroup
// per CU, the last four wavefronts load. WAVES = 4: 128 x 256 tiles, three
// stages of 32 K rows, two workgroups per CU (72 KiB of LDS each), every
// wavefront loads: for experts of few rows, whose tiles are a few stages long
// and otherwise setup, waits and stores, which the two workgroups overlap.
// A tile starts with the whole ring in flight; from step 1 on, each step
// refills the slot of the step before it.
template <int OP, int WAVES, bool LOADER, int WQ>
__device__ __forceinline__ void weight_tiles_body(const BwdParams& P, lds_t* lds, int lid, int G) {
  constexpr int QB = WAVES, BK = WAVES == 8 ? 64 : 32, S = WAVES == 8 ? 2 : 3, NW = WAVES / 4, TM = QB * 32;
  constexpr int SB = (8 + QB) * 64 * BK;  // stage bytes: 64 of each block per K row
  int tid = threadIdx.x;
  asm volatile("" : "+v"(tid));
  const int lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6), wp = w / NW, lw = w - (WAVES - 4);
  const int rows_all = OP == BWD_DW2 ? P.d : 2 * P.f, cols_all = OP == BWD_DW2 ? P.f : P.d;
  const int M = (rows_all + TM - 1) / TM, N = (cols_all + 255) / 256;
  const int64_t total = (int64_t)P.El * M * N;
  typedef RowLoads<8, BK, S, WAVES == 4> LoadsP;
  typedef RowLoads<QB, BK, S, WAVES == 4> LoadsQ;
  constexpr int LD = LoadsP::NI + LoadsQ::NI;
  for (int64_t i = lid; i < total; i += G) {
    const int e = (int)(i / (M * N));
    int m, n;
    raster((int)(i - (int64_t)e * M * N), M, N, P.group_m, m, n);
    const BwdTile t = weight_tile<OP, WAVES == 4>(P, e, m, n, TM);
    const int KT = (t.P.valid + BK - 1) / BK;
    LoadsP lp;
    LoadsQ lq;
    if constexpr (LOADER) {
      lp.init(t.P, lw, lane);
      lq.init(t.Q, lw, lane);
#pragma unroll
      for (int s = 0; s < S; ++s)
        if (s < KT) {
          lp.issue_first(s, lds + s * SB, lw, lane);
          lq.issue_first(s, lds + s * SB + 8 * 64 * BK, lw, lane);
        }
    }
    f32x16 acc[4][2];
    clear_acc(acc);
    int rd = 0, wr = S - 1;
    for (int kt = 0; kt < KT; ++kt) {
      if constexpr (LOADER) wait_stages<LD, S - 1>(min(KT - 1, kt == 0 ? S - 1 : kt + S - 2) - kt);
      lds_barrier();
      lds_t* st = lds + rd * SB;
      // K rows past the expert's last: zero on both sides
      const int left = t.P.valid - kt * BK;
      if (left < BK) {
        for (int c = left * 32 + tid; c < BK * 32; c += WAVES * 64) *(lds_i32x4*)(st + c * 16) = i32x4{0, 0, 0, 0};
        for (int c = left * (QB * 4) + tid; c < BK * (QB * 4); c += WAVES * 64)
          *(lds_i32x4*)(st + 8 * 64 * BK + c * 16) = i32x4{0, 0, 0, 0};
        lds_barrier();
      }
      bwd_stage<true, true, 8, QB, 4, BK, NW>(st, WQ, wp, lane, acc, [&]() {
        if constexpr (LOADER) {
          if (kt > 0 && kt + S - 1 < KT) {
            lp.issue(kt + S - 1, lds + wr * SB, lw, lane);
            lq.issue(kt + S - 1, lds + wr * SB + 8 * 64 * BK, lw, lane);
          }
        }
      });
      rd = rd + 1 == S ? 0 : rd + 1;
      wr = wr + 1 == S ? 0 : wr + 1;
    }
    lds_barrier();  // the ring is free
    if (wp * 64 < t.cols) {
#pragma unroll
      for (int a = 0; a < 4; ++a) {
        const int m0 = (WQ + NW * a) * 32;
        if (m0 < t.rows) store_block<OP, 2>(P, t, lds + w * 4096, acc[a], m0, wp * 64, 0, lane);
      }
    }
    lds_barrier();  // ... for the next tile's loads
  }
}

// Workgroup b's place in the tile order: consecutive places on one XCD
// (workgroups are dealt to the 8 XCDs in turn).
__device__ __forceinline__ int place(int b, int G) { return G % 8 == 0 ? (b % 8) * (G / 8) + b / 8 : b; }

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

// The weight gradients of experts with few rows.
template <int OP>
__global__ __launch_bounds__(256, 2) void weight_backward_short_kernel(BwdParams P) {
  __shared__ __attribute__((aligned(1024))) uint8_t smem[3 * 12 * 64 * 32];
  if (P.meta[META_ARG_ERR] & ARG_ERR_PLAN) return;
  weight_tiles_body<OP, 4, true, 0>(P, (lds_t*)smem, place(blockIdx.x, gridDim.x), gridDim.x);
}

template <int OP>
__global__ __launch_bounds__(kBwdThreads, 1) void expert_backward_kernel(BwdParams P) {
  __shared__ __attribute__((aligned(1024))) uint8_t smem[kGemmLds];
  lds_t* lds = (lds_t*)smem;
  const int G = gridDim.x, lid = place(blockIdx.x, G);
  // rejected row indices or offsets: nothing is computed
  if (P.meta[META_ARG_ERR] & ARG_ERR_PLAN) return;
  if constexpr (OP <= BWD_DX) {
    const int nb = P.meta[META_P];
    const int width = OP == BWD_GU ? 2 * P.f : OP == BWD_DACT ? P.f : P.d;
    const int N = (width + 255) / 256, total = nb * N, cut = total / G * G;
    // Whole rounds of 256-column tiles, then the rest as halves. Where even the
    // halves leave workgroups idle, they are cut along the band's rows too, in
    // two or four: a smaller stage takes less time and makes a deeper ring. Whole
    // calls without cuts / with two / with up to four, us: one expert of 274 rows,
    // d = 3584, f = 1024 180 / 132 / 115; of 128 rows, 2048, 1408 114 / 113 / 103; of
    // 256 rows, 4096, 4096 331 / 240 / 228; 4 experts of 256 rows, 1024, 512
    // 114 / 91 / 83.
    int cuts = 1;
    while (cuts < 4 && 4 * cuts * (total - cut) <= G) cuts *= 2;
    for (int i = lid; i < cut + 2 * cuts * (total - cut); i += G) {
      const bool wide = i < cut;
      int p, n;
      raster(wide ? i : cut + (i - cut) / (2 * cuts), nb, N, P.group_m, p, n);
      if (!wide) n = 2 * n + ((i - cut) & 1);
      BwdTile t = band_tile<OP>(P, p, n, wide ? 256 : 128);
      if (!wide) take_rows(t, (((i - cut) >> 1) & (cuts - 1)) * (kBM / cuts), kBM / cuts);
      if (t.cols <= 0 || t.rows <= 0) continue;
      // weights of an expert with one band are read once per launch (see
      // streams_once)
      const bool once = (P.band_expert[p] & kBandSingle) != 0;
      if (wide) {
        if (once) run_band_tile<OP, 8, true>(P, t, lds);
        else run_band_tile<OP, 8, false>(P, t, lds);
      } else {
        if (once) run_band_tile<OP, 4, true>(P, t, lds);
        else run_band_tile<OP, 4, false>(P, t, lds);
      }
    }
  } else {
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (w >= 8 - kLoaders) {
      if (w & 1) weight_tiles_body<OP, 8, true, 1>(P, lds, lid, G);
      else weight_tiles_body<OP, 8, true, 0>(P, lds, lid, G);
    } else {
      if (w & 1) weight_tiles_body<OP, 8, false, 1>(P, lds, lid, G);
      else weight_tiles_body<OP, 8, false, 0>(P, lds, lid, G);
    }
  }
}

}  // namespace

namespace {
// Rows per expert, if the router spreads them evenly, above kShortRows.
bool long_experts(const moe_problem_t& p) { return (int64_t)p.T * p.k > (int64_t)kShortRows * p.E_global; }
}  // namespace

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

hipError_t launch_expert_backward(const moe_problem_t& p, const Layout& L, char* ws, const void* X,
                                  const int32_t* row_src, const int32_t* offsets, const int32_t* row_dst,
                                  const void* W1, const void* W2, const void* dO, void* dxs, void* dW1, void* dW2,
                                  hipStream_t s) {
  const int G = gemm_grid(p);
  if (G <= 0) return hipErrorInvalidDevice;
  hipError_t e = launch_plan_rows(p, L, ws, offsets, row_src, row_dst, ARG_ERR_DISPATCH_CAP | ARG_ERR_LINEAR1, 0, s);
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
  auto go = [&](auto kern) {
    if (e != hipSuccess) return;
    hipLaunchKernelGGL(kern, dim3(G), dim3(kBwdThreads), 0, s, P);
    e = hipGetLastError();
  };
  auto go2 = [&](auto kern) {
    if (e != hipSuccess) return;
    hipLaunchKernelGGL(kern, dim3(2 * G), dim3(256), 0, s, P);
    e = hipGetLastError();
  };
  go(expert_backward_kernel<BWD_GU>);
  go(expert_backward_kernel<BWD_DACT>);
  go(expert_backward_kernel<BWD_DX>);
  if (!long_experts(p)) {
    go2(weight_backward_short_kernel<BWD_DW2>);
    go2(weight_backward_short_kernel<BWD_DW1>);
  } else {
    hipLaunchKernelGGL(order_rows_kernel, dim3(4096), dim3(256), 0, s, P);
    if (e == hipSuccess) e = hipGetLastError();
    go(expert_backward_kernel<BWD_DW2>);
    go(expert_backward_kernel<BWD_DW1>);
  }
  return e;
}

}  // namespace moe
