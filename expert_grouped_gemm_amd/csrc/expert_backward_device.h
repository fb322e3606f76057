// Device side of the gradient of the experts' SwiGLU products
// (moe_expert_backward, moe_expert_backward_checkpoint).
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
// (a as in the forward; the outputs are then off by 2.34e-3 of their norm, where
// rounding the exact ones costs 1.66e-3, and two bf16 terms instead of one would
// double three products); every sum is fp32, dx and the weight gradients are
// rounded once. Every output element is one workgroup's sum in one K order:
// no atomics, the same result on every call.
//
// An operand contiguous along K (KC) lies in the LDS as rows of 64 K values
// and is read 16 bytes per lane; one strided along K (KS) lies as 64 rows of K
// with the tile's 256 columns each and is read by the transposing LDS read
// (ds_read_b64_tr_b16: 16 lanes take 4 K rows x 16 columns, lane i ends with
// the 4 K values of column i), so no operand is ever transposed in memory.
//
// Measured (medians of whole calls' launches over three sets of operands in turn, us;
// rates in TFLOP/s or TB/s of the bytes the product cannot do without). The share
// (4096 rows of 32 experts, d = 7168, f = 2048), bound by HBM but for the weight
// gradients, whose tiles of two to five stages are half setup and stores: GU 364 (5.2
// TB/s), DACT 195 (4.8), DACT8 200 (from a checkpoint, 5.3 with its codes and
// results), DX 386 (4.9), DW2 320-340 (2.8), DW1 586 (3.2; 484 where the tokens' codes
// have been expanded into expert order). 16384 rows of 8 experts, d = 4096, f = 14336:
// the MFMA units at the clock that their power leaves (DX: busy 67% at 1.63 GHz, DW1:
// 56% at 1.93), and the loads, LDS reads, epilogues and last rounds that do not
// overlap with them: GU 3606 (1067), DACT 2338 (823, with the epilogue's 3.3 GB),
// DACT8 2060 (934), DX 3410-3460 (1120), DW2 1870 (1029), DW1 3530 (1090).
// No kernel here spills a register.
// Not kept: a ring of 32-wide K stages with the loads spread over the MFMAs and
// fragments read across the barrier (20% slower) and every wavefront loading
// (6%), both on eight wavefronts and while the loads still went through the
// builtin (see dma16); DACT's fp32 gate and up values all fetched ahead of its
// stores (registers spilled); every second XCD half a tile out of step with the
// others, so that their epilogues' traffic spreads (DACT8 60 us of 2053).
#pragma once

#include "gemm_device.h"

namespace moe {

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
  uint16_t* Xp;              // the token rows (MXINT8 tokens, long experts) and the output gradients
  uint16_t* dOp;             // (long experts) in expert order, [cap, d] each
  const int32_t* row_src;    // or null
  const int32_t* row_dst;
  const int32_t* offsets;
  const int32_t* band_expert;
  const int32_t* band_row0;
  const int32_t* band_rows;
  const int32_t* meta;
  const uint8_t* Xs;         // MXINT8 tokens: E8M0 scales, d/32 per row; null: X is bf16
  const int8_t* gu8;         // the checkpoint: gate and up in MXINT8, [cap, 2f] and [cap, 2f/32]
  const uint8_t* gus;
  int k, d, f, El, group_m;
};

// Whether the weight gradients take the kernel for long experts (see
// expert_backward_weights.hip), which reads ordered copies of the rows.
bool long_experts(const moe_problem_t& p);

// The parameters of a call whose intermediates lie at B in its workspace.
BwdParams backward_params(const moe_problem_t& p, const Layout& L, const BackwardLayout& B, char* ws, const void* X,
                          const int32_t* row_src, const int32_t* offsets, const int32_t* row_dst, const void* W1,
                          const void* W2, const void* dO, void* dxs, void* dW1, void* dW2);

// Launches on G workgroups that calls share, each in one translation unit (the
// kernels take minutes to compile, and their units compile in parallel).
hipError_t launch_backward_dx(const BwdParams& P, int G, hipStream_t s);
hipError_t launch_order_rows(const BwdParams& P, hipStream_t s);
hipError_t launch_weight_gradients(const BwdParams& P, bool long_rows, int G, hipStream_t s);

namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
typedef __attribute__((address_space(3))) u32x2 lds_u32x2;

// BWD_DACT8: DACT whose gate and up come from the checkpoint's codes.
enum BwdOp { BWD_GU = 0, BWD_DACT = 1, BWD_DX = 2, BWD_DW2 = 3, BWD_DW1 = 4, BWD_DACT8 = 5 };
__host__ __device__ constexpr bool p_strided(int OP) { return OP != BWD_GU; }
__host__ __device__ constexpr bool is_dact(int OP) { return OP == BWD_DACT || OP == BWD_DACT8; }

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

// dh and a of one element from its gate, up and da.
__device__ __forceinline__ void swiglu_grad(float da, float g, float u, float& a, float& dg, float& du) {
  const float s = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(g * -1.4426950408889634f));
  const float gs = g * s;
  a = gs * u;
  du = da * gs;
  dg = da * u * (s + gs * (1.0f - s));
}

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
        for (int i = 0; i < 4; ++i) swiglu_grad(v[i], g[i], u[i], a[i], dg[i], du[i]);
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

// DACT8: the checkpoint's codes and scales for a 32-row block of a wavefront, 8
// columns per lane, 4 NB lanes per row. All of a block's are fetched before the
// block before it is stored: a load that follows stores is waited for together
// with them. (Fetched as each 4 columns are stored: 16384 rows, d = 4096, f =
// 14336 2257 us instead of 2101; and 2053 with the stores past the caches, the
// share 190, 184 and 182, each timed by itself. The K loop alone takes 1588 and 165.)
template <int NB>
struct BlockCodes {
  uint2 g[2 * NB], u[2 * NB];
  uint32_t sg[2 * NB], su[2 * NB];
  // rows past the last re-read it; 32-bit offsets (cap * 2f codes are below 2^32)
  __device__ __forceinline__ void fetch(const BwdParams& P, const BwdTile& t, int m0, int c0, int lane) {
    constexpr int L = 4 * NB;
#pragma unroll
    for (int j = 0; j < 2 * NB; ++j) {
      const int r = min(m0 + j * (64 / L) + lane / L, t.rows - 1);
      const uint32_t at =
          (uint32_t)(t.row0 + r) * (2 * (uint32_t)P.f) + (uint32_t)(t.col0 + c0 + (lane & (L - 1)) * 8);
      g[j] = *reinterpret_cast<const uint2*>(P.gu8 + at);
      u[j] = *reinterpret_cast<const uint2*>(P.gu8 + (at + (uint32_t)P.f));
      sg[j] = P.gus[at >> 5];
      su[j] = P.gus[(at + (uint32_t)P.f) >> 5];
    }
  }
};

// store_block of DACT8: 8 columns per lane, whole 128-byte lines (64 with NB = 1).
template <int NB>
__device__ __forceinline__ void store_block8(const BwdParams& P, const BwdTile& t, lds_t* wl, const f32x16 (&acc)[NB],
                                             int m0, int c0, const BlockCodes<NB>& codes, int lane) {
  constexpr int C = 8 * NB, L = 4 * NB;
  const int lr = lane & 31, hi = lane >> 5;
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int q = 0; q < 4; ++q)
      *(lds_f32x4*)(wl + lr * (C * 16) + (((b * 8 + 2 * q + hi) ^ (lr & (C - 1))) << 4)) =
          f32x4{acc[b][4 * q], acc[b][4 * q + 1], acc[b][4 * q + 2], acc[b][4 * q + 3]};
  wave_lds_sync();
  const int c = lane & (L - 1);
#pragma unroll
  for (int j = 0; j < 2 * NB; ++j) {
    const int r = j * (64 / L) + lane / L;
    const lds_t* at = wl + r * (C * 16);
    const f32x4 lo = *(const lds_f32x4*)(at + (((2 * c) ^ (r & (C - 1))) << 4));
    const f32x4 up = *(const lds_f32x4*)(at + (((2 * c + 1) ^ (r & (C - 1))) << 4));
    float g[8], u[8], a[8], dg[8], du[8];
    mxint8_values8(codes.g[j], mxint8_step(codes.sg[j]), g);
    mxint8_values8(codes.u[j], mxint8_step(codes.su[j]), u);
#pragma unroll
    for (int i = 0; i < 8; ++i) swiglu_grad(i < 4 ? lo[i] : up[i - 4], g[i], u[i], a[i], dg[i], du[i]);
    if (m0 + r < t.rows) {
      const size_t row = (size_t)t.row0 + m0 + r;
      const int col = t.col0 + c0 + c * 8;
      auto put = [](uint16_t* to, const float(&v)[8]) {
        const i32x4 w = {(int)pack_bf16(v[0], v[1]), (int)pack_bf16(v[2], v[3]), (int)pack_bf16(v[4], v[5]),
                         (int)pack_bf16(v[6], v[7])};
        __builtin_nontemporal_store(w, reinterpret_cast<i32x4*>(to));
      };
      uint16_t* dh = P.dH + row * (2 * (size_t)P.f) + col;
      put(P.act + row * P.f + col, a);
      put(dh, dg);
      put(dh + P.f, du);
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
  if constexpr (OP == BWD_DACT8) {
    if (wp * (NB * 32) < t.cols) {
      BlockCodes<NB> codes[2];
      codes[0].fetch(P, t, WQ * 32, wp * (NB * 32), lane);
#pragma unroll
      for (int a = 0; a < NM; ++a) {
        const int m0 = (WQ + 2 * a) * 32;
        if (a + 1 < NM) codes[(a + 1) & 1].fetch(P, t, m0 + 64, wp * (NB * 32), lane);
        __builtin_amdgcn_sched_barrier(0);
        if (m0 < t.rows) store_block8<NB>(P, t, lds + w * 8192, acc[a], m0, wp * (NB * 32), codes[a & 1], lane);
      }
    }
  } else if (wp * (NB * 32) < t.cols) {
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
  } else if constexpr (is_dact(OP)) {
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

// Workgroup b's place in the tile order: consecutive places on one XCD
// (workgroups are dealt to the 8 XCDs in turn).
__device__ __forceinline__ int place(int b, int G) { return G % 8 == 0 ? (b % 8) * (G / 8) + b / 8 : b; }

// GU, DACT and DX. (DW2 and DW1, of other tiles, are specialised in
// expert_backward_weights.hip.)
template <int OP>
__global__ __launch_bounds__(kBwdThreads, 1) void expert_backward_kernel(BwdParams P) {
  __shared__ __attribute__((aligned(1024))) uint8_t smem[kGemmLds];
  lds_t* lds = (lds_t*)smem;
  const int G = gridDim.x, lid = place(blockIdx.x, G);
  // rejected row indices or offsets: nothing is computed
  if (P.meta[META_ARG_ERR] & ARG_ERR_PLAN) return;
  const int nb = P.meta[META_P];
  const int width = OP == BWD_GU ? 2 * P.f : is_dact(OP) ? P.f : P.d;
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
}

}  // namespace
}  // namespace moe
