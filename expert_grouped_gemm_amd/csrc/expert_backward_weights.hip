// The experts' weight gradients, dW2[e] = sum_r do a^T and dW1[e] = sum_r dh x^T
// (see expert_backward_device.h): products over an expert's rows, both operands
// strided along them.
//
// Two kernels. For few rows per expert a tile is a few stages long and
// otherwise setup, waits and stores, which two workgroups per CU overlap, and
// the rows are looked up. For many, one wavefront per SIMD holds 128 x 128
// results, so that a K step of 16 reads 8 fragments for 16 MFMAs instead of 6
// for 8 (128 x 64): the LDS, which took as long as the MFMAs, takes half. It
// reads ordered copies of the rows.
#include "expert_backward_device.h"

namespace moe {
namespace {

// Rows per expert up to which the kernel for few rows runs: the router's mean, T k /
// E_global, as the host does not see the call's offsets (a share that holds the
// favoured experts may take the kernel for few rows for long ones). The other
// kernel's gain grows with rows x d x f, its copies cost rows x d and a launch: where
// f is narrow, or all the experts' weights are few, it pays from more rows on. Whole
// calls of moe_expert_backward with the kernel for few rows / with the other one and
// its copies, us:
//   rows per expert              264          384          512
//   1 expert, d 512, f 512         64 / 72      69 / 77      79 / 85
//   8 of 2048, 1024               170 / 178    175 / 186    191 / 199
//   8 of 4096, 1024               305 / 318    323 / 331    354 / 353
//   1 of 4096, 4096               199 / 205    210 / 216    226 / 229
//   32 of 1024, 512               184 / 195    194 / 222    219 / 239
//   64 of 4096, 512              1128 / 1166  1278 / 1313  1383 / 1409
//   256 of 1024, 512             1252 / 1265  1494 / 1501  1627 / 1630
// and with 3 2^24 elements of W2 or more and a wider f:
//   24 of 2048, 1024              433 / 446    492 / 492    582 / 568
//   12 of 2048, 2048              457 / 455    511 / 498    616 / 589
//   3 of 4096, 4096               435 / 431    491 / 484    601 / 578
//   64 of 4096, 768              1600 / 1576  1859 / 1820  2038 / 1975
//   32 of 7168, 2048             3603 / 3426 (300 rows)    4449 / 4132
//   8 of 4096, 14336             3649 / 3411 (300 rows)    4398 / 3967
// (128 and 192 rows of the last two: 1689 / 1783 and 2222 / 2209, 1751 / 1785 and
// 2263 / 2229.)
constexpr int kShortRows = 256, kShortRowsOfLittle = 512;

// ------------------------------------------------------------- few rows

constexpr int kShortBK = 32, kShortRing = 3;         // K rows of a stage, stages
constexpr int kShortStage = 12 * 64 * kShortBK;      // 64 bytes of each 32-column block per K row

// An expert's rows as K (KS), kShortBK of them a stage, perhaps through idx. Lane kk
// holds the offset of K row kk of a stage for all lanes; rows past the last
// re-read it (the stage's LDS rows are zeroed). Offsets through idx fit 32 bits
// (the problem limits keep T * d and cap * d below 2^31 elements) and are
// fetched ahead: those of a tile's first kShortRing stages together, a later stage's
// when the stage before it is issued. Without idx they count from the stage's
// first row.
template <int BLOCKS>
struct RowLoads {
  static constexpr int CPR = BLOCKS * 4, RPI = 64 / CPR, NI = kShortBK * BLOCKS / 64;
  const uint8_t* base;
  uint32_t pitch, lane_off, ahead[kShortRing];
  const int32_t* idx;
  int div, valid;

  __device__ __forceinline__ uint32_t look_up(int kt, int lane) const {
    return (uint32_t)(idx[min(kt * kShortBK + (lane & (kShortBK - 1)), valid - 1)] / div) * pitch;
  }
  __device__ __forceinline__ void init(const Side& s, int lw, int lane) {
    base = s.base;
    pitch = s.pitch;
    idx = s.idx;
    div = s.div;
    valid = s.valid;
    const int kk = lw * RPI + lane / CPR;
    lane_off = (((lane % CPR) ^ ks_swizzle(kk)) & (s.chunks - 1)) << 4;
    if (idx && valid > 0) {
#pragma unroll
      for (int i = 0; i < kShortRing; ++i) ahead[i] = look_up(i, lane);
    }
  }
  __device__ __forceinline__ void issue_rows(int kt, uint32_t rows, lds_t* st, int lw, int lane) {
    const int kk = lw * RPI + lane / CPR, left = valid - kt * kShortBK;
    const uint8_t* b0 = idx ? base : base + (size_t)kt * kShortBK * pitch;
    if (!idx && left >= kShortBK) {
      const uint32_t off = kk * pitch + lane_off;
#pragma unroll
      for (int j = 0; j < NI; ++j)
        dma16<false>(b0 + (size_t)(4 * j * RPI) * pitch, off, st + (4 * j + lw) * 1024);
      return;
    }
    if (!idx) rows = min(lane & (kShortBK - 1), left - 1) * pitch;
#pragma unroll
    for (int j = 0; j < NI; ++j)
      dma16<false>(b0, (uint32_t)__shfl((int)rows, 4 * j * RPI + kk, 64) + lane_off, st + (4 * j + lw) * 1024);
  }
  // stage kt < kShortRing, of the tile's first ones
  __device__ __forceinline__ void issue_first(int kt, lds_t* st, int lw, int lane) {
    issue_rows(kt, ahead[kt], st, lw, lane);
    if (kt == kShortRing - 1 && idx) ahead[0] = look_up(kShortRing, lane);
  }
  // a later stage
  __device__ __forceinline__ void issue(int kt, lds_t* st, int lw, int lane) {
    const uint32_t rows = ahead[0];
    if (idx && (kt + 1) * kShortBK < valid) ahead[0] = look_up(kt + 1, lane);
    issue_rows(kt, rows, st, lw, lane);
  }
};

// Tile (m, n) of an expert's weight gradient: 128 x 256, the rows of X and dO
// looked up.
template <int OP>
__device__ __forceinline__ BwdTile short_tile(const BwdParams& P, int e, int m, int n) {
  BwdTile t;
  t.e = e;
  const int r0 = P.offsets[e], cnt = P.offsets[e + 1] - r0;
  t.row0 = m * 128;
  t.rows = 128;
  t.col0 = n * 256;
  t.cols = min(256, (OP == BWD_DW2 ? P.f : P.d) - t.col0);
  const uint32_t db = (uint32_t)P.d * 2, fb = (uint32_t)P.f * 2;
  if constexpr (OP == BWD_DW2) {
    t.P = Side{reinterpret_cast<const uint8_t*>(P.act) + (size_t)r0 * fb + (size_t)t.col0 * 2, fb, cnt, t.cols / 8,
               nullptr, 1};
    t.Q = Side{P.dO + (size_t)t.row0 * 2, db, cnt, 16, P.row_dst + r0, 1};
  } else {
    t.P = P.row_src ? Side{P.X + (size_t)t.col0 * 2, db, cnt, t.cols / 8, P.row_src + r0, P.k}
                    : Side{P.X + (size_t)r0 * db + (size_t)t.col0 * 2, db, cnt, t.cols / 8, nullptr, 1};
    t.Q = Side{reinterpret_cast<const uint8_t*>(P.dH) + (size_t)r0 * (2 * fb) + (size_t)t.row0 * 2, 2 * fb, cnt, 16,
               nullptr, 1};
  }
  return t;
}

// 128 x 256 tiles, three stages of 32 K rows, two workgroups per CU (72 KiB of
// LDS each), every wavefront loads. A tile starts with the whole ring in
// flight; from step 1 on, each step refills the slot of the step before it.
// (One stream of stages over a workgroup's tiles, the next one's first loads
// issued before the last one's stores, was no faster: share dW1 508 against 502
// us; nor were 128 x 128 tiles with three workgroups per CU, 485 against 462, nor
// parts of every expert kept on one XCD, 464. MFMAs, LDS and stores, 123, 140 and
// 345 us of them, are what does not overlap. All timed by themselves; in whole calls
// the share's dW1 takes 484 to 586.)
template <int OP>
__global__ __launch_bounds__(256, 2) void weight_backward_short_kernel(BwdParams P) {
  __shared__ __attribute__((aligned(1024))) uint8_t smem[kShortRing * kShortStage];
  if (P.meta[META_ARG_ERR] & ARG_ERR_PLAN) return;
  lds_t* lds = (lds_t*)smem;
  const int G = gridDim.x;
  int tid = threadIdx.x;
  asm volatile("" : "+v"(tid));
  const int lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int M = (OP == BWD_DW2 ? P.d : 2 * P.f) / 128, N = ((OP == BWD_DW2 ? P.f : P.d) + 255) / 256;
  const int64_t total = (int64_t)P.El * M * N;
  constexpr int LD = RowLoads<8>::NI + RowLoads<4>::NI;
  for (int64_t i = place(blockIdx.x, G); i < total; i += G) {
    const int e = (int)(i / (M * N));
    int m, n;
    raster((int)(i - (int64_t)e * M * N), M, N, P.group_m, m, n);
    const BwdTile t = short_tile<OP>(P, e, m, n);
    const int KT = (t.P.valid + kShortBK - 1) / kShortBK;
    RowLoads<8> lp;
    RowLoads<4> lq;
    lp.init(t.P, w, lane);
    lq.init(t.Q, w, lane);
#pragma unroll
    for (int s = 0; s < kShortRing; ++s)
      if (s < KT) {
        lp.issue_first(s, lds + s * kShortStage, w, lane);
        lq.issue_first(s, lds + s * kShortStage + 8 * 64 * kShortBK, w, lane);
      }
    f32x16 acc[4][2];
    clear_acc(acc);
    int rd = 0, wr = kShortRing - 1;
    for (int kt = 0; kt < KT; ++kt) {
      wait_stages<LD, kShortRing - 1>(min(KT - 1, kt == 0 ? kShortRing - 1 : kt + kShortRing - 2) - kt);
      lds_barrier();
      lds_t* st = lds + rd * kShortStage;
      // K rows past the expert's last: zero on both sides
      const int left = t.P.valid - kt * kShortBK;
      if (left < kShortBK) {
        for (int c = left * 32 + tid; c < kShortBK * 32; c += 256) *(lds_i32x4*)(st + c * 16) = i32x4{0, 0, 0, 0};
        for (int c = left * 16 + tid; c < kShortBK * 16; c += 256)
          *(lds_i32x4*)(st + 8 * 64 * kShortBK + c * 16) = i32x4{0, 0, 0, 0};
        lds_barrier();
      }
      bwd_stage<true, true, 8, 4, 4, kShortBK, 1>(st, 0, w, lane, acc, [&]() {
        if (kt > 0 && kt + kShortRing - 1 < KT) {
          lp.issue(kt + kShortRing - 1, lds + wr * kShortStage, w, lane);
          lq.issue(kt + kShortRing - 1, lds + wr * kShortStage + 8 * 64 * kShortBK, w, lane);
        }
      });
      rd = rd + 1 == kShortRing ? 0 : rd + 1;
      wr = wr + 1 == kShortRing ? 0 : wr + 1;
    }
    lds_barrier();  // the ring is free
    if (w * 64 < t.cols) {
#pragma unroll
      for (int a = 0; a < 4; ++a) store_block<OP, 2>(P, t, lds + w * 4096, acc[a], a * 32, w * 64, 0, lane);
    }
    lds_barrier();  // ... for the next tile's loads
  }
}

// ------------------------------------------------------------- many rows

constexpr int kLongRing = 5, kLongStage = 32 * 1024;  // stages of 32 K rows of 256 + 256 columns
constexpr int kLongLoads = 8;                         // a wavefront's loads of a stage

typedef const __attribute__((address_space(4))) int32_t* scalar_ptr;  // read through the scalar cache

// A tile: 256 x 256 of expert e's gradient (128 where the matrix ends).
struct LongTile {
  const uint8_t *p, *q;      // the expert's first row of either operand, at the tile's columns
  uint32_t pitch_p, pitch_q;
  int e, k_rows;             // the expert's rows
  int row0, col0, rows, cols;
};

template <int OP>
__device__ __forceinline__ LongTile long_tile(const BwdParams& P, int64_t i, int M, int N) {
  LongTile t;
  t.e = (int)(i / (M * N));
  int m, n;
  raster((int)(i - (int64_t)t.e * M * N), M, N, P.group_m, m, n);
  const scalar_ptr off = (scalar_ptr)(uintptr_t)P.offsets;
  const int r0 = off[t.e];
  t.k_rows = off[t.e + 1] - r0;
  t.row0 = m * 256;
  t.col0 = n * 256;
  t.rows = min(256, (OP == BWD_DW2 ? P.d : 2 * P.f) - t.row0);
  t.cols = min(256, (OP == BWD_DW2 ? P.f : P.d) - t.col0);
  const uint32_t db = (uint32_t)P.d * 2, fb = (uint32_t)P.f * 2;
  if constexpr (OP == BWD_DW2) {
    t.p = reinterpret_cast<const uint8_t*>(P.act) + (size_t)r0 * fb + (size_t)t.col0 * 2;
    t.pitch_p = fb;
    t.q = reinterpret_cast<const uint8_t*>(P.dOp) + (size_t)r0 * db + (size_t)t.row0 * 2;
    t.pitch_q = db;
  } else {
    t.p = (P.row_src ? reinterpret_cast<const uint8_t*>(P.Xp) : P.X) + (size_t)r0 * db + (size_t)t.col0 * 2;
    t.pitch_p = db;
    t.q = reinterpret_cast<const uint8_t*>(P.dH) + (size_t)r0 * (2 * fb) + (size_t)t.row0 * 2;
    t.pitch_q = 2 * fb;
  }
  return t;
}

// A wavefront's 128 x 128 results, without the LDS (whose ring holds the next
// tile's stages by now). Lane l of an accumulator block has row l % 32 and, in
// elements 4 q .. 4 q + 3, the columns 8 q + 4 (l / 32) .. + 3. Rounded and packed,
//   permlane32_swap makes 16-byte chunks: lane l has chunks l / 32 and 2 + l / 32
//     of its row's four;
//   permlane16_swap makes a lane's two chunks one of row l % 16 and one of row
//     16 + l % 16: four lanes hold a row's 64 bytes;
//   a rotation by 8 within 16 lanes does the same with the next block's: eight
//     lanes hold 128 bytes of a row, and every store writes whole lines of 8 rows.
// (Partial lines past the caches are slow: 64 bytes at a time 3.1 TB/s, 128 5.2.)
template <int OP>
__device__ __forceinline__ void long_store(const BwdParams& P, const LongTile& t, int wq, int wp, int lane,
                                           const f32x16 (&acc)[4][4]) {
  const size_t ld = OP == BWD_DW2 ? P.f : P.d;
  uint16_t* out = (OP == BWD_DW2 ? P.dW2 + (size_t)t.e * P.d * P.f : P.dW1 + (size_t)t.e * 2 * P.f * P.d) +
                  (size_t)(t.row0 + wq * 128 + (lane & 7)) * ld + t.col0 + wp * 128 + ((lane >> 3) & 1) * 32 +
                  ((lane >> 5) + 2 * ((lane >> 4) & 1)) * 8;
#pragma unroll
  for (int a = 0; a < 4; ++a)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      i32x4 v[2][2];
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        uint32_t d[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) d[i] = pack_bf16(acc[a][2 * h + b][2 * i], acc[a][2 * h + b][2 * i + 1]);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const auto x = __builtin_amdgcn_permlane32_swap(d[i], d[2 + i], false, false);
          const auto y = __builtin_amdgcn_permlane32_swap(d[4 + i], d[6 + i], false, false);
          const auto lo = __builtin_amdgcn_permlane16_swap(x[0], y[0], false, false);
          const auto up = __builtin_amdgcn_permlane16_swap(x[1], y[1], false, false);
          v[b][0][i] = (int)lo[0];
          v[b][1][i] = (int)lo[1];
          v[b][0][2 + i] = (int)up[0];
          v[b][1][2 + i] = (int)up[1];
        }
      }
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        i32x4 lo, up;  // rows 0 .. 7 and 8 .. 15 of the 16
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          lo[i] = __builtin_amdgcn_update_dpp(v[0][r][i], v[1][r][i], 0x128, 0xF, 0xC, false);
          up[i] = __builtin_amdgcn_update_dpp(v[1][r][i], v[0][r][i], 0x128, 0xF, 0x3, false);
        }
        uint16_t* at = out + (size_t)(a * 32 + r * 16) * ld + h * 64;
        __builtin_nontemporal_store(lo, reinterpret_cast<i32x4*>(at));
        __builtin_nontemporal_store(up, reinterpret_cast<i32x4*>(at + 8 * ld));
      }
    }
}

// A workgroup's tiles, one after the other, their stages one stream: loads run
// kLongRing stages ahead, across tiles. One barrier per stage, between its two K
// steps: it shows the next stage complete and this one read, so that its slot
// takes the stage kLongRing further while the second step's MFMAs run. The
// fragments of a step are read behind the MFMAs of the step before it, in an
// order that the compiler is held to; with one wavefront per SIMD nothing else
// fills a gap. Nothing in the loop depends on the stream's end: behind the last
// tile its last stage is loaded again, into slots that nothing reads.
// 16384 rows of 8 experts, d = 4096, f = 14336, in whole calls, us (TFLOP/s): DW2 1870
// (1029), DW1 3530 (1090), the MFMAs busy 55% of the time at the 1.96 GHz the chip
// holds. (256 x 256 tiles on eight wavefronts, 128 x 64 each, two stages of 64: 1875
// and 3730; whole calls of 512 rows per expert 4398 instead of 3967. Counts of what
// each wait may leave in flight, and the reads in another order: 2220 and 4370.)
template <int OP>
__device__ __forceinline__ void weight_tiles_long(const BwdParams& P, lds_t* lds) {
  const int G = gridDim.x;
  int tid = threadIdx.x;
  asm volatile("" : "+v"(tid));
  const int lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6), wq = w & 1, wp = w >> 1;
  const int M = ((OP == BWD_DW2 ? P.d : 2 * P.f) + 255) / 256, N = ((OP == BWD_DW2 ? P.f : P.d) + 255) / 256;
  const int64_t total = (int64_t)P.El * M * N;

  // the stage to load next: its first row of either operand, lk rows into the
  // tile's; a load takes 2 rows of 512 bytes, a wavefront's are 8 rows apart
  int64_t li = place(blockIdx.x, G);
  int lk = 0, l_rows = 0, wr = 0;
  const uint8_t *bp = nullptr, *bq = nullptr;
  uint32_t pitch_p = 0, pitch_q = 0, off_p = 0, off_q = 0;
  const int kk = w * 2 + (lane >> 5);
  auto next_load_tile = [&]() {
    for (; li < total; li += G) {
      const LongTile t = long_tile<OP>(P, li, M, N);
      if (t.k_rows <= 0) continue;  // an expert without rows has no stages
      bp = t.p;
      bq = t.q;
      pitch_p = t.pitch_p;
      pitch_q = t.pitch_q;
      l_rows = t.k_rows;
      // where only 128 columns exist, the others re-read those
      off_p = (((lane & 31) ^ ks_swizzle(kk)) & ((t.cols >> 3) - 1)) << 4;
      off_q = (((lane & 31) ^ ks_swizzle(kk)) & ((t.rows >> 3) - 1)) << 4;
      lk = 0;
      break;
    }
  };
  auto load_one = [&](int j) {
    lds_t* st = lds + wr * kLongStage + w * 1024;
    const uint32_t row = min(8 * (j & 3) + kk, l_rows - lk - 1);  // rows past the last re-read it
    if (j < 4) dma16<false>(bp, row * pitch_p + off_p, st + j * 4096);
    else dma16<false>(bq, row * pitch_q + off_q, st + 16384 + (j - 4) * 4096);
  };
  auto issued = [&]() {
    wr = wr + 1 == kLongRing ? 0 : wr + 1;
    if (lk + 32 < l_rows) {
      lk += 32;
      bp += (size_t)32 * pitch_p;
      bq += (size_t)32 * pitch_q;
    } else if (li < total) {
      li += G;
      next_load_tile();
    }
  };
  // The oldest stage in flight: complete, its K rows from `left` on zeroed by the
  // lanes that loaded them, and shown to every wavefront. Of the ring's stages
  // one is being read, this one and kLongRing - 2 after it are in flight (at the
  // start one more; stores in between, too, only make the wait longer).
  auto arrive = [&](int slot, int left) {
    wait_vmcnt<kLongLoads * (kLongRing - 2)>();
    if (left < 32) {
      lds_t* st = lds + slot * kLongStage + w * 1024 + lane * 16;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (8 * j + kk >= left) {
          *(lds_i32x4*)(st + j * 4096) = i32x4{0, 0, 0, 0};
          *(lds_i32x4*)(st + j * 4096 + 16384) = i32x4{0, 0, 0, 0};
        }
    }
    lds_barrier();
  };

  bf16x8 fp[2][4], fq[2][4];
  auto read_p = [&](const lds_t* st, int ks, int b) { fp[ks][b] = fragment<true, 8>(st, 4 * wp + b, ks, lane); };
  auto read_q = [&](const lds_t* st, int ks, int a) { fq[ks][a] = fragment<true, 8>(st + 16384, 4 * wq + a, ks, lane); };
  next_load_tile();
  int rd = 0;
  if (l_rows > 0) {
    const int first = l_rows;
    for (int s = 0; s < kLongRing; ++s) {
#pragma unroll
      for (int j = 0; j < kLongLoads; ++j) load_one(j);
      issued();
    }
    arrive(0, first);
#pragma unroll
    for (int b = 0; b < 4; ++b) read_p(lds, 0, b);
#pragma unroll
    for (int a = 0; a < 4; ++a) read_q(lds, 0, a);
  }
  // The next tile that has rows, and their number. Looked for once from each tile
  // that has any: from every tile, runs of experts without rows took a time that
  // grows with their square (256 experts, 2048 x 2048, rows on one of them: a call of
  // 2040 us instead of 1380, in which it stores 6.4 GB of zeros).
  int64_t next = 0;
  int next_rows = 0;
  for (int64_t i = place(blockIdx.x, G); i < total; i += G) {
    const LongTile t = long_tile<OP>(P, i, M, N);
    if (next <= i) {
      next_rows = 0;
      for (next = i + G; next < total; next += G) {
        const scalar_ptr off = (scalar_ptr)(uintptr_t)P.offsets;
        const int e = (int)(next / (M * N));
        next_rows = off[e + 1] - off[e];
        if (next_rows > 0) break;
      }
    }
    f32x16 acc[4][4];
    clear_acc(acc);
    for (int k = 0; k < t.k_rows; k += 32) {
      const lds_t* st = lds + rd * kLongStage;
#pragma unroll
      for (int b = 0; b < 4; ++b) read_p(st, 1, b);
#pragma unroll
      for (int a = 0; a < 4; ++a) read_q(st, 1, a);
#pragma unroll
      for (int a = 0; a < 4; ++a)
#pragma unroll
        for (int b = 0; b < 4; ++b)
          acc[a][b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fp[0][b], fq[0][a], acc[a][b], 0, 0, 0);
      // two LDS reads behind each of the first eight MFMAs: all have come at the barrier
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
        __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
      }
      __builtin_amdgcn_sched_group_barrier(0x8, 8, 0);
      rd = rd + 1 == kLongRing ? 0 : rd + 1;
      const int left = t.k_rows - k - 32;
      arrive(rd, left > 0 ? left : next_rows);
      st = lds + rd * kLongStage;
#pragma unroll
      for (int a = 0; a < 4; ++a) {
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          acc[a][b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fp[1][b], fq[1][a], acc[a][b], 0, 0, 0);
          const int x = 2 * a + (b >> 1);  // a fragment, a load, in turn
          if (b & 1) load_one(x);
          else if (x < 4) read_p(st, 0, x);
          else read_q(st, 0, x - 4);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      issued();
    }
    if (wq * 128 < t.rows && wp * 128 < t.cols) long_store<OP>(P, t, wq, wp, lane, acc);
  }
  wait_vmcnt<0>();  // the loads behind the last tile
}

constexpr int kLongThreads = 256;
template <>
__global__ __launch_bounds__(kLongThreads, 1) void expert_backward_kernel<BWD_DW2>(BwdParams P) {
  __shared__ __attribute__((aligned(1024))) uint8_t smem[kLongRing * kLongStage];
  if (P.meta[META_ARG_ERR] & ARG_ERR_PLAN) return;
  weight_tiles_long<BWD_DW2>(P, (lds_t*)smem);
}
template <>
__global__ __launch_bounds__(kLongThreads, 1) void expert_backward_kernel<BWD_DW1>(BwdParams P) {
  __shared__ __attribute__((aligned(1024))) uint8_t smem[kLongRing * kLongStage];
  if (P.meta[META_ARG_ERR] & ARG_ERR_PLAN) return;
  weight_tiles_long<BWD_DW1>(P, (lds_t*)smem);
}

}  // namespace

bool long_experts(const moe_problem_t& p) {
  const bool little = p.f <= 512 || (int64_t)(p.e_end - p.e_begin) * p.d * p.f < 3 << 24;
  return (int64_t)p.T * p.k > (int64_t)(little ? kShortRowsOfLittle : kShortRows) * p.E_global;
}

hipError_t launch_weight_gradients(const BwdParams& P, bool long_rows, int G, hipStream_t s) {
  hipError_t e = hipSuccess;
  auto go = [&](auto kern, int grid, int threads) {
    if (e != hipSuccess) return;
    hipLaunchKernelGGL(kern, dim3(grid), dim3(threads), 0, s, P);
    e = hipGetLastError();
  };
  if (long_rows) {
    go(expert_backward_kernel<BWD_DW2>, G, kLongThreads);
    go(expert_backward_kernel<BWD_DW1>, G, kLongThreads);
  } else {
    go(weight_backward_short_kernel<BWD_DW2>, 2 * G, 256);
    go(weight_backward_short_kernel<BWD_DW1>, 2 * G, 256);
  }
  return e;
}

}  // namespace moe
