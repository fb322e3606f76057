// Gradients of the two permutations of the share: the weighted combine with
// the router's softmax behind it, and the dispatch's gather. (Forward: Cui et
// al., "Fine-grained Computation-Communication Overlap via Tile-level
// Signaling and Scheduling for MoE", Section 2.1 steps (1), (2) and (5).)
//
// With O[p] the expert output in token-order slot p, w[t, j] the gate weight
// of slot j of token t and q(t) the token's output row, the forward is
//   Y[q(t)] = sum over the local slots j of w[t, j] O[p(t, j)],
// so for a gradient dY
//   dO[p(t, j)] = w[t, j] dY[q(t)]
//   dw[t, j]    = <dY[q(t)], O[p(t, j)]>        (0 for an expert held elsewhere)
// and through w = softmax of the k selected logits, the unselected ones having
// no part in the result,
//   dl[t, e] = sum over j with idx[t, j] = e of w_j (dw_j - sum_i w_i dw_i).
// dl is linear in dw: the shares' partial results add up to the layer's.
// The gather X_perm[r] = X[t(r)] has the adjoint dX[t] = sum over the token's
// slots of the rows' gradients.
//
// Every sum has one owner and one order: no atomics.
#include "moe_internal.h"

namespace moe {
namespace {

__device__ __forceinline__ void unpack8(const uint4& u, float (&v)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
  uint4 o;
  o.x = pack_bf16(v[0], v[1]);
  o.y = pack_bf16(v[2], v[3]);
  o.z = pack_bf16(v[4], v[5]);
  o.w = pack_bf16(v[6], v[7]);
  return o;
}

__device__ __forceinline__ float wave_sum(float x) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) x += __shfl_xor(x, off, 64);
  return x;
}

constexpr int kMaxK = 16;

// One workgroup per token, slot by slot (dY's row, read again for each, is in the
// caches by then); the dots are summed over the workgroup at the end. Bound by
// HBM: on the share (4096 tokens, 4100 slots, d = 7168, 256 logits) 53 us for 239
// MB, 4.5 TB/s where a large copy reaches 5.2.
template <bool BF16_IN>
__global__ __launch_bounds__(256) void combine_backward_kernel(
    const uint16_t* __restrict__ dY, const void* __restrict__ buf, const int32_t* __restrict__ tok_off,
    const int32_t* __restrict__ topk_idx, const float* __restrict__ topk_w, int T, int d, int k, int E, int e_begin,
    int El, int S, int cap, uint16_t* __restrict__ dO, float* __restrict__ d_w, float* __restrict__ d_logits) {
  __shared__ float part[kMaxK][4];
  __shared__ float s_dl[kMaxK];
  __shared__ int s_idx[kMaxK];
  const int t = blockIdx.x, lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int q = y_row_of_token(t, T, S);
  // lane j holds slot j of the token (every wavefront alike)
  const int idx = lane < k ? topk_idx[(size_t)t * k + lane] : -1;
  const float w = lane < k ? topk_w[(size_t)t * k + lane] : 0.0f;
  const bool local = lane < k && (unsigned)(idx - e_begin) < (unsigned)El;
  const uint64_t mask = __ballot(local);
  const int p0 = tok_off[q], p1 = tok_off[q + 1];
  // the slot range comes from device memory: one that does not lie inside the
  // buffer, or does not match the token's local experts, gives NaN gradients
  // and touches no slot
  const bool ok = 0 <= p0 && p1 <= cap && p1 - p0 == __popcll(mask);
  const int vec = d >> 3;
  const uint4* dy_row = reinterpret_cast<const uint4*>(dY + (size_t)q * d);
  if (ok) {
    uint64_t left = mask;
    for (int p = p0; left; ++p) {
      const int j = __ffsll((unsigned long long)left) - 1;
      left &= left - 1;
      const float wj = __shfl(w, j, 64);
      float acc = 0.0f;
      for (int c = threadIdx.x; c < vec; c += 256) {
        float dy[8], o[8];
        unpack8(dy_row[c], dy);
        combine_load8<BF16_IN>(buf, (size_t)p, d, c, o);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          acc = fmaf(dy[i], o[i], acc);
          dy[i] *= wj;
        }
        reinterpret_cast<uint4*>(dO + (size_t)p * d)[c] = pack8(dy);
      }
      acc = wave_sum(acc);
      if (lane == 0) part[j][wv] = acc;
    }
  }
  __syncthreads();
  if (wv == 0) {
    float dw = 0.0f;
    if (local) dw = (part[lane][0] + part[lane][1]) + (part[lane][2] + part[lane][3]);
    if (!ok) dw = __builtin_nanf("");
    const float mean = wave_sum(lane < k ? w * dw : 0.0f);
    if (lane < k) {
      d_w[(size_t)t * k + lane] = dw;
      s_dl[lane] = w * (dw - mean);
      s_idx[lane] = idx;
    }
  }
  if (!d_logits) return;
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += 256) {
    float v = ok ? 0.0f : __builtin_nanf("");
    for (int j = 0; j < k; ++j)
      if (s_idx[j] == e) v += s_dl[j];
    d_logits[(size_t)t * E + e] = v;
  }
}

// Rows of at most 1024 columns: one wavefront per token, in which groups of GS
// lanes take a slot each (a row of 128 columns is 16 lanes' 8 columns: four
// slots at once). Against a workgroup per token, us: 14817 tokens of d = 128, k = 5
// 41 -> 13; 16384 tokens, k = 6, d = 512 77 -> 59, 768 95 -> 95, 1024 119 -> 127,
// 1280 152 -> 171; 2048 tokens, 512 10.7 -> 8.7, 1024 14.7 -> 14.3, 2048 26.6 -> 27.5; 64
// tokens the same up to 1536, then slower (3584: 8.3 -> 13.5).
template <bool BF16_IN, int GS>
__global__ __launch_bounds__(256) void combine_backward_narrow_kernel(
    const uint16_t* __restrict__ dY, const void* __restrict__ buf, const int32_t* __restrict__ tok_off,
    const int32_t* __restrict__ topk_idx, const float* __restrict__ topk_w, int T, int d, int k, int E, int e_begin,
    int El, int S, int cap, uint16_t* __restrict__ dO, float* __restrict__ d_w, float* __restrict__ d_logits) {
  __shared__ float s_dw[4][kMaxK];
  __shared__ int s_gate[4][kMaxK];  // gate of the token's n-th slot
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, t = blockIdx.x * 4 + wv;
  if (t >= T) return;  // whole wavefronts; nothing below waits for another one
  const int q = y_row_of_token(t, T, S);
  const int idx = lane < k ? topk_idx[(size_t)t * k + lane] : -1;
  const float w = lane < k ? topk_w[(size_t)t * k + lane] : 0.0f;
  const bool local = lane < k && (unsigned)(idx - e_begin) < (unsigned)El;
  const uint64_t mask = __ballot(local);
  const int p0 = tok_off[q], p1 = tok_off[q + 1], cnt = __popcll(mask);
  const bool ok = 0 <= p0 && p1 <= cap && p1 - p0 == cnt;  // as above
  if (lane < kMaxK) s_dw[wv][lane] = 0.0f;
  if (local) s_gate[wv][__popcll(mask & ((1ull << lane) - 1ull))] = lane;
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  if (ok) {
    const int vec = d >> 3, g = lane / GS, c0 = lane % GS;
    const uint4* dy_row = reinterpret_cast<const uint4*>(dY + (size_t)q * d);
    for (int n = g; n < cnt; n += 64 / GS) {
      const int j = s_gate[wv][n], p = p0 + n;
      const float wj = topk_w[(size_t)t * k + j];  // (the groups' loops differ in length: no shuffle here)
      float acc = 0.0f;
      for (int c = c0; c < vec; c += GS) {
        float dy[8], o[8];
        unpack8(dy_row[c], dy);
        combine_load8<BF16_IN>(buf, (size_t)p, d, c, o);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          acc = fmaf(dy[i], o[i], acc);
          dy[i] *= wj;
        }
        reinterpret_cast<uint4*>(dO + (size_t)p * d)[c] = pack8(dy);
      }
#pragma unroll
      for (int off = GS / 2; off > 0; off >>= 1) acc += __shfl_xor(acc, off, GS);
      if (c0 == 0) s_dw[wv][j] = acc;
    }
  }
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  float dw = lane < k ? s_dw[wv][lane] : 0.0f;
  if (!ok) dw = __builtin_nanf("");
  const float mean = wave_sum(lane < k ? w * dw : 0.0f);
  const float dl = w * (dw - mean);
  if (lane < k) d_w[(size_t)t * k + lane] = dw;
  if (!d_logits) return;
  for (int e0 = 0; e0 < E; e0 += 64) {
    const int e = e0 + lane;
    float v = ok ? 0.0f : __builtin_nanf("");
    for (int j = 0; j < k; ++j) {
      const int ej = __shfl(idx, j, 64);
      const float dj = __shfl(dl, j, 64);
      if (ej == e) v += dj;
    }
    if (e < E) d_logits[(size_t)t * E + e] = v;
  }
}

// dX[t] = the sum of the token's slots, ascending, in fp32, rounded once.
// Streaming: one thread per 8 columns of a token. Bound by HBM: on the share 25 us
// for 117 MB, 4.7 TB/s; 32768 tokens with four slots of d = 2048 120 us for 671
// MB (5.6 TB/s, part of it out of the last-level cache).
__global__ __launch_bounds__(256) void dispatch_backward_kernel(const uint16_t* __restrict__ dxs,
                                                                const int32_t* __restrict__ tok_off, int T, int d,
                                                                int S, int cap, uint16_t* __restrict__ dX,
                                                                float* __restrict__ dX32) {
  const int vec = d >> 3, n = T * vec;
  for (int i = blockIdx.x * 256 + threadIdx.x; i < n; i += gridDim.x * 256) {
    const int t = i / vec, c = i - t * vec;
    const int q = y_row_of_token(t, T, S);
    const int p0 = tok_off[q], p1 = tok_off[q + 1];
    const bool ok = 0 <= p0 && p0 <= p1 && p1 <= cap;
    float acc[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[j] = ok ? 0.0f : __builtin_nanf("");
    if (ok) {
      for (int p = p0; p < p1; ++p) {
        float v[8];
        unpack8(reinterpret_cast<const uint4*>(dxs + (size_t)p * d)[c], v);
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[j] += v[j];
      }
    }
    reinterpret_cast<uint4*>(dX + (size_t)t * d)[c] = pack8(acc);
    if (dX32) {
      float4* dst = reinterpret_cast<float4*>(dX32 + (size_t)t * d) + 2 * c;
      dst[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
      dst[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
    }
  }
}

}  // namespace

hipError_t launch_combine_backward(const moe_problem_t& p, const void* dY, const void* combine_buf,
                                   const int32_t* tok_off, const int32_t* topk_idx, const float* topk_w, void* dO,
                                   float* d_w, float* d_logits, hipStream_t s) {
  auto go = [&](auto kern, int blocks) {
    hipLaunchKernelGGL(kern, dim3(blocks), dim3(256), 0, s, static_cast<const uint16_t*>(dY), combine_buf, tok_off,
                       topk_idx, topk_w, p.T, p.d, p.k, p.E_global, p.e_begin, p.e_end - p.e_begin, p.num_segments,
                       (int)row_capacity(p), static_cast<uint16_t*>(dO), d_w, d_logits);
  };
  const bool bf16 = (p.flags & MOE_FLAG_BF16_COMBINE_BUF) != 0;
  const int four = (p.T + 3) / 4;
  if (p.d > 1024) {
    if (bf16) go(combine_backward_kernel<true>, p.T);
    else go(combine_backward_kernel<false>, p.T);
  } else if (p.d > 256) {
    if (bf16) go(combine_backward_narrow_kernel<true, 64>, four);
    else go(combine_backward_narrow_kernel<false, 64>, four);
  } else if (p.d > 128) {
    if (bf16) go(combine_backward_narrow_kernel<true, 32>, four);
    else go(combine_backward_narrow_kernel<false, 32>, four);
  } else {
    if (bf16) go(combine_backward_narrow_kernel<true, 16>, four);
    else go(combine_backward_narrow_kernel<false, 16>, four);
  }
  return hipGetLastError();
}

hipError_t launch_dispatch_backward(const moe_problem_t& p, const void* d_x_slots, const int32_t* tok_off, void* dX,
                                    float* dX_fp32, hipStream_t s) {
  const int64_t n = ((int64_t)p.T * (p.d >> 3) + 255) / 256;
  hipLaunchKernelGGL(dispatch_backward_kernel, dim3((unsigned)(n < 16384 ? n : 16384)), dim3(256), 0, s,
                     static_cast<const uint16_t*>(d_x_slots), tok_off, p.T, p.d, p.num_segments,
                     (int)row_capacity(p), static_cast<uint16_t*>(dX), dX_fp32);
  return hipGetLastError();
}

}  // namespace moe
