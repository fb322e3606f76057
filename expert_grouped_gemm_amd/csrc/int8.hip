// 8-bit integer codecs: rows with one fp32 scale each (the operands of
// moe_int8_linear1 / moe_int8_linear2), and OCP MXINT8 (one E8M0 scale per 32
// consecutive elements of a row: the checkpoints of activations).
#include <type_traits>

#include "moe_internal.h"

namespace moe {
namespace {

// ---------------------------------------------------------- values and codes

// 8 consecutive values as fp32 bits.
template <bool F32_IN>
__device__ __forceinline__ void load_bits8(const void* x, int64_t i, uint32_t (&b)[8]) {
  if constexpr (F32_IN) {
    const uint4* src = static_cast<const uint4*>(x) + 2 * i;
    const uint4 lo = src[0], hi = src[1];
    b[0] = lo.x; b[1] = lo.y; b[2] = lo.z; b[3] = lo.w;
    b[4] = hi.x; b[5] = hi.y; b[6] = hi.z; b[7] = hi.w;
  } else {
    const uint4 u = static_cast<const uint4*>(x)[i];
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      b[2 * j] = w[j] << 16;
      b[2 * j + 1] = w[j] & 0xFFFF0000u;
    }
  }
}

// Magnitudes compare as integers (infinities and NaN above all others).
__device__ __forceinline__ uint32_t max_magnitude(const uint32_t (&b)[8], uint32_t m) {
#pragma unroll
  for (int j = 0; j < 8; ++j) m = max(m, b[j] & 0x7FFFFFFFu);
  return m;
}

// A row's code of x is 127 x / amax rounded to nearest even, exactly: ratios
// of bf16 values often lie halfway between two codes. With x = X 2^a, amax =
// M 2^b and X, M of n bits, a quotient that is no tie is off every tie by
// 1 / (254 X) of it at least: 2^-16 for bf16 (n = 8), 2^-32 for fp32 (n = 24).
// The quotient by the rounded reciprocal is off by two roundings, far less, so
// rounding it to a few bits less than its format holds puts ties where they
// are and moves nothing else across one:
//   bf16: in fp32 (error below 2^-22), to 20 bits of mantissa (2^-21);
//   fp32: in fp64 (error below 2^-51), to 40 bits (2^-41).
// Adding 1.5 2^23 (2^52) then rounds to nearest even, and the low byte of the
// sum is the code in two's complement.
template <bool F32_IN>
struct RowCode;
template <>
struct RowCode<false> {
  float r;
  __device__ __forceinline__ explicit RowCode(float amax) : r(fminf(127.0f / amax, 0x1p126f)) {}
  __device__ __forceinline__ uint32_t operator()(uint32_t bits) const {
    const uint32_t q = (__float_as_uint(__uint_as_float(bits) * r) + 4u) & ~7u;
    return __float_as_uint(__uint_as_float(q) + 12582912.0f);
  }
};
template <>
struct RowCode<true> {
  double r;
  __device__ __forceinline__ explicit RowCode(float amax) : r(fmin(127.0 / (double)amax, 0x1p126)) {}
  __device__ __forceinline__ uint32_t operator()(uint32_t bits) const {
    const double p = (double)__uint_as_float(bits) * r;
    const uint64_t q = (__builtin_bit_cast(uint64_t, p) + 0x800u) & ~(uint64_t)0xFFF;
    return (uint32_t)__builtin_bit_cast(uint64_t, __builtin_bit_cast(double, q) + 6755399441055744.0);
  }
};

// The scale of a row: amax / 127, at least 2^-126 so that it and its reciprocal
// are normal numbers, and at most the largest whose 127-fold is finite (fp32's
// largest number / 127 rounds above it); 1 for a row of zeros.
__device__ __forceinline__ float row_scale(float amax) {
  return amax > 0.0f ? fminf(fmaxf(amax / 127.0f, 0x1p-126f), 0x1.020406p+121f) : 1.0f;
}

// ------------------------------------------------------ rows of 8-bit integers

// A row per LPR lanes, its values in registers between the maximum and the
// codes (CH groups of 8 per lane; a row with more is read again), so that a row
// is read once. Bound by HBM: 16384 x 14336 bf16 values 138 us for 705 MB, 5.1
// TB/s, over three sets of arrays in turn (160 between calls of the inverse, whose
// 940 MB of results are still on their way), fp32 ones 212 us for 1175 MB, 5.5 (243).
// The fewest lanes of 16, 64, 256 and 512 whose registers hold the row
// (bf16, us, with 16 / 64 / 256 / 512 lanes): 65536 x 128 7.7 / 22 / 63 / 136,
// x 512 19 / 24 / 66 / 142, x 2048 - / 77 / 96 / 177, 32768 x 7168 - / - / 130 /
// 147, 16384 x 14336 - / - / 134 / 131 (1024 lanes 192).
template <bool F32_IN, int LPR, int CH>
__global__ __launch_bounds__(LPR > 256 ? LPR : 256) void int8_quantize_kernel(const void* __restrict__ x, int64_t rows,
                                                                             int64_t g, uint2* __restrict__ codes,
                                                                             float* __restrict__ scales) {
  constexpr int NT = LPR > 256 ? LPR : 256, RPB = NT / LPR;  // rows per workgroup
  __shared__ uint32_t part[LPR > 64 ? NT / 64 : 1];
  const int l = threadIdx.x % LPR;
  for (int64_t r0 = (int64_t)blockIdx.x * RPB; r0 < rows; r0 += (int64_t)gridDim.x * RPB) {
    const int64_t r = r0 + threadIdx.x / LPR;
    const int64_t mine = r < rows ? g : 0, base = r * g;  // groups of this lane's row
    uint32_t b[CH][8];
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < CH; ++j)
      if (l + j * LPR < mine) load_bits8<F32_IN>(x, base + l + j * LPR, b[j]);
#pragma unroll
    for (int j = 0; j < CH; ++j)
      if (l + j * LPR < mine) m = max_magnitude(b[j], m);
    for (int64_t c = l + CH * LPR; c < mine; c += LPR) {
      uint32_t v[8];
      load_bits8<F32_IN>(x, base + c, v);
      m = max_magnitude(v, m);
    }
#pragma unroll
    for (int off = 1; off < (LPR < 64 ? LPR : 64); off <<= 1) m = max(m, (uint32_t)__shfl_xor((int)m, off, 64));
    if constexpr (LPR > 64) {
      __syncthreads();  // the last row's maxima have been read
      if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = m;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < NT / 64; ++i) m = max(m, part[i]);
    }
    const bool bad = m >= 0x7F800000u;
    const float amax = __uint_as_float(m);
    const RowCode<F32_IN> code(amax);
    auto put = [&](int64_t c, const uint32_t(&v)[8]) {
      uint2 o = make_uint2(0, 0);
      if (m != 0 && !bad) {
        o.x = low_bytes(code(v[0]), code(v[1]), code(v[2]), code(v[3]));
        o.y = low_bytes(code(v[4]), code(v[5]), code(v[6]), code(v[7]));
      }
      codes[base + c] = o;
    };
#pragma unroll
    for (int j = 0; j < CH; ++j)
      if (l + j * LPR < mine) put(l + j * LPR, b[j]);
    for (int64_t c = l + CH * LPR; c < mine; c += LPR) {
      uint32_t v[8];
      load_bits8<F32_IN>(x, base + c, v);
      put(c, v);
    }
    if (l == 0 && mine) scales[r] = bad ? __builtin_nanf("") : row_scale(amax);
  }
}

// code * scale: four values per lane. A lane's group and row advance by the
// grid's step, drow rows and dcol groups of gpr to a row. Bound by HBM: 16384 x
// 14336 to fp32 212 us for 1175 MB, 5.5 TB/s, to bf16 146 for 705, 4.8.
template <bool F32_OUT>
__global__ __launch_bounds__(256) void int8_dequantize_kernel(const uint32_t* __restrict__ codes,
                                                              const float* __restrict__ scales, int64_t n4,
                                                              int64_t gpr, int64_t drow, int64_t dcol,
                                                              void* __restrict__ out) {
  int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  int64_t row = i / gpr, col = i - row * gpr;
  for (; i < n4; i += (int64_t)gridDim.x * 256) {
    const int c = (int)codes[i];
    const float s = scales[row];
    const float v[4] = {(float)(int8_t)c * s, (float)(int8_t)(c >> 8) * s, (float)(int8_t)(c >> 16) * s,
                        (float)(c >> 24) * s};
    if constexpr (F32_OUT) static_cast<float4*>(out)[i] = make_float4(v[0], v[1], v[2], v[3]);
    else static_cast<uint2*>(out)[i] = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
    row += drow;
    col += dcol;
    if (col >= gpr) {
      col -= gpr;
      ++row;
    }
  }
}

// ------------------------------------------------------------------- MXINT8

// Per block of 32: scale 2^floor(log2 amax) as the byte exponent + 127 (at
// least byte 7, so that an element's step 2^(byte - 133) is a normal number;
// byte 127 for zeros, 255 where an element is infinite or NaN), element = x /
// step rounded to nearest even, at most 127 in magnitude. The step is a power
// of two, so the quotient is exact and so is every value read back, in bf16
// too (7 bits of magnitude). Four consecutive lanes hold a block, 8 elements
// each. Bound by HBM: 32768 x 7168 bf16 values 138 us for 712 MB, 5.2 TB/s, and
// back 115 us, 6.2; fp32 ones 217 us for 1182 MB, 5.4, and back 296, 4.0.
template <bool F32_IN>
__global__ __launch_bounds__(256) void mxint8_quantize_kernel(const void* __restrict__ x, int64_t n8,
                                                              uint2* __restrict__ codes,
                                                              uint8_t* __restrict__ scales) {
  // n8 (groups of 8 elements) is a multiple of 4, so a block's lanes run together
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n8; i += (int64_t)gridDim.x * 256) {
    uint32_t b[8];
    load_bits8<F32_IN>(x, i, b);
    uint32_t m = max_magnitude(b, 0);
    m = max(m, (uint32_t)__shfl_xor((int)m, 1, 64));
    m = max(m, (uint32_t)__shfl_xor((int)m, 2, 64));
    const uint32_t byte = mxint8_scale(m);
    uint32_t c[8];
    const float inv = mxint8_inverse_step(byte);
#pragma unroll
    for (int j = 0; j < 8; ++j) c[j] = mxint8_code(__uint_as_float(b[j]), inv);
    uint2 o = make_uint2(low_bytes(c[0], c[1], c[2], c[3]), low_bytes(c[4], c[5], c[6], c[7]));
    if (byte == 255) o = make_uint2(0, 0);
    codes[i] = o;
    if ((i & 3) == 0) scales[i >> 2] = (uint8_t)byte;
  }
}

template <bool F32_OUT>
__global__ __launch_bounds__(256) void mxint8_dequantize_kernel(const uint2* __restrict__ codes,
                                                                const uint8_t* __restrict__ scales, int64_t n8,
                                                                void* __restrict__ out) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n8; i += (int64_t)gridDim.x * 256) {
    float v[8];
    mxint8_values8(codes[i], mxint8_step(scales[i >> 2]), v);
    if constexpr (F32_OUT) {
      float4* dst = static_cast<float4*>(out) + 2 * i;
      dst[0] = make_float4(v[0], v[1], v[2], v[3]);
      dst[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
      static_cast<uint4*>(out)[i] = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
                                               pack_bf16(v[6], v[7]));
    }
  }
}

unsigned codec_blocks(int64_t lanes) {
  const int64_t b = (lanes + 255) / 256;
  return (unsigned)(b < 32768 ? b : 32768);
}

}  // namespace

hipError_t launch_int8_quantize(const void* x, bool f32, int64_t rows, int64_t cols, int8_t* codes, float* scales,
                                hipStream_t s) {
  if (rows == 0) return hipSuccess;
  auto go = [&](auto kern, int lpr) {
    const int nt = lpr > 256 ? lpr : 256;
    const int64_t blocks = (rows + nt / lpr - 1) / (nt / lpr);
    hipLaunchKernelGGL(kern, dim3((unsigned)(blocks < (1 << 20) ? blocks : (1 << 20))), dim3(nt), 0, s, x, rows,
                       cols / 8, reinterpret_cast<uint2*>(codes), scales);
  };
  auto pick = [&](auto f) {
    constexpr bool F = decltype(f)::value;
    if (cols <= 512) go(int8_quantize_kernel<F, 16, 4>, 16);
    else if (cols <= 2048) go(int8_quantize_kernel<F, 64, 4>, 64);
    else if (cols <= 8192) go(int8_quantize_kernel<F, 256, 4>, 256);
    else go(int8_quantize_kernel<F, 512, 4>, 512);
  };
  if (f32) pick(std::true_type{});
  else pick(std::false_type{});
  return hipGetLastError();
}

hipError_t launch_int8_dequantize(const int8_t* codes, const float* scales, int64_t rows, int64_t cols, void* out,
                                  bool f32, hipStream_t s) {
  if (rows == 0) return hipSuccess;
  const int64_t n4 = rows * (cols / 4), gpr = cols / 4;
  const unsigned blocks = codec_blocks(n4);
  const int64_t step = (int64_t)blocks * 256;
  auto go = [&](auto kern) {
    hipLaunchKernelGGL(kern, dim3(blocks), dim3(256), 0, s, reinterpret_cast<const uint32_t*>(codes), scales, n4, gpr,
                       step / gpr, step % gpr, out);
  };
  if (f32) go(int8_dequantize_kernel<true>);
  else go(int8_dequantize_kernel<false>);
  return hipGetLastError();
}

hipError_t launch_mxint8_quantize(const void* x, bool f32, int64_t n, int8_t* codes, uint8_t* scales, hipStream_t s) {
  if (n == 0) return hipSuccess;
  auto go = [&](auto kern) {
    hipLaunchKernelGGL(kern, dim3(codec_blocks(n / 8)), dim3(256), 0, s, x, n / 8, reinterpret_cast<uint2*>(codes),
                       scales);
  };
  if (f32) go(mxint8_quantize_kernel<true>);
  else go(mxint8_quantize_kernel<false>);
  return hipGetLastError();
}

hipError_t launch_mxint8_dequantize(const int8_t* codes, const uint8_t* scales, int64_t n, void* out, bool f32,
                                    hipStream_t s) {
  if (n == 0) return hipSuccess;
  auto go = [&](auto kern) {
    hipLaunchKernelGGL(kern, dim3(codec_blocks(n / 8)), dim3(256), 0, s, reinterpret_cast<const uint2*>(codes), scales,
                       n / 8, out);
  };
  if (f32) go(mxint8_dequantize_kernel<true>);
  else go(mxint8_dequantize_kernel<false>);
  return hipGetLastError();
}

}  // namespace moe
