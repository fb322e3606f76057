// MXFP4 codec (OCP Microscaling Formats, MXFP4: E2M1 elements, one E8M0 scale
// per 32 consecutive elements of a row).
//
// Per block of 32, with amax its largest magnitude:
//   scale   = 2^(floor(log2 amax) - 2), as the byte exponent + 127 (2 is the
//             largest E2M1 exponent; at least 2^-127; byte 127 for a block of
//             zeros; byte 255, the format's NaN, if an element is infinite or NaN)
//   element = E2M1 of x / scale, round to nearest even, at most 6 in magnitude
//             (a quotient in (6, 8) saturates; the sign of a zero is kept).
// Two elements per byte, the even one in the low nibble.
#include "moe_internal.h"

namespace moe {
namespace {

// 4 consecutive lanes hold a block, 8 elements each: 16 or 32 bytes in and 4
// out per lane, whole lines per wavefront. The quotients come from a multiply
// with the power of two 2^(127 - byte), which is exact wherever the element is
// not rounded to zero, and the hardware conversion rounds them (to nearest
// even, saturating). Bound by HBM: with the inverse behind it, 28672 x 4096 fp32
// values take 165 us for 830 MB, 5.0 TB/s.
template <bool F32_IN>
__global__ __launch_bounds__(256) void mxfp4_quantize_kernel(const void* __restrict__ x, int64_t n8,
                                                             uint32_t* __restrict__ codes,
                                                             uint8_t* __restrict__ scales) {
  // n8 (groups of 8 elements) is a multiple of 4, so a block's lanes run together
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n8; i += (int64_t)gridDim.x * 256) {
    uint32_t b[8];
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
    // magnitudes compare as integers (infinities and NaN above all others)
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, b[j] & 0x7FFFFFFFu);
    m = max(m, (uint32_t)__shfl_xor((int)m, 1, 64));
    m = max(m, (uint32_t)__shfl_xor((int)m, 2, 64));
    const bool bad = m >= 0x7F800000u;
    const int e = (int)(m >> 23) - 2;  // byte of floor(log2 amax) - 2 (fp32 subnormals: below 0)
    const int byte = m == 0 ? 127 : e > 0 ? e : 0;
    const float inv = bad ? 0.0f : __uint_as_float((uint32_t)(254 - byte) << 23);  // 2^(127 - byte)
    uint32_t c = 0;
    if (!bad) {
      c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, __uint_as_float(b[0]) * inv, __uint_as_float(b[1]) * inv, 1.0f, 0);
      c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, __uint_as_float(b[2]) * inv, __uint_as_float(b[3]) * inv, 1.0f, 1);
      c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, __uint_as_float(b[4]) * inv, __uint_as_float(b[5]) * inv, 1.0f, 2);
      c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, __uint_as_float(b[6]) * inv, __uint_as_float(b[7]) * inv, 1.0f, 3);
    }
    codes[i] = c;
    if ((i & 3) == 0) scales[i >> 2] = bad ? 255 : (uint8_t)byte;
  }
}

// The values codes and scales stand for: 8 elements per lane. The magnitude's
// bits, placed over fp32's exponent and top mantissa bit, are its value times
// 2^-126 (E2M1's one subnormal, 0.5, included), so two exact multiplies decode
// it.
template <bool F32_OUT>
__global__ __launch_bounds__(256) void mxfp4_dequantize_kernel(const uint32_t* __restrict__ codes,
                                                               const uint8_t* __restrict__ scales, int64_t n8,
                                                               void* __restrict__ out) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n8; i += (int64_t)gridDim.x * 256) {
    const uint32_t c = codes[i];
    const uint32_t byte = scales[i >> 2];
    const float s = byte == 255 ? __builtin_nanf("")
                                : __uint_as_float(byte ? byte << 23 : 1u << 22);  // 2^(byte - 127)
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t nib = c >> (4 * j);
      const float mag = __uint_as_float((nib & 7u) << 22) * 0x1p126f;
      v[j] = __uint_as_float(__float_as_uint(mag) | ((nib & 8u) << 28)) * s;
    }
    if constexpr (F32_OUT) {
      float4* dst = static_cast<float4*>(out) + 2 * i;
      dst[0] = make_float4(v[0], v[1], v[2], v[3]);
      dst[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
      uint4 o;
      o.x = pack_bf16(v[0], v[1]);
      o.y = pack_bf16(v[2], v[3]);
      o.z = pack_bf16(v[4], v[5]);
      o.w = pack_bf16(v[6], v[7]);
      static_cast<uint4*>(out)[i] = o;
    }
  }
}

unsigned codec_blocks(int64_t n8) {
  const int64_t b = (n8 + 255) / 256;
  return (unsigned)(b < 32768 ? b : 32768);
}

}  // namespace

hipError_t launch_mxfp4_quantize(const void* x, bool f32, int64_t n, uint8_t* codes, uint8_t* scales, hipStream_t s) {
  if (n == 0) return hipSuccess;
  auto go = [&](auto kern) {
    hipLaunchKernelGGL(kern, dim3(codec_blocks(n / 8)), dim3(256), 0, s, x, n / 8, reinterpret_cast<uint32_t*>(codes),
                       scales);
  };
  if (f32) go(mxfp4_quantize_kernel<true>);
  else go(mxfp4_quantize_kernel<false>);
  return hipGetLastError();
}

hipError_t launch_mxfp4_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t n, void* out, bool f32,
                                   hipStream_t s) {
  if (n == 0) return hipSuccess;
  auto go = [&](auto kern) {
    hipLaunchKernelGGL(kern, dim3(codec_blocks(n / 8)), dim3(256), 0, s, reinterpret_cast<const uint32_t*>(codes),
                       scales, n / 8, out);
  };
  if (f32) go(mxfp4_dequantize_kernel<true>);
  else go(mxfp4_dequantize_kernel<false>);
  return hipGetLastError();
}

}  // namespace moe
