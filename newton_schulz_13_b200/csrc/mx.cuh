// 8-bit activation checkpoints: e4m3 elements in blocks of 32 along a row, each block under one
// power-of-two scale (the OCP "microscaling" MXFP8 layout: e4m3 element codes, e8m0 scale codes).
//
// The scale is 2^e for the smallest e with max |x| <= 448 2^e (448 is e4m3's largest value), so no
// element saturates, with e held to [-117, 119]: with e >= -117 every restored value (at least
// 2^-9 2^-117 unless zero) is a normal bf16 number and so exact in bf16, and 448 2^119 is the
// largest product that bf16 holds (larger inputs saturate there). A block that holds an infinity
// or a NaN gets the NaN scale (code 255) and restores as NaN everywhere: an 8-bit block has no
// scale that would keep its other elements.
#pragma once

#include <cuda_fp8.h>
#include <stdint.h>

namespace muon {

constexpr int kMxBlock = 32;
constexpr int kMxExpMin = -117, kMxExpMax = 119;
constexpr uint32_t kMxNan = 255;

// Code of the scale for the largest |x| of a block, given as the bits of that float (an unsigned
// maximum of |x| bits orders finite values, then infinity, then NaN).
__device__ __forceinline__ uint32_t mx_scale_code(uint32_t amax_bits) {
  if (amax_bits >= 0x7f800000u) return kMxNan;
  // 448 = 1.75 2^8: x = f 2^E with f in [1, 2) needs e = E - 8, or one more when f > 1.75 (then the
  // sum carries into the exponent)
  const int code = (int)((amax_bits + 0x1fffffu) >> 23) - 8;
  return (uint32_t)max(kMxExpMin + 127, min(kMxExpMax + 127, code));
}

// Bits of max |v| of eight values; NaN if one of them is.
__device__ __forceinline__ uint32_t mx_amax8(const float (&v)[8]) {
  float m = fabsf(v[0]);
  asm("max.NaN.f32 %0, %0, %1, %2;" : "+f"(m) : "f"(fabsf(v[1])), "f"(fabsf(v[2])));
  asm("max.NaN.f32 %0, %0, %1, %2;" : "+f"(m) : "f"(fabsf(v[3])), "f"(fabsf(v[4])));
  asm("max.NaN.f32 %0, %0, %1, %2;" : "+f"(m) : "f"(fabsf(v[5])), "f"(fabsf(v[6])));
  asm("max.NaN.f32 %0, %0, %1;" : "+f"(m) : "f"(fabsf(v[7])));
  return __float_as_uint(m) & 0x7fffffffu;
}

// 2^-e as a float for a scale code that mx_scale_code returned (not for the NaN code).
__device__ __forceinline__ float mx_inv_scale(uint32_t code) {
  return __uint_as_float((254u - code) << 23);
}

// 2^e as a float for any e8m0 code: 2^-127 (code 0) is a subnormal float, code 255 is NaN.
__device__ __forceinline__ float mx_scale(uint32_t code) {
  return code == 0u ? __uint_as_float(0x00400000u)
                    : (code == kMxNan ? __uint_as_float(0x7fc00000u) : __uint_as_float(code << 23));
}

// Two e4m3 codes of a and b (rounded to nearest even, saturating), a in the low byte.
__device__ __forceinline__ uint32_t mx_pack2(float a, float b) {
  return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}

// Codes of v under scale code `code`; NaN codes for a NaN block.
__device__ __forceinline__ uint32_t mx_pack1(float v, uint32_t code) {
  if (code == kMxNan) return 0x7fu;
  return __nv_cvt_float_to_fp8(v * mx_inv_scale(code), __NV_SATFINITE, __NV_E4M3);
}

__device__ __forceinline__ uint2 mx_pack8(const float (&v)[8], uint32_t code) {
  if (code == kMxNan) return make_uint2(0x7f7f7f7fu, 0x7f7f7f7fu);
  const float2 s = make_float2(mx_inv_scale(code), mx_inv_scale(code));
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = __fmul2_rn(make_float2(v[2 * i], v[2 * i + 1]), s);
    c[i] = mx_pack2(p.x, p.y);
  }
  return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

// Values of the two e4m3 codes in the low 16 bits.
__device__ __forceinline__ float2 mx_unpack2(uint32_t codes) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(codes & 0xffffu), __NV_E4M3);
  return __half22float2(__half2(h));
}

}  // namespace muon
