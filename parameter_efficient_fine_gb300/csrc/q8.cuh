// The 8-bit form of a matrix, on the device: one E4M3 byte per element and one
// E8M0 byte b, a scale 2^(b - 127), per block of 128 columns.
//
// The scale of a block is the smallest power of two that brings its largest
// finite magnitude to at most 448 = 1.75 * 2^8 (the largest E4M3 value), and
// at least 2^-117, so that every value an 8-bit form stands for is exact in
// bf16 (4 significant bits, no exponent below 2^-126).  A power of two makes
// the division by the scale exact and is what the tensor core's block scaling
// takes.  A NaN or an infinity becomes NaN (0x7f) and does not enter its
// block's scale.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace {

constexpr int kQBlock = 128;       // columns per scale
constexpr int kMinScale = 10;      // 2^-117

// bits of |v|; 0 for a NaN or an infinity
__device__ __forceinline__ uint32_t finite_bits(float v) {
  const uint32_t a = __float_as_uint(v) & 0x7fffffffu;
  return a < 0x7f800000u ? a : 0u;
}
constexpr uint32_t kInfBits = 0x7f800000u;
// scale byte of a block whose largest finite magnitude has the bits `amax`:
// the exponent rounded up past 1.75, minus 8
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax) {
  const int e = static_cast<int>((amax + 0x1fffffu) >> 23) - 8;
  return static_cast<uint32_t>(max(e, kMinScale));
}
__device__ __forceinline__ float scale_value(uint32_t byte) { return __uint_as_float(byte << 23); }
__device__ __forceinline__ float scale_inverse(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }

// two values / scale as E4M3 bytes (a low, b high); a NaN gives 0x7f
__device__ __forceinline__ uint32_t quant2(float a, float b, float inv) {
  return __nv_cvt_float2_to_fp8x2(make_float2(a * inv, b * inv), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ uint32_t quant4(const float *v, float inv) {
  return quant2(v[0], v[1], inv) | (quant2(v[2], v[3], inv) << 16);
}
// an infinity as the NaN that it is stored as (the conversion would saturate it)
__device__ __forceinline__ float inf_to_nan(float v) { return fmaf(v, 0.0f, v); }
// two E4M3 bytes (low half of w) times the scale
__device__ __forceinline__ float2 dequant2(uint32_t w, float s) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w), __NV_E4M3);
  const float2 f = __half22float2(__half2(h));
  return make_float2(f.x * s, f.y * s);
}
__device__ __forceinline__ void dequant4(uint32_t w, float s, float *v) {
  const float2 a = dequant2(w & 0xffffu, s), b = dequant2(w >> 16, s);
  v[0] = a.x;
  v[1] = a.y;
  v[2] = b.x;
  v[3] = b.y;
}

}  // namespace
