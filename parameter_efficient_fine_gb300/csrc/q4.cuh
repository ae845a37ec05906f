// The 4-bit form of a matrix, on the device: one E2M1 value per element (0, .5,
// 1, 1.5, 2, 3, 4, 6 and a sign), two a byte with the even column in the low
// half, and one E8M0 byte b, a scale 2^(b - 127), per 32 columns of a row.
//
// The scale of a group is the smallest power of two that brings its largest
// magnitude to at most 6 = 1.5 * 2^2, and at least 2^-125, so that every value
// that a store gives is exact in bf16 (2 significant bits, no exponent below
// 2^-126) and the division by the scale is exact.  E2M1 has no NaN: a group that
// holds a NaN or an infinity gets the byte 255, which makes all of it NaN.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp4.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace {

constexpr int kQ4Group = 32;       // columns per scale
constexpr int kQ4MinScale = 2;     // 2^-125
constexpr int kQ4Nan = 255;

// scale byte of a group whose largest magnitude has the bits `amax` (0x7f800000
// and above: not finite): the exponent rounded up past 1.5, minus 2
__device__ __forceinline__ uint32_t q4_scale_byte(uint32_t amax) {
  const int e = static_cast<int>((amax + 0x3fffffu) >> 23) - 2;
  return amax >= 0x7f800000u ? kQ4Nan : static_cast<uint32_t>(max(e, kQ4MinScale));
}
// 1 / scale; 0 for the NaN byte, whose group stores zeros
__device__ __forceinline__ float q4_inverse(uint32_t byte) {
  return byte == kQ4Nan ? 0.0f : __uint_as_float((254u - byte) << 23);
}
// 2^(byte - 127) for every byte: 0 is a subnormal number, 255 NaN
__device__ __forceinline__ float q4_scale(uint32_t byte) {
  const uint32_t bits = byte == 0 ? 0x400000u : byte << 23;
  return __uint_as_float(byte == kQ4Nan ? 0x7fc00000u : bits);
}
// two values / scale as a byte, a in the low half.  A NaN stores as a number: its
// group's scale says NaN
__device__ __forceinline__ uint32_t q4_quant2(float a, float b, float inv) {
  return __nv_cvt_float2_to_fp4x2(make_float2(a * inv, b * inv), __NV_E2M1, cudaRoundNearest);
}
// the two values of a byte, unscaled
__device__ __forceinline__ float2 q4_value2(uint32_t byte) {
  const __half2_raw h = __nv_cvt_fp4x2_to_halfraw2(static_cast<__nv_fp4x2_storage_t>(byte), __NV_E2M1);
  return __half22float2(__half2(h));
}

// ---------------------------------------------------------------------------
// Values as bf16, for the tensor cores.  The three magnitude bits at bits 8-6 of a
// bf16 are the value times 2^-126, its subnormal range included, so one
// multiplication by 2^(b - 1) scales it.  That factor is a bf16 up to b = 128;
// above, 2^127 and a second factor.  A nibble times 2^12 + 2^6 has its sign at bit
// 15 and its magnitude at bits 8-6, and two of them 16 bits apart do not meet: for
// 8 values 11 instructions of the integer pipe, which bounds the conversion, and 8
// of the other.
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t q4_twice(uint32_t bf16) { return bf16 * 0x10001u; }
__device__ __forceinline__ uint32_t q4_factor(uint32_t byte) {
  return q4_twice(byte == kQ4Nan ? 0x7fc0u : (min(byte, 128u) + 126u) << 7);
}
__device__ __forceinline__ uint32_t q4_mul2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// bytes of a and b by `selector`'s four-bit fields; 8 on a field whose byte is below 128 gives zero
__device__ __forceinline__ uint32_t q4_prmt(uint32_t a, uint32_t b, uint32_t selector) {
  uint32_t d;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(selector));
  return d;
}
// the eight values of four bytes, in order, two a register
__device__ __forceinline__ void q4_bf16x8(uint32_t w, uint32_t factor, uint32_t *out) {
  const uint32_t even = w & 0x0f0f0f0fu, odd = (w >> 4) & 0x0f0f0f0fu;
  out[0] = q4_mul2(q4_prmt(even, odd, 0xc480) * 0x1040u & 0x81c081c0u, factor);
  out[1] = q4_mul2(q4_prmt(even, odd, 0xd591) * 0x1040u & 0x81c081c0u, factor);
  out[2] = q4_mul2(q4_prmt(even, odd, 0xe6a2) * 0x1040u & 0x81c081c0u, factor);
  out[3] = q4_mul2(q4_prmt(even, odd, 0xf7b3) * 0x1040u & 0x81c081c0u, factor);
}
// a group's 32 values
__device__ __forceinline__ void q4_bf16x32(uint4 w, uint32_t byte, uint32_t *out) {
  const uint32_t f = q4_factor(byte);
  q4_bf16x8(w.x, f, out);
  q4_bf16x8(w.y, f, out + 4);
  q4_bf16x8(w.z, f, out + 8);
  q4_bf16x8(w.w, f, out + 12);
  if (byte > 128 && byte != kQ4Nan) {
    const uint32_t g = q4_twice((byte - 1u) << 7);     // 2^(b - 128)
#pragma unroll
    for (int i = 0; i < 16; ++i) out[i] = q4_mul2(out[i], g);
  }
}

}  // namespace
