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
// Values as bf16, for the tensor cores.  The eight magnitudes of a group, scaled, are
// a table of eight bf16, kept as their low and their high bytes; a byte permute looks
// up four values' bytes at once, by three bits each.  The sign bits are put on the
// high bytes before the two are laced: 15 integer instructions for 8 values, where
// shifting each pair's fields into place and multiplying takes 19 and 4 products.
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t q4_twice(uint32_t bf16) { return bf16 * 0x10001u; }
__device__ __forceinline__ uint32_t q4_mul2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
struct Q4Table {
  uint32_t lo[2], hi[2];
};
// the magnitudes times 2^(b - 127), a subnormal bf16 for b = 0
__device__ __forceinline__ Q4Table q4_table(uint32_t byte) {
  const uint32_t f = q4_twice(byte == kQ4Nan ? 0x7fc0u : byte == 0 ? 0x40u : byte << 7);
  // 0, 0.5 | 1, 1.5 | 2, 3 | 4, 6
  const uint32_t v0 = q4_mul2(0x3f000000u, f), v1 = q4_mul2(0x3fc03f80u, f), v2 = q4_mul2(0x40404000u, f),
                 v3 = q4_mul2(0x40c04080u, f);
  return {{__byte_perm(v0, v1, 0x6420), __byte_perm(v2, v3, 0x6420)}, {__byte_perm(v0, v1, 0x7531), __byte_perm(v2, v3, 0x7531)}};
}
// the eight values of four bytes, in order, two a register
__device__ __forceinline__ void q4_bf16x8(uint32_t w, const Q4Table &t, uint32_t *out) {
  const uint32_t m = w & 0x77777777u, m1 = m >> 16, up = w << 4;
  // the sign of value i at bit 7 of byte i: the even ones' come up by four bits
  const uint32_t s0 = __byte_perm(w, up, 0x1504), s1 = __byte_perm(w, up, 0x3726);
  const uint32_t h0 = __byte_perm(t.hi[0], t.hi[1], m) | (s0 & 0x80808080u), h1 = __byte_perm(t.hi[0], t.hi[1], m1) | (s1 & 0x80808080u);
  const uint32_t l0 = __byte_perm(t.lo[0], t.lo[1], m), l1 = __byte_perm(t.lo[0], t.lo[1], m1);
  out[0] = __byte_perm(l0, h0, 0x5140);
  out[1] = __byte_perm(l0, h0, 0x7362);
  out[2] = __byte_perm(l1, h1, 0x5140);
  out[3] = __byte_perm(l1, h1, 0x7362);
}
// a group's 32 values
__device__ __forceinline__ void q4_bf16x32(uint4 w, uint32_t byte, uint32_t *out) {
  const Q4Table t = q4_table(byte);
  q4_bf16x8(w.x, t, out);
  q4_bf16x8(w.y, t, out + 4);
  q4_bf16x8(w.z, t, out + 8);
  q4_bf16x8(w.w, t, out + 12);
}

}  // namespace
