// Rounding to cache codes, shared by the kernels that write caches: fp32 values
// to int8, float8 e4m3fn and e2m1 codes, and back where a kernel needs it.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

#include "device.cuh"

namespace i8kv {

// A product with a rounded reciprocal is within its 2^-22 of the rounded quotient: codes of
// both ends of a wider interval that agree are the quotient's.
constexpr float kLoBound = 1.f - 0x1p-21f;
constexpr float kHiBound = 1.f + 0x1p-21f;

__device__ __forceinline__ float nan_to_zero(float q) { return q != q ? 0.f : q; }

__device__ __forceinline__ float int8_code(float q) {
  return fminf(fmaxf(rintf(q), -127.f), 127.f);
}

__device__ __forceinline__ uint32_t int8_byte(float c) {
  return static_cast<uint32_t>(static_cast<int32_t>(c)) & 0xFFu;
}

// Two floats -> two float8 e4m3fn bytes (lo in bits 0..7), nearest even,
// saturating to the largest finite magnitude.
__device__ __forceinline__ uint32_t e4m3x2_of(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// Eight floats -> eight e2m1 codes, value j in nibble j: nearest even,
// saturating to +-6.
__device__ __forceinline__ uint32_t e2m1x8_of(const float (&q)[8]) {
  uint32_t r;
  asm("{\n .reg .b8 b0, b1, b2, b3;\n"
      " cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n"
      " cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n"
      " cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n"
      " cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n"
      " mov.b32 %0, {b0, b1, b2, b3};\n}\n"
      : "=r"(r)
      : "f"(q[0]), "f"(q[1]), "f"(q[2]), "f"(q[3]), "f"(q[4]), "f"(q[5]), "f"(q[6]), "f"(q[7]));
  return r;
}

// The value of one float8 e4m3fn byte.
__device__ __forceinline__ float e4m3_value(uint32_t byte) {
  uint32_t lo, hi;
  e4m3x4_to_h2x2(byte, lo, hi);
  return __half2float(__ushort_as_half(static_cast<unsigned short>(lo & 0xFFFFu)));
}

// Eight e2m1 codes (nibble j: value j) -> four half2 (2j, 2j + 1), exact.
__device__ __forceinline__ void e2m1x8_to_h2x4(uint32_t w, uint32_t& h0, uint32_t& h1,
                                               uint32_t& h2, uint32_t& h3) {
  asm("{\n .reg .b8 b0, b1, b2, b3;\n mov.b32 {b0, b1, b2, b3}, %4;\n"
      " cvt.rn.f16x2.e2m1x2 %0, b0;\n cvt.rn.f16x2.e2m1x2 %1, b1;\n"
      " cvt.rn.f16x2.e2m1x2 %2, b2;\n cvt.rn.f16x2.e2m1x2 %3, b3;\n}\n"
      : "=r"(h0), "=r"(h1), "=r"(h2), "=r"(h3)
      : "r"(w));
}

// Byte offset of the record of (slot, KV head g) in an MX4 cache, and the token's
// place in it.
__device__ __forceinline__ long long mx4_record(int slot, int g, int Hkv, int D, int bs,
                                                int bs_shift, int& tok) {
  const int blk = bs_shift >= 0 ? slot >> bs_shift : slot / bs;
  const int off = slot - blk * bs;
  tok = off & 15;
  return (((long long)blk * Hkv + g) * (bs >> 4) + (off >> 4)) * (18LL * D);
}

}  // namespace i8kv
