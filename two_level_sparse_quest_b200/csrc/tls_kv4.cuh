// tls_kv4.cuh -- the 4-bit KV cache's record and its conversions.
//
// One record per (sequence, KV head, token), 9 d / 8 bytes:
//   [K codes d/2][K scales d/16][V scales d/16][V codes d/2]
// A code is an e2m1 number (0, .5, 1, 1.5, 2, 3, 4, 6 and their negatives),
// channel 2i in the low nibble of byte i.  Sixteen channels share a scale
// byte b, the fp16 number with the bits b << 7 (five exponent bits, three
// mantissa bits, no sign).  Its range, 2^-17 to 10240 as written here, is why
// it is not e4m3: keys and values of any usual size need no second scale.
// A value code * scale has at most six significant bits and lies between
// 2^-18 and 61440, so it is exact in fp16 and in bf16: reading a row rounds
// nothing.  Scale byte 0xff is an fp16 NaN: a group of channels that held an
// infinity or a NaN reads back as NaN, as it would from a 16-bit cache.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

#include "tls_device.cuh"

namespace tls {

template <int D>
struct Kv4Rec {
  static constexpr int kCodes = D / 2;          // bytes of one row's codes
  static constexpr int kScales = D / 16;        // bytes of one row's scales
  static constexpr int kKS = kCodes;            // offset of the K scales
  static constexpr int kVS = kCodes + kScales;  // offset of the V scales
  static constexpr int kVC = kCodes + 2 * kScales;
  static constexpr int kBytes = 9 * D / 8;
  static constexpr int kChunk = D / 8;          // a record is nine of these; 16 bytes (d 128) or 8 (d 64)
};

constexpr int kKv4MaxScale = 0xE2;  // 10240: the largest scale whose product with a code fits fp16
constexpr int kKv4NanScale = 0xFF;

__device__ __forceinline__ float kv4_scale_value(int b) {
  return __half2float(__ushort_as_half(static_cast<unsigned short>(b << 7)));
}

// Scale byte of a group whose largest magnitude is amax (finite): amax / 6
// rounded to nearest even.  Above 2^-14 the byte is the fp32 number's exponent
// and top three mantissa bits; below, the scales are the multiples of 2^-17.
__device__ __forceinline__ int kv4_scale_byte(float amax) {
  const float s = __fdiv_rn(amax, 6.0f);
  if (s < 6.103515625e-05f) return __float2int_rn(s * 131072.0f);
  const uint32_t u = __float_as_uint(s);
  const int b = static_cast<int>((u + 0x7ffffu + ((u >> 20) & 1u)) >> 20) - (112 << 3);
  return min(b, kKv4MaxScale);
}

// Two fp32 -> one byte of e2m1 codes (x0 in the low nibble), nearest even, clamped to +-6.
__device__ __forceinline__ uint32_t e2m1_pack(float x0, float x1) {
  uint32_t r;
  asm("{\n .reg .b8 t;\n cvt.rn.satfinite.e2m1x2.f32 t, %2, %1;\n cvt.u32.u8 %0, t;\n}\n" : "=r"(r) : "f"(x0), "f"(x1));
  return r;
}

// The four bytes of w (eight codes) -> four fp16 pairs, low nibble first.
__device__ __forceinline__ void e2m1_unpack(uint32_t w, uint32_t &h0, uint32_t &h1, uint32_t &h2, uint32_t &h3) {
  asm("{\n .reg .b8 a, b, c, d;\n mov.b32 {a, b, c, d}, %4;\n"
      " cvt.rn.f16x2.e2m1x2 %0, a;\n cvt.rn.f16x2.e2m1x2 %1, b;\n"
      " cvt.rn.f16x2.e2m1x2 %2, c;\n cvt.rn.f16x2.e2m1x2 %3, d;\n}\n"
      : "=r"(h0), "=r"(h1), "=r"(h2), "=r"(h3)
      : "r"(w));
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// c += A B, fp16 in, fp32 accumulate; A 16 x 16 (row), B 16 x 8 (col).
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// One lane's part of a query row as fp16 pairs, for the contraction with fp16
// keys.  The row is multiplied by a power of two that puts its largest finite
// magnitude into [2^14, 2^15): bf16 has 8 significant bits, so every element
// down to 2^-28 of the largest is exact, and what is smaller loses less than
// 2^-39 of it.  `exps` is the largest biased exponent among the finite
// elements of the whole row; *undo receives the factor that undoes the
// multiplication.
__device__ __forceinline__ float q_norm(uint32_t exps, float *undo) {
  const int me = min(max(268 - static_cast<int>(exps), 1), 253);
  *undo = __uint_as_float(static_cast<uint32_t>(254 - me) << 23);
  return __uint_as_float(static_cast<uint32_t>(me) << 23);
}
// Largest biased exponent of the two bf16 in w that are finite (0 if none).
__device__ __forceinline__ uint32_t bf16_exps(uint32_t w) {
  const uint32_t a = (w >> 7) & 0xffu, b = (w >> 23) & 0xffu;
  return max(a == 0xffu ? 0u : a, b == 0xffu ? 0u : b);
}
__device__ __forceinline__ uint32_t q_to_f16(uint32_t w, float mult) {
  const __half2 h = __floats2half2_rn(bf16_lo(w) * mult, bf16_hi(w) * mult);
  return *reinterpret_cast<const uint32_t *>(&h);
}

}  // namespace tls
