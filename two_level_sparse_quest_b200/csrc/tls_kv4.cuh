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

// x / y for a y whose approximate reciprocal is r, by one residual correction
// (q + r (x - q y), P. Markstein, IBM J. Res. Dev. 34, 1990): it leaves the
// quotient within 2^-40, which rounds an exact one (the ties below) exactly.
__device__ __forceinline__ float quotient(float x, float y, float r) {
  const float q = x * r;
  return fmaf(fmaf(-q, y, x), r, q);
}
__device__ __forceinline__ float rcp_approx(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Scale byte of a group whose largest magnitude is amax (a finite bf16):
// amax / 6 rounded to nearest even.  Above 2^-14 the byte is the fp32 number's
// exponent and top three mantissa bits; below, the scales are the multiples of
// 2^-17.  (amax has 8 significant bits: amax / 6 is a tie exactly, or further
// from one than fp32's rounding.)
__device__ __forceinline__ int kv4_scale_byte(float amax) {
  const float s = quotient(amax, 6.0f, 0.16666667f);
  if (s < 6.103515625e-05f) return __float2int_rn(s * 131072.0f);
  const uint32_t u = __float_as_uint(s);
  const int b = static_cast<int>((u + 0x7ffffu + ((u >> 20) & 1u)) >> 20) - (112 << 3);
  return min(b, kKv4MaxScale);
}

// Eight bf16 (w[0..3]) over the scale s (reciprocal about r) -> eight e2m1
// codes, nearest even, clamped to +-6, the first in the low nibble.
__device__ __forceinline__ uint32_t e2m1_codes(const uint32_t (&w)[4], float s, float r) {
  unsigned long long ns, rr;
  asm("mov.b64 %0, {%1, %1};" : "=l"(ns) : "f"(-s));
  asm("mov.b64 %0, {%1, %1};" : "=l"(rr) : "f"(r));
  float q[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {  // quotient(), two channels at once
    unsigned long long x, t, e;
    asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(bf16_lo(w[i])), "f"(bf16_hi(w[i])));
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(t) : "l"(x), "l"(rr));
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(e) : "l"(t), "l"(ns), "l"(x));
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(t) : "l"(e), "l"(rr), "l"(t));
    asm("mov.b64 {%0, %1}, %2;" : "=f"(q[2 * i]), "=f"(q[2 * i + 1]) : "l"(t));
  }
  uint32_t c;
  asm("{\n .reg .b8 a, b, c, d;\n"
      " cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
      " cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n"
      " mov.b32 %0, {a, b, c, d};\n}\n"
      : "=r"(c)
      : "f"(q[0]), "f"(q[1]), "f"(q[2]), "f"(q[3]), "f"(q[4]), "f"(q[5]), "f"(q[6]), "f"(q[7]));
  return c;
}

// The four bytes of w (eight codes) -> four fp16 pairs, low nibble first.
// (This, hmul2 and mma_f16 are volatile to keep the order in which their callers
// alternate the three pipes: 1.4 % of the attention over every token.)
__device__ __forceinline__ void e2m1_unpack(uint32_t w, uint32_t &h0, uint32_t &h1, uint32_t &h2, uint32_t &h3) {
  asm volatile("{\n .reg .b8 a, b, c, d;\n mov.b32 {a, b, c, d}, %4;\n"
      " cvt.rn.f16x2.e2m1x2 %0, a;\n cvt.rn.f16x2.e2m1x2 %1, b;\n"
      " cvt.rn.f16x2.e2m1x2 %2, c;\n cvt.rn.f16x2.e2m1x2 %3, d;\n}\n"
      : "=r"(h0), "=r"(h1), "=r"(h2), "=r"(h3)
      : "r"(w));
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm volatile("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// c += A B, fp16 in, fp32 accumulate; A 16 x 16 (row), B 16 x 8 (col).
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
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
