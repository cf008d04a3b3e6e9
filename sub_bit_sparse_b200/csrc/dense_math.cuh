// Arithmetic shared by the 8-bit integer and gated feed-forward kernels.
#pragma once

#include "device_common.cuh"
#include "small_kernels.cuh"

namespace stq1 {

// ---- rows of signed 8-bit codes ----
// s = amax / 127 and inv = 127 / amax (IEEE divisions), code = the fp32 product
// src * inv rounded to nearest, ties to even.  |src * inv| <= 127 * (1 + 2^-23),
// so a code never leaves [-127, 127].  A row whose amax is below 2^-119, where
// 127 / amax nears the end of fp32's range, counts as zero (codes and scale 0).
// A row with an Inf or NaN gets codes 0 and that value / 127 as its scale, so
// that every product with it is NaN: 0 * Inf and 0 * NaN.
constexpr float kI8Max = 127.f;
constexpr float kI8MinAmax = 1.504632769052528e-36f;   // 2^-119

struct I8Scale {
  float inv, scale;
};
// amax_bits: the fp32 bits of max |src|, found by comparing bits as integers,
// which orders Inf and NaN above every finite value.
__device__ __forceinline__ I8Scale i8_scale(uint32_t amax_bits) {
  const float amax = __uint_as_float(amax_bits);
  I8Scale r;
  if (amax_bits >= 0x7F800000u) {
    r.inv = 0.f;
    r.scale = __fdiv_rn(amax, kI8Max);
  } else if (amax >= kI8MinAmax) {
    r.inv = __fdiv_rn(kI8Max, amax);
    r.scale = __fdiv_rn(amax, kI8Max);
  } else {
    r.inv = 0.f;
    r.scale = 0.f;
  }
  return r;
}

// Four codes in one word (first value in the low byte).  Adding 1.5 * 2^23
// rounds the product to an integer, ties to even, whose two's complement is
// then in the low mantissa bits.  With inv = 0 (a zero or non-finite row) the
// values must not be used: 0 * Inf is NaN.
__device__ __forceinline__ uint32_t i8_code(float v, float inv) {
  return __float_as_uint(__fadd_rn(__fmul_rn(v, inv), 12582912.f));
}
__device__ __forceinline__ uint32_t i8_pack4(float a, float b, float c, float d, float inv) {
  if (inv == 0.f) return 0u;
  const uint32_t lo = __byte_perm(i8_code(a, inv), i8_code(b, inv), 0x0040);
  const uint32_t hi = __byte_perm(i8_code(c, inv), i8_code(d, inv), 0x0040);
  return __byte_perm(lo, hi, 0x5410);
}

// Product of codes: the exact 32-bit sum, rounded to fp32, times the token's
// scale, times the channel's scale, each product rounded.
__device__ __forceinline__ float i8_value(int acc, float sx, float sw) {
  return __fmul_rn(__fmul_rn(__int2float_rn(acc), sx), sw);
}

// ---- the gated activation ----
__device__ __noinline__ uint32_t swiglu_bf16_slow(float g, float u) {
  const double gd = g;
  return bf16_bits_from_f64(gd / (1.0 + exp(-gd)) * static_cast<double>(u));
}

// bf16 bits of SiLU(g) * u, rounded once: the bits that swiglu_kernel's fp64
// evaluation gives.  In fp32, expf, the sum, the division and the product are
// together off by less than 8 units in the last place (1.01 + 0.5 + 2 + 0.5 of
// them, the division's approximation being good to 2), so the fp32 result decides the bf16 rounding unless its lower half lies
// within 16 units of the midpoint.  Those values (one in about 2000), the ones
// near the ends of fp32's range and NaN are evaluated in fp64.
__device__ __forceinline__ uint32_t swiglu_bf16(float g, float u) {
  const float s = __fdividef(g, 1.f + expf(-g));
  const float v = s * u;
  const uint32_t b = __float_as_uint(v);
  const uint32_t low = b & 0xFFFFu;
  const bool clear = low - 0x7FF0u > 0x20u;
  if (clear && fabsf(s) > 1e-30f && fabsf(v) > 1e-30f && fabsf(v) < 1e38f)
    return (b + 0x7FFFu + ((b >> 16) & 1u)) >> 16;
  return swiglu_bf16_slow(g, u);
}

__device__ __forceinline__ uint32_t bf16_bits_rn(float v) {
  return static_cast<uint32_t>(__bfloat16_as_ushort(__float2bfloat16_rn(v)));
}

// d/dg and d/du of dact * SiLU(g) * u.
__device__ __forceinline__ void glu_grads(float d, float g, float u, float& dg, float& du) {
  const float sg = __fdividef(1.f, 1.f + expf(-g));
  const float t = d * sg;
  dg = t * u * fmaf(g, 1.f - sg, 1.f);
  du = t * g;
}

}  // namespace stq1
