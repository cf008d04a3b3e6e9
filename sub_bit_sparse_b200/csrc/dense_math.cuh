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
// bf16 bits of SiLU(g) * u, rounded once: the bits that swiglu_kernel's fp64
// evaluation gives, in three steps.
//
// 1. fp32: expf (1 unit in the last place), the sum (1/2), the division (2)
//    and the product (1/2) are together off by at most 4 halves of a binade's
//    unit, so by less than 9 units of the result.  It decides the rounding
//    unless its lower half lies within 9 units of the midpoint: one value in
//    about 3400.
// 2. Those, in fp64 by a short evaluation good to 2^-44: e^-g as 2^k times the
//    Taylor polynomial on |r| <= ln(2) / 2 (r^12 / 12! < 2^-47), the
//    reciprocal by one Newton step from fp32's.  Short, because a warp comes
//    here about once per tile: with exp, a division and a general rounding the
//    instruction fetches alone took the 4096-token int8 layer from 163 to 196 us.
//    It builds 2^k in the exponent's bits and so takes gates below 700 only
//    (k > -1011; from below, |SiLU(g)| > 1e-30 keeps g above -74), and leaves to
//    step 3 what lies within 2^-40 of the midpoint, exact midpoints among it: its
//    own error then decides nothing.
// 3. Those, farther gates, values near the ends of fp32's range and NaN as
//    swiglu_kernel does.
__device__ __noinline__ uint32_t swiglu_bf16_ends(float g, float u) {
  const double gd = g;
  return bf16_bits_from_f64(gd / (1.0 + exp(-gd)) * static_cast<double>(u));
}
__device__ __noinline__ uint32_t swiglu_bf16_border(float g, float u) {
  const double x = -static_cast<double>(g);
  const int k = __float2int_rn(g * -1.44269504f);
  const double r = fma(static_cast<double>(k), -0.693147180559945309, x);
  double e = 1.0 / 39916800.0;                       // 1 / 11!
#pragma unroll
  for (int n = 11; n >= 1; --n) {
    constexpr double kInvFact[11] = {1.0, 1.0, 1.0 / 2, 1.0 / 6, 1.0 / 24, 1.0 / 120, 1.0 / 720, 1.0 / 5040,
                                     1.0 / 40320, 1.0 / 362880, 1.0 / 3628800};
    e = fma(e, r, kInvFact[n - 1]);
  }
  e = __hiloint2double(__double2hiint(e) + (k << 20), __double2loint(e));
  const double d = 1.0 + e;
  double rc = static_cast<double>(__frcp_rn(static_cast<float>(d)));
  rc = fma(rc, fma(-d, rc, 1.0), rc);
  const double v = static_cast<double>(g) * static_cast<double>(u) * rc;
  // 19 bits: sign, 11 of exponent, 7 of mantissa, rounded to nearest; 2^12 of the
  // 52 mantissa bits' units are 2^-40
  const unsigned long long b = static_cast<unsigned long long>(__double_as_longlong(v));
  if ((b & ((1ull << 45) - 1)) - ((1ull << 44) - (1ull << 12)) <= 1ull << 13) return swiglu_bf16_ends(g, u);
  const uint32_t q = static_cast<uint32_t>((b + (1ull << 44)) >> 45);
  return ((q & 0x3FFFFu) - (896u << 7)) | ((q >> 18) << 15);
}
// The fp32 step: bits rounded from v; false where another step must decide.
__device__ __forceinline__ bool swiglu_bf16_fast(float g, float u, uint32_t& bits) {
  const float s = __fdividef(g, 1.f + expf(-g));
  const float v = s * u;
  const uint32_t b = __float_as_uint(v);
  bits = (b + 0x7FFFu + ((b >> 16) & 1u)) >> 16;
  return fabsf(s) > 1e-30f && fabsf(v) > 1e-30f && fabsf(v) < 1e38f && (b & 0xFFFFu) - 0x7FF7u > 18u;
}
__device__ __noinline__ uint32_t swiglu_bf16_slow(float g, float u) {
  const float s = __fdividef(g, 1.f + expf(-g)), v = s * u;
  // a zero gate or up, as a padded batch has whole rows of (0 * Inf is NaN and goes on);
  // its sign is that of the factors, as s may itself have been flushed to a zero of any sign
  if (v == 0.f && (g == 0.f || u == 0.f)) return ((__float_as_uint(g) ^ __float_as_uint(u)) >> 31) << 15;
  if (fabsf(s) > 1e-30f && fabsf(v) > 1e-30f && fabsf(v) < 1e38f && g < 700.f) return swiglu_bf16_border(g, u);
  return swiglu_bf16_ends(g, u);
}
__device__ __forceinline__ uint32_t swiglu_bf16(float g, float u) {
  uint32_t bits;
  return swiglu_bf16_fast(g, u, bits) ? bits : swiglu_bf16_slow(g, u);
}
// N values, two to a word: the fp32 steps without a branch between them, so
// that their latencies overlap, then the few that need more.  (A branch per
// value left the 4096-token int8 layer's epilogue longer than its MMAs.)
template <int N>
__device__ __forceinline__ void swiglu_bf16_pack(const float (&g)[N], const float (&u)[N], uint32_t* words) {
  uint32_t slow = 0;
  uint32_t bits[N];
#pragma unroll
  for (int i = 0; i < N; ++i) slow |= swiglu_bf16_fast(g[i], u[i], bits[i]) ? 0u : 1u << i;
  if (__any_sync(0xffffffffu, slow != 0)) {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if ((slow >> i) & 1u) bits[i] = swiglu_bf16_slow(g[i], u[i]);
  }
#pragma unroll
  for (int i = 0; i < N; i += 2) words[i / 2] = bits[i] | (bits[i + 1] << 16);
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
