// Signed 8-bit codes of matrix rows, one fp32 scale per row.
#pragma once

#include "dense_math.cuh"

namespace stq1 {

constexpr int kQi8Warps = 8;       // rows per CTA where a row is a warp's

// Eight consecutive values of a row as fp32 and the largest magnitude's bits.
template <bool F32>
struct Row8;
template <>
struct Row8<false> {
  uint4 v;
  __device__ __forceinline__ void load(const void* row, int i) { v = reinterpret_cast<const uint4*>(row)[i]; }
  __device__ __forceinline__ void zero() { v = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ uint32_t amax_bits() const {
    const uint32_t m = 0x7FFF7FFFu;
    const uint32_t a = __vmaxu2(__vmaxu2(v.x & m, v.y & m), __vmaxu2(v.z & m, v.w & m));
    return max(a & 0xFFFFu, a >> 16) << 16;
  }
  __device__ __forceinline__ uint2 codes(float inv) const {
    auto lo = [](uint32_t w) { return __uint_as_float(w << 16); };
    auto hi = [](uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); };
    return make_uint2(i8_pack4(lo(v.x), hi(v.x), lo(v.y), hi(v.y), inv),
                      i8_pack4(lo(v.z), hi(v.z), lo(v.w), hi(v.w), inv));
  }
};
template <>
struct Row8<true> {
  float4 a, b;
  __device__ __forceinline__ void load(const void* row, int i) {
    a = reinterpret_cast<const float4*>(row)[2 * i];
    b = reinterpret_cast<const float4*>(row)[2 * i + 1];
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ uint32_t amax_bits() const {
    auto m = [](float x) { return __float_as_uint(x) & 0x7FFFFFFFu; };
    return max(max(max(m(a.x), m(a.y)), max(m(a.z), m(a.w))), max(max(m(b.x), m(b.y)), max(m(b.z), m(b.w))));
  }
  __device__ __forceinline__ uint2 codes(float inv) const {
    return make_uint2(i8_pack4(a.x, a.y, a.z, a.w, inv), i8_pack4(b.x, b.y, b.z, b.w, inv));
  }
};

// TPR threads per row (a warp, or a CTA of that size): the row's largest
// magnitude, then its codes.  A thread's first kKeep vectors stay in registers
// between the two (rows of up to 8 * TPR * kKeep values are read once); longer
// rows read the rest again.  clear: one word per row to set to zero (for a
// later kernel's maxima), or NULL.
//
// Bound by HBM when the rows are many ([4096, 7168] fp32: 22.5 us, 6.5 TB/s,
// the copy rate), by latency when they are few ([16, 7168]: 1.7 us).
template <bool F32, int TPR, int kKeep>
__global__ void __launch_bounds__(TPR == 32 ? 32 * kQi8Warps : TPR)
quant_i8_kernel(const void* __restrict__ src, long long R, long long K, int8_t* __restrict__ q,
                float* __restrict__ scales, uint32_t* __restrict__ clear) {
  constexpr bool kWarp = TPR == 32;
  __shared__ uint32_t s_red[kWarp ? 1 : TPR / 32];
  const long long r = kWarp ? blockIdx.x * static_cast<long long>(kQi8Warps) + (threadIdx.x >> 5) : blockIdx.x;
  const int at = kWarp ? threadIdx.x & 31 : threadIdx.x;
  griddep_wait();
  griddep_launch_dependents();
  if (kWarp && r >= R) return;
  const char* row = static_cast<const char*>(src) + r * K * (F32 ? 4 : 2);
  const int nv = static_cast<int>(K / 8);
  Row8<F32> keep[kKeep];
  uint32_t m = 0u;
#pragma unroll
  for (int j = 0; j < kKeep; ++j) {
    const int i = at + j * TPR;
    if (i < nv) keep[j].load(row, i);
    else keep[j].zero();
  }
#pragma unroll
  for (int j = 0; j < kKeep; ++j) m = max(m, keep[j].amax_bits());
  for (int i = at + kKeep * TPR; i < nv; i += TPR) {
    Row8<F32> v;
    v.load(row, i);
    m = max(m, v.amax_bits());
  }
  m = __reduce_max_sync(0xffffffffu, m);
  if constexpr (!kWarp) {
    if ((threadIdx.x & 31) == 0) s_red[threadIdx.x >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < TPR / 32; ++i) m = max(m, s_red[i]);
  }
  const I8Scale sc = i8_scale(m);
  if (at == 0) {
    scales[r] = sc.scale;
    if (clear) clear[r] = 0u;
  }
  uint2* out = reinterpret_cast<uint2*>(q + r * K);
#pragma unroll
  for (int j = 0; j < kKeep; ++j) {
    const int i = at + j * TPR;
    if (i < nv) out[i] = keep[j].codes(sc.inv);
  }
  for (int i = at + kKeep * TPR; i < nv; i += TPR) {
    Row8<F32> v;
    v.load(row, i);
    out[i] = v.codes(sc.inv);
  }
}

}  // namespace stq1
