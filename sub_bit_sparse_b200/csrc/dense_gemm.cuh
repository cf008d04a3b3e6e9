// Products of the 8-bit integer and bf16 gated layers.
#pragma once

#include "dense_math.cuh"

namespace stq1 {

// C[m, n] = sum_k A(m, k) B(n, k), with A(m, k) at a + m * sam + k * sak and
// B likewise; what becomes of a sum is the epilogue's.
enum DenseEpi {
  kEpiI8F32,      // int8: fp32 y[m, n]
  kEpiI8Bf16,     // int8: bf16 y[m, n]
  kEpiI8Glu,      // int8: bf16 act[m, n] of gate channel n and up channel N + n
  kEpiGlu,        // bf16: the same, and optionally bf16 y [m, 2N]
  kEpiBf16,       // bf16: bf16 y[m, n]
};

struct DenseArgs {
  const void *a, *b;
  long long sam, sak, sbn, sbk;
  long long M, N, K;                 // N: outputs (for the gated forms half of B's rows)
  const float *sx, *sw;              // int8: scales of A's rows and of B's rows
  void* out;                         // [M, N]
  uint16_t* y;                       // kEpiGlu: [M, 2N] or NULL
};

constexpr int kDnTile = 64, kDnK = 16;

template <int EPI>
__global__ void __launch_bounds__(256)
dense_gemm_kernel(const DenseArgs p) {
  constexpr bool I8 = EPI == kEpiI8F32 || EPI == kEpiI8Bf16 || EPI == kEpiI8Glu;
  constexpr bool GLU = EPI == kEpiI8Glu || EPI == kEpiGlu;
  constexpr int NB = GLU ? 2 : 1;
  using Acc = std::conditional_t<I8, int, float>;
  __shared__ Acc sa[kDnK][kDnTile + 1], sb[NB][kDnK][kDnTile + 1];
  griddep_wait();
  griddep_launch_dependents();
  const long long m0 = static_cast<long long>(blockIdx.x) * kDnTile;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  auto at = [](const void* p, long long i) -> Acc {
    if constexpr (I8) return static_cast<const int8_t*>(p)[i];
    else return bf16_bits_to_f32(static_cast<const uint16_t*>(p)[i]);
  };
  for (long long n0 = static_cast<long long>(blockIdx.y) * kDnTile; n0 < p.N;
       n0 += static_cast<long long>(gridDim.y) * kDnTile) {
    Acc acc[NB][4][4] = {};
    for (long long k0 = 0; k0 < p.K; k0 += kDnK) {
      for (int i = threadIdx.x; i < kDnTile * kDnK; i += 256) {
        const int r = i / kDnK, k = i % kDnK;
        const bool kin = k0 + k < p.K;
        sa[k][r] = kin && m0 + r < p.M ? at(p.a, (m0 + r) * p.sam + (k0 + k) * p.sak) : Acc(0);
#pragma unroll
        for (int b = 0; b < NB; ++b)
          sb[b][k][r] = kin && n0 + r < p.N ? at(p.b, (b * p.N + n0 + r) * p.sbn + (k0 + k) * p.sbk) : Acc(0);
      }
      __syncthreads();
#pragma unroll
      for (int k = 0; k < kDnK; ++k)
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[b][i][j] += sa[k][ty + 16 * i] * sb[b][k][tx + 16 * j];
      __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const long long m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
        if (m >= p.M || n >= p.N) continue;
        float v[NB];
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          if constexpr (I8) v[b] = i8_value(acc[b][i][j], p.sx[m], p.sw[b * p.N + n]);
          else v[b] = acc[b][i][j];
        }
        if constexpr (EPI == kEpiI8F32) static_cast<float*>(p.out)[m * p.N + n] = v[0];
        else if constexpr (GLU) static_cast<uint16_t*>(p.out)[m * p.N + n] = static_cast<uint16_t>(swiglu_bf16(v[0], v[1]));
        else static_cast<uint16_t*>(p.out)[m * p.N + n] = static_cast<uint16_t>(bf16_bits_rn(v[0]));
        if constexpr (EPI == kEpiGlu)
          if (p.y) {
            p.y[m * 2 * p.N + n] = static_cast<uint16_t>(bf16_bits_rn(v[0]));
            p.y[m * 2 * p.N + p.N + n] = static_cast<uint16_t>(bf16_bits_rn(v[1]));
          }
      }
  }
}

// dY = [dG | dU] in bf16 from dact and the kept gate/up rows.
__global__ void __launch_bounds__(256)
glu_dy_kernel(const uint16_t* __restrict__ dact, const uint16_t* __restrict__ y, uint16_t* __restrict__ dy, long long T,
              long long half) {
  griddep_wait();
  griddep_launch_dependents();
  const long long per = half / 8, total = T * per;
  for (long long i = blockIdx.x * 256LL + threadIdx.x; i < total; i += 256LL * gridDim.x) {
    const long long t = i / per, j = (i - t * per) * 8;
    const uint4 dv = *reinterpret_cast<const uint4*>(dact + t * half + j);
    const uint4 gv = *reinterpret_cast<const uint4*>(y + t * 2 * half + j);
    const uint4 uv = *reinterpret_cast<const uint4*>(y + t * 2 * half + half + j);
    const uint32_t d[4] = {dv.x, dv.y, dv.z, dv.w}, g[4] = {gv.x, gv.y, gv.z, gv.w}, u[4] = {uv.x, uv.y, uv.z, uv.w};
    uint32_t og[4], ou[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      float g0, u0, g1, u1;
      glu_grads(__uint_as_float(d[q] << 16), __uint_as_float(g[q] << 16), __uint_as_float(u[q] << 16), g0, u0);
      glu_grads(__uint_as_float(d[q] & 0xFFFF0000u), __uint_as_float(g[q] & 0xFFFF0000u),
                __uint_as_float(u[q] & 0xFFFF0000u), g1, u1);
      og[q] = bf16_bits_rn(g0) | (bf16_bits_rn(g1) << 16);
      ou[q] = bf16_bits_rn(u0) | (bf16_bits_rn(u1) << 16);
    }
    *reinterpret_cast<uint4*>(dy + t * 2 * half + j) = make_uint4(og[0], og[1], og[2], og[3]);
    *reinterpret_cast<uint4*>(dy + t * 2 * half + half + j) = make_uint4(ou[0], ou[1], ou[2], ou[3]);
  }
}

}  // namespace stq1
