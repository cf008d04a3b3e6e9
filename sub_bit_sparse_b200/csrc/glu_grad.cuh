// The gradient at the gate and up sums of the gated block.
#pragma once

#include "dense_math.cuh"

namespace stq1 {

// dY = [dG | dU] in bf16 from dact and the kept gate/up rows, eight columns per
// thread.  Bound by HBM: 4096 tokens by 4096 rows read 50 MB and write 34, 15.2 us
// (5.5 TB/s).  A kernel of its own because both products read all of dY.
//
// dY is rounded to bf16 because a tensor-core product takes both operands in one
// 16-bit type: two bf16 terms for it would double the products' MMAs.  With it the
// gradients are off by 2.4e-3 of their size in the mean square (200 and 4096 tokens,
// against fp64), 1.7e-3 of it by their own rounding to bf16.
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
