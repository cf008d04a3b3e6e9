// Products of the 8-bit integer and bf16 gated layers with few tokens: the
// weights are read once, straight into the registers that mma.sync takes.
//
// A contraction may take its k in any order as long as both operands agree on
// it.  So a lane's share of an A fragment need not be the 4-byte pieces that
// mma.sync's layout spreads over a row: lane (g, t) loads 16 consecutive bytes
// of rows g and g + 8 at 16 t of a 64-byte piece of K and feeds them to two
// MMAs (words 0, 1 and words 2, 3), and the same 16 bytes of token g make the
// B fragments.  8-bit and bf16 operands have the same word layout.
//
// For the gated forms a fragment's rows 0-7 are gate rows and its rows 8-15
// the up rows of the same outputs: a lane then holds g and u of one output.
#pragma once

#include "dense_math.cuh"
#include "dense_tile.cuh"
#include "quant_i8.cuh"

namespace stq1 {

constexpr int kGvThreads = 256;
constexpr int kGvWarps = kGvThreads / 32;
constexpr int kGvMaxTokens = 32;

struct GemvArgs {
  const void* w;               // [N or 2N, K]
  const void* x;               // [T, K] codes or bf16
  const float *sx, *sw;
  void* out;
  uint16_t* y;
  long long N, K;              // outputs (for the gated forms half of w's rows); values per row
  int T;
};

__device__ __forceinline__ uint4 ldg_stream(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

__device__ __forceinline__ void gv_mma(int (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void gv_mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// QX: x is bf16 and its codes are made here (each CTA finds the tokens' scales
// itself: T * K values from L2 against a launch of its own).  NT: groups of 8
// tokens.  U: pieces of K whose loads are in flight per warp.
template <int EPI, bool QX, int NT, int U>
__global__ void __launch_bounds__(kGvThreads)
dense_gemv_kernel(const GemvArgs p) {
  constexpr bool I8 = epi_i8(EPI), GLU = epi_glu(EPI);
  static_assert(I8 || !QX, "codes are made for 8-bit weights");
  using Acc = std::conditional_t<I8, int, float>;
  constexpr int ES = I8 ? 1 : 2;
  __shared__ Acc s_red[kGvWarps][NT][32][4];
  __shared__ float s_scale[8 * NT], s_inv[8 * NT];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  griddep_wait();
  griddep_launch_dependents();

  const long long kbytes = p.K * ES;
  const int pieces = static_cast<int>((kbytes + 63) / 64);
  const long long row0 = GLU ? blockIdx.x * 8LL + g : blockIdx.x * 16LL + g;      // rows of fragment rows g and g + 8
  const long long row1 = GLU ? p.N + row0 : row0 + 8;
  const bool ok0 = GLU || row0 < p.N, ok1 = GLU || row1 < p.N;
  const char* w0 = static_cast<const char*>(p.w) + (ok0 ? row0 : 0) * kbytes + 16 * t;
  const char* w1 = static_cast<const char*>(p.w) + (ok1 ? row1 : 0) * kbytes + 16 * t;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  auto load_w = [&](int c, uint4& a, uint4& b) {
    const bool in = c < pieces && 64LL * c + 16 * t < kbytes;
    a = in && ok0 ? ldg_stream(w0 + 64LL * c) : zero;
    b = in && ok1 ? ldg_stream(w1 + 64LL * c) : zero;
  };
  uint4 a0[U], a1[U];
#pragma unroll
  for (int u = 0; u < U; ++u) load_w(warp + kGvWarps * u, a0[u], a1[u]);

  float inv[NT];
  if constexpr (QX) {
    // the tokens' largest magnitudes, a warp per token in turn
    for (int k = warp; k < p.T; k += kGvWarps) {
      const char* xr = static_cast<const char*>(p.x) + k * p.K * 2;
      uint32_t m = 0u;
      for (int i = lane; i < p.K / 8; i += 32) {
        Row8<false> v;
        v.load(xr, i);
        m = max(m, v.amax_bits());
      }
      m = __reduce_max_sync(0xffffffffu, m);
      if (lane == 0) {
        const I8Scale s = i8_scale(m);
        s_inv[k] = s.inv;
        s_scale[k] = s.scale;
      }
    }
    __syncthreads();
#pragma unroll
    for (int n = 0; n < NT; ++n) inv[n] = 8 * n + g < p.T ? s_inv[8 * n + g] : 0.f;
  }
  auto load_x = [&](int c, int n) -> uint4 {
    const int tok = 8 * n + g;
    if (tok >= p.T || c >= pieces || 64LL * c + 16 * t >= kbytes) return zero;
    if constexpr (QX) {
      const char* xp = static_cast<const char*>(p.x) + (tok * p.K + 64LL * c + 16 * t) * 2;
      Row8<false> lo, hi;
      lo.load(xp, 0);
      hi.load(xp, 1);
      const uint2 l = lo.codes(inv[n]), h = hi.codes(inv[n]);
      return make_uint4(l.x, l.y, h.x, h.y);
    } else {
      return __ldg(reinterpret_cast<const uint4*>(static_cast<const char*>(p.x) + tok * kbytes + 64LL * c + 16 * t));
    }
  };

  Acc acc[NT][4] = {};
  for (int c = warp; c < pieces; c += kGvWarps * U) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint4 f0 = a0[u], f1 = a1[u];
      load_w(c + kGvWarps * (U + u), a0[u], a1[u]);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const uint4 b = load_x(c + kGvWarps * u, n);
        gv_mma(acc[n], f0.x, f1.x, f0.y, f1.y, b.x, b.y);
        gv_mma(acc[n], f0.z, f1.z, f0.w, f1.w, b.z, b.w);
      }
    }
  }
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) s_red[warp][n][lane][i] = acc[n][i];
  __syncthreads();

  // sums over the warps, in their order; consecutive threads take consecutive outputs of one token
  constexpr int kOut = GLU ? 8 : 16;
  for (int e = threadIdx.x; e < kOut * p.T; e += kGvThreads) {
    const int r = e % kOut, tok = e / kOut;
    const int src = (r & 7) * 4 + ((tok & 7) >> 1);
    auto total = [&](int reg) {
      Acc v = s_red[0][tok >> 3][src][reg];
#pragma unroll
      for (int q = 1; q < kGvWarps; ++q) v += s_red[q][tok >> 3][src][reg];
      return v;
    };
    const long long n = blockIdx.x * static_cast<long long>(kOut) + r;
    if (n >= p.N) continue;
    float sx = 0.f;
    if constexpr (QX) sx = s_scale[tok];
    else if constexpr (I8) sx = p.sx[tok];
    auto value = [&](Acc v, long long row) -> float {
      if constexpr (I8) return i8_value(v, sx, p.sw[row]);
      else return v;
    };
    if constexpr (GLU) {
      const float gv = value(total(tok & 1), n), uv = value(total(2 + (tok & 1)), p.N + n);
      static_cast<uint16_t*>(p.out)[tok * p.N + n] = static_cast<uint16_t>(swiglu_bf16(gv, uv));
      if constexpr (EPI == kEpiGlu)
        if (p.y) {
          p.y[tok * 2 * p.N + n] = static_cast<uint16_t>(bf16_bits_rn(gv));
          p.y[tok * 2 * p.N + p.N + n] = static_cast<uint16_t>(bf16_bits_rn(uv));
        }
    } else {
      const float v = value(total(2 * (r >> 3) + (tok & 1)), n);
      if constexpr (EPI == kEpiI8F32) static_cast<float*>(p.out)[tok * p.N + n] = v;
      else static_cast<uint16_t*>(p.out)[tok * p.N + n] = static_cast<uint16_t>(bf16_bits_rn(v));
    }
  }
}

}  // namespace stq1
