// Entry points of the 8-bit integer and gated feed-forward operators.
// Included by stq1_device.cu after its launch helpers.
#pragma once

#include "dense_gemm.cuh"
#include "quant_i8.cuh"

namespace stq1 {
namespace {

constexpr long long kDenseMaxDim = 1LL << 30;
constexpr long long kI8MaxK = 131056;    // 128 * 128 * K stays below 2^31

bool dense_shape_ok(long long a, long long b, long long c) {
  return a > 0 && b > 0 && c > 0 && a <= kDenseMaxDim && b <= kDenseMaxDim && c <= kDenseMaxDim &&
         a <= (1LL << 40) / b && a <= (1LL << 40) / c && b <= (1LL << 40) / c;
}

template <int EPI>
int launch_dense(const DenseArgs& p, cudaStream_t s) {
  const long long gx = (p.M + kDnTile - 1) / kDnTile;
  const long long gy = std::min<long long>((p.N + kDnTile - 1) / kDnTile, 65535);
  return launch_pdl_cluster(dense_gemm_kernel<EPI>, dim3(static_cast<unsigned>(gx), static_cast<unsigned>(gy)), 256, 0,
                            s, 1u, p);
}

int launch_quant_i8(const void* src, int type, long long R, long long K, int8_t* q, float* scales, cudaStream_t s) {
  if (type == STQ1_TYPE_F32)
    return launch_pdl(quant_i8_kernel<true>, static_cast<unsigned>(R), kQi8Threads, 0, s, src, K, q, scales);
  return launch_pdl(quant_i8_kernel<false>, static_cast<unsigned>(R), kQi8Threads, 0, s, src, K, q, scales);
}

DenseArgs i8_args(const int8_t* xq, const float* sx, const int8_t* wq, const float* sw, void* out, long long T,
                  long long N, long long K) {
  DenseArgs p{};
  p.a = xq;
  p.b = wq;
  p.sam = p.sbn = K;
  p.sak = p.sbk = 1;
  p.M = T;
  p.N = N;
  p.K = K;
  p.sx = sx;
  p.sw = sw;
  p.out = out;
  return p;
}

struct I8FfnPlan {
  size_t xq_off, sx_off, act_off, aq_off, sa_off, total;
};
I8FfnPlan plan_i8_ffn(long long T, long long N, long long H) {
  I8FfnPlan f{};
  size_t off = 0;
  auto take = [&](size_t bytes) { const size_t o = off; off += (bytes + 15) & ~static_cast<size_t>(15); return o; };
  f.xq_off = take(static_cast<size_t>(T) * H);
  f.sx_off = take(static_cast<size_t>(T) * 4);
  f.act_off = take(static_cast<size_t>(T) * N);          // bf16 [T, N/2]
  f.aq_off = take(static_cast<size_t>(T) * (N / 2));
  f.sa_off = take(static_cast<size_t>(T) * 4);
  f.total = off;
  return f;
}
bool i8_ffn_shape_ok(long long T, long long N, long long H) {
  return dense_shape_ok(T, N, H) && N % 32 == 0 && H % 16 == 0 && H <= kI8MaxK && N / 2 <= kI8MaxK;
}
bool glu_shape_ok(long long T, long long N, long long K) {
  return dense_shape_ok(T, N, K) && N % 16 == 0 && K % 8 == 0;
}

}  // namespace
}  // namespace stq1

extern "C" int stq1_quantize_i8(const void* src, int type, int64_t R, int64_t K, int8_t* q, float* scales,
                                void* stream) {
  NvtxRange nvtx_range("stq1_quantize_i8");
  if (!src || !q || !scales) return STQ1_ERR_NULL;
  if (type != STQ1_TYPE_F32 && type != STQ1_TYPE_BF16) return STQ1_ERR_ARG;
  if (!dense_shape_ok(R, K, 1) || K % 16) return STQ1_ERR_SHAPE;
  if (!aligned16(src) || !aligned16(q) || (reinterpret_cast<uintptr_t>(scales) & 3)) return STQ1_ERR_ALIGN;
  return launch_quant_i8(src, type, R, K, q, scales, static_cast<cudaStream_t>(stream));
}

extern "C" int stq1_i8_matmul(const int8_t* xq, const float* x_scales, const int8_t* wq, const float* w_scales, void* y,
                              int type, int64_t T, int64_t N, int64_t K, void* stream) {
  NvtxRange nvtx_range("stq1_i8_matmul");
  if (!xq || !x_scales || !wq || !w_scales || !y) return STQ1_ERR_NULL;
  if (type != STQ1_TYPE_F32 && type != STQ1_TYPE_BF16) return STQ1_ERR_ARG;
  if (!dense_shape_ok(T, N, K) || K % 16 || K > kI8MaxK) return STQ1_ERR_SHAPE;
  if (!aligned16(xq) || !aligned16(wq) || !aligned16(y) || (reinterpret_cast<uintptr_t>(x_scales) & 3) ||
      (reinterpret_cast<uintptr_t>(w_scales) & 3))
    return STQ1_ERR_ALIGN;
  const DenseArgs p = i8_args(xq, x_scales, wq, w_scales, y, T, N, K);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return type == STQ1_TYPE_F32 ? launch_dense<kEpiI8F32>(p, s) : launch_dense<kEpiI8Bf16>(p, s);
}

extern "C" int stq1_glu(const uint16_t* x, const uint16_t* W, uint16_t* act, uint16_t* y, int64_t T, int64_t N,
                        int64_t K, void* stream) {
  NvtxRange nvtx_range("stq1_glu");
  if (!x || !W || !act) return STQ1_ERR_NULL;
  if (!glu_shape_ok(T, N, K)) return STQ1_ERR_SHAPE;
  if (!aligned16(x) || !aligned16(W) || !aligned16(act) || !aligned16(y)) return STQ1_ERR_ALIGN;
  DenseArgs p{};
  p.a = x;
  p.b = W;
  p.sam = p.sbn = K;
  p.sak = p.sbk = 1;
  p.M = T;
  p.N = N / 2;
  p.K = K;
  p.out = act;
  p.y = y;
  return launch_dense<kEpiGlu>(p, static_cast<cudaStream_t>(stream));
}

extern "C" size_t stq1_glu_backward_workspace(int64_t T, int64_t N, int64_t K) {
  return glu_shape_ok(T, N, K) ? static_cast<size_t>(T) * N * 2 : 0;
}

extern "C" int stq1_glu_backward(const uint16_t* dact, const uint16_t* y, const uint16_t* x, const uint16_t* W,
                                 uint16_t* dx, uint16_t* dW, int64_t T, int64_t N, int64_t K, void* ws,
                                 size_t ws_bytes, void* stream) {
  NvtxRange nvtx_range("stq1_glu_backward");
  if (!dact || !y || (!dx && !dW) || (dx && !W) || (dW && !x)) return STQ1_ERR_NULL;
  if (!glu_shape_ok(T, N, K)) return STQ1_ERR_SHAPE;
  if (!ws || ws_bytes < stq1_glu_backward_workspace(T, N, K)) return STQ1_ERR_WORKSPACE;
  if (!aligned16(dact) || !aligned16(y) || !aligned16(x) || !aligned16(W) || !aligned16(dx) || !aligned16(dW) ||
      !aligned16(ws))
    return STQ1_ERR_ALIGN;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  uint16_t* dy = static_cast<uint16_t*>(ws);
  const long long grid = std::min<long long>((T * (N / 16) + 255) / 256, 148LL * 16);
  int rc = launch_pdl(glu_dy_kernel, static_cast<unsigned>(grid), 256, 0, s, dact, y, dy, static_cast<long long>(T),
                      static_cast<long long>(N / 2));
  if (rc != STQ1_OK) return rc;
  DenseArgs p{};
  p.a = dy;
  if (dx) {                              // dX[t, k] = sum_n dY[t, n] W[n, k]
    p.b = W;
    p.sam = N;
    p.sak = 1;
    p.sbn = 1;
    p.sbk = K;
    p.M = T;
    p.N = K;
    p.K = N;
    p.out = dx;
    rc = launch_dense<kEpiBf16>(p, s);
    if (rc != STQ1_OK) return rc;
  }
  if (dW) {                              // dW[n, k] = sum_t dY[t, n] x[t, k]
    p.b = x;
    p.sam = 1;
    p.sak = N;
    p.sbn = 1;
    p.sbk = K;
    p.M = N;
    p.N = K;
    p.K = T;
    p.out = dW;
    rc = launch_dense<kEpiBf16>(p, s);
  }
  return rc;
}

extern "C" size_t stq1_i8_ffn_workspace(int64_t T, int64_t N, int64_t H) {
  return i8_ffn_shape_ok(T, N, H) ? plan_i8_ffn(T, N, H).total : 0;
}

extern "C" int stq1_i8_ffn(const uint16_t* x, const int8_t* gateup_q, const float* gateup_scales, const int8_t* down_q,
                           const float* down_scales, float* out, int64_t T, int64_t N, int64_t H, void* ws,
                           size_t ws_bytes, void* stream) {
  NvtxRange nvtx_range("stq1_i8_ffn");
  if (!x || !gateup_q || !gateup_scales || !down_q || !down_scales || !out) return STQ1_ERR_NULL;
  if (!i8_ffn_shape_ok(T, N, H)) return STQ1_ERR_SHAPE;
  const I8FfnPlan f = plan_i8_ffn(T, N, H);
  if (!ws || ws_bytes < f.total) return STQ1_ERR_WORKSPACE;
  if (!aligned16(x) || !aligned16(gateup_q) || !aligned16(down_q) || !aligned16(out) || !aligned16(ws) ||
      (reinterpret_cast<uintptr_t>(gateup_scales) & 3) || (reinterpret_cast<uintptr_t>(down_scales) & 3))
    return STQ1_ERR_ALIGN;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  uint8_t* wsb = static_cast<uint8_t*>(ws);
  int8_t* xq = reinterpret_cast<int8_t*>(wsb + f.xq_off);
  float* sx = reinterpret_cast<float*>(wsb + f.sx_off);
  uint16_t* act = reinterpret_cast<uint16_t*>(wsb + f.act_off);
  int8_t* aq = reinterpret_cast<int8_t*>(wsb + f.aq_off);
  float* sa = reinterpret_cast<float*>(wsb + f.sa_off);
  int rc = launch_quant_i8(x, STQ1_TYPE_BF16, T, H, xq, sx, s);
  if (rc != STQ1_OK) return rc;
  rc = launch_dense<kEpiI8Glu>(i8_args(xq, sx, gateup_q, gateup_scales, act, T, N / 2, H), s);
  if (rc != STQ1_OK) return rc;
  rc = launch_quant_i8(act, STQ1_TYPE_BF16, T, N / 2, aq, sa, s);
  if (rc != STQ1_OK) return rc;
  return launch_dense<kEpiI8F32>(i8_args(aq, sa, down_q, down_scales, out, T, H, N / 2), s);
}
