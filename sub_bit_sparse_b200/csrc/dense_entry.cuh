// Entry points of the 8-bit integer and gated feed-forward operators.
// Included by stq1_device.cu after its launch helpers.
#pragma once

#include "dense_few.cuh"
#include "dense_tile.cuh"
#include "glu_grad.cuh"
#include "quant_i8.cuh"

namespace stq1 {
namespace {

constexpr long long kDenseMaxDim = 1LL << 30;
constexpr long long kI8MaxK = 131056;    // 128 * 128 * K stays below 2^31

bool dense_shape_ok(long long a, long long b, long long c) {
  return a > 0 && b > 0 && c > 0 && a <= kDenseMaxDim && b <= kDenseMaxDim && c <= kDenseMaxDim &&
         a <= (1LL << 40) / b && a <= (1LL << 40) / c && b <= (1LL << 40) / c;
}

// 2-D map over a row-major matrix [rows, cols] whose boxes are 128 bytes of a
// row by box_rows rows, in the 128-byte swizzle or plain; what lies outside reads as zero.
bool make_operand_map(CUtensorMap* map, const void* base, bool i8, long long rows, long long cols, int box_rows,
                      bool swizzle = true) {
  auto fn = encode_fn();
  if (!fn) return false;
  const int es = i8 ? 1 : 2;
  cuuint64_t gdim[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  cuuint64_t gstride[1] = {static_cast<cuuint64_t>(cols) * es};
  cuuint32_t box[2] = {static_cast<cuuint32_t>(kDnStepBytes / es), static_cast<cuuint32_t>(box_rows)};
  cuuint32_t es1[2] = {1, 1};
  return fn(map, i8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), gdim,
            gstride, box, es1, CU_TENSOR_MAP_INTERLEAVE_NONE,
            swizzle ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// 2-D map over results [rows, cols] (row stride ld elements) for copies of
// blocks of 32 rows by `width` bytes; a map that cannot be (a row's bytes are
// no multiple of 16) is left as it is, and the kernel does not use it.
bool make_result_map(CUtensorMap* map, void* base, bool f32, long long rows, long long cols, long long ld, int width) {
  auto fn = encode_fn();
  if (!fn) return false;
  const int es = f32 ? 4 : 2;
  if (!base || cols * es % 16) return true;
  cuuint64_t gdim[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  cuuint64_t gstride[1] = {static_cast<cuuint64_t>(ld) * es};
  cuuint32_t box[2] = {static_cast<cuuint32_t>(width / es), 32};
  cuuint32_t es1[2] = {1, 1};
  return fn(map, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, base, gdim, gstride, box,
            es1, CU_TENSOR_MAP_INTERLEAVE_NONE, width == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
            CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

std::atomic<bool> g_dense_configured[kMaxDevices];
constexpr int kFewAllSmem = 232448;        // of one CTA on an SM
constexpr int kFewHalfSmem = 233472 / 2 - 1024;   // two CTAs of so much fit (an SM has 228 KB and keeps 1 KB per CTA)
template <int EPI, bool MADE, int MT, int NT>
bool few_config_one() {
  return cudaFuncSetAttribute(dense_few_kernel<EPI, MADE, MT, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              kFewAllSmem) == cudaSuccess;
}
template <int EPI, bool MADE>
bool few_config() {
  return few_config_one<EPI, MADE, 2, 1>() && few_config_one<EPI, MADE, 2, 2>() && few_config_one<EPI, MADE, 4, 1>() &&
         few_config_one<EPI, MADE, 4, 2>();
}
std::atomic<int> g_max_clusters[kMaxDevices][3];   // clusters of 2, 4, 8 CTAs of the split kernel that run at once
template <int EPI, bool AMN, bool BMN, bool DUAL, int S>
bool split_config() {
  return cudaFuncSetAttribute(dense_split_kernel<EPI, AMN, BMN, DUAL, S>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              kSplitSmemBytes) == cudaSuccess;
}
template <int EPI, bool AMN, bool BMN, bool DUAL>
bool tile_config() {
  return cudaFuncSetAttribute(dense_pair_kernel<EPI, AMN, BMN, DUAL>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              kPairSmemBytes) == cudaSuccess &&
         split_config<EPI, AMN, BMN, DUAL, 1>() && split_config<EPI, AMN, BMN, DUAL, 2>() &&
         split_config<EPI, AMN, BMN, DUAL, 4>() && split_config<EPI, AMN, BMN, DUAL, 8>();
}
// How many clusters of S CTAs, one CTA per SM, the device runs at once: clusters
// stay inside a GPC, so this is less than SMs / S.
template <int S>
int query_clusters() {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(1, S);
  cfg.blockDim = dim3(kSplitThreads);
  cfg.dynamicSmemBytes = kSplitSmemBytes;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 1;
  attr[0].val.clusterDim.y = S;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, dense_split_kernel<kEpiI8F32, false, false, false, S>, &cfg) != cudaSuccess) {
    cudaGetLastError();
    n = 0;
  }
  return n;
}
int ensure_dense_configured() {
  const int dev = current_device();
  if (dev < 0) return STQ1_ERR_CUDA;
  if (g_dense_configured[dev].load(std::memory_order_acquire)) return STQ1_OK;
  std::lock_guard<std::mutex> lock(g_config_mutex);
  if (g_dense_configured[dev].load(std::memory_order_relaxed)) return STQ1_OK;
  if (!(tile_config<kEpiI8F32, false, false, false>() && tile_config<kEpiI8Bf16, false, false, false>() &&
        tile_config<kEpiI8Glu, false, false, false>() && tile_config<kEpiGlu, false, false, false>() &&
        tile_config<kEpiBf16, false, true, false>() && tile_config<kEpiBf16, true, true, false>() &&
        tile_config<kEpiBf16, false, true, true>() &&
        few_config<kEpiI8F32, false>() && few_config<kEpiI8F32, true>() && few_config<kEpiI8Bf16, false>() &&
        few_config<kEpiI8Glu, false>() && few_config<kEpiGlu, false>())) {
    cudaGetLastError();
    return STQ1_ERR_CUDA;
  }
  g_max_clusters[dev][0].store(query_clusters<2>(), std::memory_order_relaxed);
  g_max_clusters[dev][1].store(query_clusters<4>(), std::memory_order_relaxed);
  g_max_clusters[dev][2].store(query_clusters<8>(), std::memory_order_relaxed);
  g_dense_configured[dev].store(true, std::memory_order_release);
  return STQ1_OK;
}

// A product for the tile kernels: operand a [M rows] and b, each K-major
// ([rows, K]) or MN-major ([K, rows]).
struct DenseProduct {
  const void *a, *b;
  long long M, N, K;                 // N: outputs; the gated forms have 2N rows in b
  const float *sx, *sw;
  void* out;
  uint16_t* y;
  int missing;                       // bytes of A per step that no copy brings (the self-test; else 0)
};

// One product on the tile kernels, or two (DUAL: d1's A is MN-major) as one launch.
template <bool I8, bool GLU, bool AMN, bool BMN>
bool operand_maps(const DenseProduct& d, int box_a, CUtensorMap* ma, CUtensorMap* mb) {
  const long long rows_b = GLU ? 2 * d.N : d.N;
  return make_operand_map(ma, d.a, I8, AMN ? d.K : d.M, AMN ? d.M : d.K, box_a) &&
         make_operand_map(mb, d.b, I8, BMN ? d.K : rows_b, BMN ? rows_b : d.K, 64);
}
int k_steps(long long K, bool i8) { return static_cast<int>((K * (i8 ? 1 : 2) + kDnStepBytes - 1) / kDnStepBytes); }
template <bool I8>
DenseArgs tile_args(const DenseProduct& d, long long tiles_m, long long tiles_n, int a_rows) {
  DenseArgs p{};
  p.M = d.M;
  p.N = d.N;
  p.n_k = k_steps(d.K, I8);
  p.a_bytes = a_rows * kDnStepBytes + d.missing;
  p.tiles_m = static_cast<int>(tiles_m);
  p.tiles_n = static_cast<int>(tiles_n);
  p.sx = d.sx;
  p.sw = d.sw;
  p.out = d.out;
  p.y = d.y;
  return p;
}
// 128 x 128 tiles of a product (for the gated forms of 64 outputs)
template <bool GLU>
long long single_tiles(const DenseProduct& d) {
  return (d.M + 127) / 128 * (((GLU ? 2 * d.N : d.N) + 127) / 128);
}

// Maps of the results: of d0, and of d1 (DUAL) or of the two halves of y.
template <int EPI, bool DUAL>
bool result_maps(const DenseProduct& d0, const DenseProduct& d1, CUtensorMap* o0, CUtensorMap* o1, CUtensorMap* o2) {
  constexpr int kWidth = epi_glu(EPI) ? 64 : 128;
  if (!make_result_map(o0, d0.out, EPI == kEpiI8F32, d0.M, d0.N, d0.N, kWidth)) return false;
  if (DUAL) return make_result_map(o1, d1.out, false, d1.M, d1.N, d1.N, kWidth);
  if (EPI != kEpiGlu || !d0.y) return true;
  return make_result_map(o1, d0.y, false, d0.M, d0.N, 2 * d0.N, kWidth) &&
         make_result_map(o2, d0.y + d0.N, false, d0.M, d0.N, 2 * d0.N, kWidth);
}

template <int EPI, bool AMN, bool BMN, bool DUAL>
int launch_pairs(const DenseProduct& d0, const DenseProduct& d1, cudaStream_t s) {
  constexpr bool I8 = epi_i8(EPI), GLU = epi_glu(EPI);
  CUtensorMap a0, b0, a1, b1;
  if (!operand_maps<I8, GLU, AMN, BMN>(d0, 64, &a0, &b0)) return STQ1_ERR_CUDA;
  if (DUAL ? !operand_maps<I8, GLU, true, BMN>(d1, 64, &a1, &b1) : (a1 = a0, b1 = b0, false)) return STQ1_ERR_CUDA;
  const DenseProduct* d[2] = {&d0, &d1};
  long long tiles[2] = {0, 0};
  PairArgs args{};
  for (int i = 0; i < (DUAL ? 2 : 1); ++i) {
    const long long tm = (d[i]->M + 255) / 256, tn = ((GLU ? 2 * d[i]->N : d[i]->N) + 255) / 256;
    tiles[i] = tm * tn;
    if (tiles[i] >= (1LL << 29)) return STQ1_ERR_SHAPE;
    args.p[i] = tile_args<I8>(*d[i], tm, tn, kDnRows);
  }
  CUtensorMap o0{}, o1{}, o2{};
  if (!result_maps<EPI, DUAL>(d0, d1, &o0, &o1, &o2)) return STQ1_ERR_CUDA;
  const int pairs = sm_count() / 2;
  int rest_tiles = static_cast<int>(tiles[0]);       // of the list's last part
  if (DUAL) {
    args.long_prob = args.p[0].n_k >= args.p[1].n_k ? 0 : 1;
    const int other = 1 - args.long_prob;
    args.long_tiles = static_cast<int>(tiles[args.long_prob]);
    args.late = args.long_tiles % pairs;
    rest_tiles = static_cast<int>(tiles[other]);
    const int short_of = pairs - args.late;          // pairs with one long tile fewer (all, if the tiles came out even)
    // (a tile weighs at least its epilogue, about 12 steps: 300 tokens by [4096,
    // 7168], whose short tiles have 5, take 49 us so and 60 by the steps alone)
    auto weight = [&](int i) { return std::max(args.p[i].n_k, 12); };
    args.lead = args.late ? std::min(weight(args.long_prob) / weight(other), rest_tiles / short_of) : 0;
    rest_tiles -= args.lead * short_of;
  }
  // a last round that would leave more than half of the pairs idle goes by half
  // tiles: 1% at 4096 tokens by [4096, 7168] (81.9 us against 82.9)
  const int last = rest_tiles % pairs, done = (DUAL ? args.lead * (pairs - args.late) : 0) + rest_tiles - last;
  args.full = 2 * last <= pairs ? done : done + last;
  args.units = args.full + (2 * last <= pairs ? 2 * last : 0);
  // one product: no more pairs than units.  Two always run on all pairs: the list is laid out for them.
  const int grid = DUAL ? pairs : std::min(args.units, pairs);
  return launch_pdl(dense_pair_kernel<EPI, AMN, BMN, DUAL>, 2u * static_cast<unsigned>(grid), kPairThreads,
                    kPairSmemBytes, s, a0, b0, a1, b1, o0, o1, o2, args);
}

// Pieces of K for so many tiles of n_k steps, `least` steps each at least: as
// many as run at once.  (Clusters of eight for 17 tiles, of which the GPCs hold 16
// at a time: 9.3 us for [2053, 2048] weights and 77 tokens; clusters of four: 5.6.)
int split_pieces(long long tiles, int n_k, int least) {
  const int dev = current_device();
  int S = 1;
  for (int i = 1; i <= 3; ++i)
    if (dev >= 0 && tiles <= g_max_clusters[dev][i - 1].load(std::memory_order_relaxed) && (least << i) <= n_k) S = 1 << i;
  return S;
}
// Joining the pieces costs about four steps whatever their number, less where
// there are few rows to join or where it spreads the activation's work: int8, 120
// tokens by [1024, K], whole / two / four / eight pieces: 4 steps 4.3, 5.0, 5.1,
// 5.1 us, 8 steps 5.3, 5.5, 5.4, 5.5, 10 steps 5.8, 5.8, 5.6, 5.5, 16 steps 7.1, 6.5,
// 5.8, 5.7; 64 tokens, 8 steps 4.9, 4.6, 4.4, 4.5; gated, 120 tokens, 8 steps 7.2
// whole and 6.4 in four.  So short products of many rows stay whole, and else a
// piece has two steps.
int least_steps(long long M, int n_k, bool glu) { return glu || M <= 64 || n_k >= 10 ? 2 : n_k; }

template <int EPI, bool AMN, bool BMN, bool DUAL>
int launch_split(const DenseProduct& d0, const DenseProduct& d1, int S, bool early, cudaStream_t s) {
  constexpr bool I8 = epi_i8(EPI), GLU = epi_glu(EPI);
  // a lone row of tiles copies no more rows of A than there are (the sums of the others are never stored)
  const int a_rows = !AMN && d0.M < kDnRows ? static_cast<int>((d0.M + 7) / 8 * 8) : kDnRows;
  CUtensorMap a0, b0, a1, b1;
  if (!operand_maps<I8, GLU, AMN, BMN>(d0, AMN ? 64 : a_rows, &a0, &b0)) return STQ1_ERR_CUDA;
  if (DUAL ? !operand_maps<I8, GLU, true, BMN>(d1, 64, &a1, &b1) : (a1 = a0, b1 = b0, false)) return STQ1_ERR_CUDA;
  const DenseProduct* d[2] = {&d0, &d1};
  long long tiles = 0;
  SplitArgs args{};
  args.early = early;
  for (int i = 0; i < (DUAL ? 2 : 1); ++i) {
    const long long tm = (d[i]->M + 127) / 128, tn = ((GLU ? 2 * d[i]->N : d[i]->N) + 127) / 128;
    if (i == 1) args.tiles0 = static_cast<int>(tiles);
    tiles += tm * tn;
    args.p[i] = tile_args<I8>(*d[i], tm, tn, i == 0 ? a_rows : kDnRows);
  }
  CUtensorMap o0{}, o1{}, o2{};
  if (S == 1 && !result_maps<EPI, DUAL>(d0, d1, &o0, &o1, &o2)) return STQ1_ERR_CUDA;
  auto launch = [&](auto kernel) {
    return launch_pdl_cluster(kernel, dim3(static_cast<unsigned>(tiles), static_cast<unsigned>(S)), kSplitThreads,
                              kSplitSmemBytes, s, static_cast<unsigned>(S), a0, b0, a1, b1, o0, o1, o2, args);
  };
  switch (S) {
    case 1: return launch(dense_split_kernel<EPI, AMN, BMN, DUAL, 1>);
    case 2: return launch(dense_split_kernel<EPI, AMN, BMN, DUAL, 2>);
    case 4: return launch(dense_split_kernel<EPI, AMN, BMN, DUAL, 4>);
    default: return launch(dense_split_kernel<EPI, AMN, BMN, DUAL, 8>);
  }
}

// More 128 x 128 tiles than SMs: pairs on 256 x 256 tiles; else one tile per
// CTA, K split.  At the border, int8 with [4096, 7168] weights: 512 tokens (128
// tiles) take 17.1 us split and 20.2 on pairs, 600 tokens (160 tiles, two rounds
// of single tiles) 23.8 us on pairs.
template <int EPI, bool AMN, bool BMN>
int launch_tiles(const DenseProduct& d, bool early, cudaStream_t s) {
  int rc = ensure_dense_configured();
  if (rc != STQ1_OK) return rc;
  if (single_tiles<epi_glu(EPI)>(d) > sm_count()) return launch_pairs<EPI, AMN, BMN, false>(d, d, s);
  return launch_split<EPI, AMN, BMN, false>(d, d, split_pieces(single_tiles<epi_glu(EPI)>(d), k_steps(d.K, epi_i8(EPI)),
                                                               least_steps(d.M, k_steps(d.K, epi_i8(EPI)), epi_glu(EPI))), early, s);
}

// How a product with few tokens is laid out: outputs per CTA so that every SM
// has one CTA's share (or several in even rounds), and as many steps in flight
// per warp as fit.
struct FewPlan {
  int rows, pad, n_k, n_slots;
  size_t smem;
};
// false: the tile kernels take it.  made: the kernel makes the tokens' codes.
// The rules, each with both sides measured:
// - a CTA whose weights are read quickly (up to 256 KB) has at most four steps in
//   flight per warp, more queue up before HBM (int8 [2048, 7168] at one token 5.9
//   us with six, 5.4 with four); with more bytes, gated [4096, 7168], they count
//   for more: 10.9 us with six, 11.4 with three.
// - one CTA per SM, but for the shortest: two hide a part of the next launch (int8
//   [4096, 7168] 5.7 -> 5.0 us), until two of the same launch come to share an SM
//   and others stand idle, which then stays so from call to call: 12 us.
// - more outputs than one round of CTAs, and single tiles that run at once: the
//   tiles (int8 [11008, 4096]: 12.7 us and 11.5 on tiles at one token, 14.4 and
//   11.8 at 16; [18944, 4096] 16.0 and 14.9, 19.9 and 15.3; the other way for
//   [11008, 2048], 5.7 and 6.5, and [11008, 8192], 18.5 and 19.5 at one token; gated
//   [14336, 4096] at 12 tokens 26.0 and 24.8), except gated up to 8 tokens
//   ([11008, 4096] 17.8 and 21.0 at one, 19.1 and 21.3 at 8).
// - more tiles than that: int8 above 8 tokens on tiles ([65536, 2048], 12 tokens:
//   40.1 and 36.3 us; 8 tokens: 34.6 and 36.2), the gated form here ([28672, 4096],
//   12 tokens: 47.9 and 64.1).
bool plan_few(FewPlan* f, long long T, long long N, long long kbytes, bool glu, bool made = false) {
  if (T > kFewMaxTokens) return false;
  const int sms = sm_count(), unit = glu ? 8 : 16;         // the gate rows end on a whole swizzle atom
  const long long round_rows = sms * (glu ? 32LL : 64LL), rounds = (N + round_rows - 1) / round_rows;
  f->rows = static_cast<int>((N + sms * rounds - 1) / (sms * rounds));
  f->pad = (f->rows + unit - 1) / unit * unit * (glu ? 2 : 1);
  f->n_k = static_cast<int>((kbytes + kDnStepBytes - 1) / kDnStepBytes);
  const int mt = f->pad > 32 ? 4 : 2, nt = T > 8 ? 2 : 1;
  const long long x = made ? few_pitch(f->n_k) * T : 0;
  const long long per_warp = (f->n_k + kFewWarps - 1) / kFewWarps;
  // one slot per warp, with its tokens
  const long long step = (static_cast<long long>(f->pad) * kDnStepBytes + few_x_bytes(static_cast<int>(T), made)) * kFewWarps;
  const long long bytes = f->rows * (glu ? 2 : 1) * kbytes;
  const long long slots = std::min<long long>(std::min<long long>((kFewAllSmem - 1024 - kFewHead - x) / step, per_warp),
                                              bytes <= 256 * 1024 ? 4 : kFewMaxSlots);
  if (slots < std::min<long long>(2, per_warp)) return false;
  if (rounds > 1) {
    const long long tiles = ((glu ? 2 * N : N) + 127) / 128;
    if (tiles <= sms ? !(glu && T <= 8) : !glu && T > 8) return false;
  }
  f->n_slots = static_cast<int>(slots);
  const long long sums = 512LL * kFewWarps * mt * nt;      // the warps' sums take the place of slots and tokens
  f->smem = static_cast<size_t>(1024 + kFewHead + std::max(slots * step + x, sums));
  if (bytes > 64 * 1024) f->smem = std::max(f->smem, static_cast<size_t>(kFewHalfSmem + 16));
  return true;
}

// early: the kernel before does not write the weights.  amax: see FewArgs.
template <int EPI, bool MADE>
int launch_few(const FewPlan& f, const DenseProduct& d, bool early, uint32_t* amax, cudaStream_t s) {
  constexpr bool I8 = epi_i8(EPI), GLU = epi_glu(EPI);
  int rc = ensure_dense_configured();
  if (rc != STQ1_OK) return rc;
  FewArgs p{};
  p.x = d.a;
  p.sx = d.sx;
  p.sw = d.sw;
  p.out = d.out;
  p.y = d.y;
  p.N = d.N;
  p.K = d.K;
  p.T = static_cast<int>(d.M);
  p.rows = f.rows;
  p.pad = f.pad;
  p.n_k = f.n_k;
  p.n_slots = f.n_slots;
  p.early = early;
  p.amax = amax;
  CUtensorMap mw, mx{};
  if (!make_operand_map(&mw, d.b, I8, GLU ? 2 * d.N : d.N, d.K, f.rows) ||
      (!MADE && !make_operand_map(&mx, d.a, I8, d.M, d.K, static_cast<int>(d.M), d.M > 1)))
    return STQ1_ERR_CUDA;
  const unsigned grid = static_cast<unsigned>((d.N + f.rows - 1) / f.rows);
  auto launch = [&](auto kernel) { return launch_pdl(kernel, grid, kFewThreads, f.smem, s, mw, mx, p); };
  if (f.pad > 32)
    return d.M > 8 ? launch(dense_few_kernel<EPI, MADE, 4, 2>) : launch(dense_few_kernel<EPI, MADE, 4, 1>);
  return d.M > 8 ? launch(dense_few_kernel<EPI, MADE, 2, 2>) : launch(dense_few_kernel<EPI, MADE, 2, 1>);
}

// A product of K-major operands: few tokens take the streaming kernel (int8,
// [4096, 7168]: 5.2-6.4 us at one token, 6.8-7.4 at 16; the split kernel 7.4 and 7.8).
template <int EPI>
int launch_product(const DenseProduct& d, bool early, cudaStream_t s) {
  FewPlan f;
  if (plan_few(&f, d.M, d.N, d.K * (epi_i8(EPI) ? 1 : 2), epi_glu(EPI)))
    return launch_few<EPI, false>(f, d, early, nullptr, s);
  return launch_tiles<EPI, false, false>(d, early, s);
}

// Threads per row by its length, so that enough rows are in flight; measured on
// 4096 bf16 rows, against the next larger choice: 256 values 2.2 us (2.9), 1024
// 2.8 (3.4), 2048 5.5 (9.7), 4096 8.8 (10.6), 7168 14.4 (15.6); with fp32 rows
// the last step turns round, 7168 values 22.4 us with 256 threads (23.3 with 128).
template <bool F32>
int launch_quant_rows(const void* src, long long R, long long K, int8_t* q, float* scales, uint32_t* clear,
                      cudaStream_t s) {
  const unsigned warps = static_cast<unsigned>((R + kQi8Warps - 1) / kQi8Warps), rows = static_cast<unsigned>(R);
  auto launch = [&](auto kernel, unsigned grid, int threads) {
    return launch_pdl(kernel, grid, static_cast<unsigned>(threads), 0, s, src, R, K, q, scales, clear);
  };
  if (K <= 1024) return launch(quant_i8_kernel<F32, 32, 4>, warps, 32 * kQi8Warps);
  if (K <= 2048) return launch(quant_i8_kernel<F32, 32, 8>, warps, 32 * kQi8Warps);
  if (K <= 4096) return launch(quant_i8_kernel<F32, 128, 4>, rows, 128);
  if constexpr (!F32)
    if (K <= 8192) return launch(quant_i8_kernel<F32, 128, 8>, rows, 128);
  return launch(quant_i8_kernel<F32, 256, 4>, rows, 256);
}
int launch_quant_i8(const void* src, int type, long long R, long long K, int8_t* q, float* scales, cudaStream_t s,
                    uint32_t* clear = nullptr) {
  return type == STQ1_TYPE_F32 ? launch_quant_rows<true>(src, R, K, q, scales, clear, s)
                               : launch_quant_rows<false>(src, R, K, q, scales, clear, s);
}

DenseProduct i8_product(const int8_t* xq, const float* sx, const int8_t* wq, const float* sw, void* out, long long T,
                        long long N, long long K) {
  return {xq, wq, T, N, K, sx, sw, out, nullptr, 0};
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
  const DenseProduct p = i8_product(xq, x_scales, wq, w_scales, y, T, N, K);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return type == STQ1_TYPE_F32 ? launch_product<kEpiI8F32>(p, false, s) : launch_product<kEpiI8Bf16>(p, false, s);
}

extern "C" int stq1_selftest_product(const int8_t* xq, const float* x_scales, const int8_t* wq, const float* w_scales,
                                     float* y, int64_t T, int64_t N, int64_t K, int arrive, void* stream) {
  NvtxRange nvtx_range("stq1_selftest_product");
  if (!xq || !x_scales || !wq || !w_scales || !y) return STQ1_ERR_NULL;
  if (arrive != 0 && arrive != 1) return STQ1_ERR_ARG;
  if (!dense_shape_ok(T, N, K) || K % 16 || K > kI8MaxK) return STQ1_ERR_SHAPE;
  if (!aligned16(xq) || !aligned16(wq) || !aligned16(y) || (reinterpret_cast<uintptr_t>(x_scales) & 3) ||
      (reinterpret_cast<uintptr_t>(w_scales) & 3))
    return STQ1_ERR_ALIGN;
  DenseProduct p = i8_product(xq, x_scales, wq, w_scales, y, T, N, K);
  p.missing = arrive ? 0 : 16;
  return launch_tiles<kEpiI8F32, false, false>(p, false, static_cast<cudaStream_t>(stream));
}

extern "C" int stq1_glu(const uint16_t* x, const uint16_t* W, uint16_t* act, uint16_t* y, int64_t T, int64_t N,
                        int64_t K, void* stream) {
  NvtxRange nvtx_range("stq1_glu");
  if (!x || !W || !act) return STQ1_ERR_NULL;
  if (!glu_shape_ok(T, N, K)) return STQ1_ERR_SHAPE;
  if (!aligned16(x) || !aligned16(W) || !aligned16(act) || !aligned16(y)) return STQ1_ERR_ALIGN;
  return launch_product<kEpiGlu>({x, W, T, N / 2, K, nullptr, nullptr, act, y}, false, static_cast<cudaStream_t>(stream));
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
  const DenseProduct px{dy, W, T, K, N, nullptr, nullptr, dx, nullptr};    // dX[t, k] = sum_n dY[t, n] W[n, k]
  const DenseProduct pw{dy, x, N, K, T, nullptr, nullptr, dW, nullptr};    // dW[n, k] = sum_t dY[t, n] x[t, k]
  rc = ensure_dense_configured();
  if (rc != STQ1_OK) return rc;
  // one launch for both where the same kernel suits both; a gradient has the
  // same bits whether the other is asked for or not, so few tiles are split
  // as for both in any case
  const long long tx = single_tiles<false>(px), tw = single_tiles<false>(pw);
  if (tx + tw <= sm_count()) {
    const int S = split_pieces(tx + tw, std::max(k_steps(N, false), k_steps(T, false)), 4);
    if (dx && dW) return launch_split<kEpiBf16, false, true, true>(px, pw, S, false, s);
    return dx ? launch_split<kEpiBf16, false, true, false>(px, px, S, false, s)
              : launch_split<kEpiBf16, true, true, false>(pw, pw, S, false, s);
  }
  if (dx && dW && tx > sm_count() && tw > sm_count()) return launch_pairs<kEpiBf16, false, true, true>(px, pw, s);
  if (dx) {
    rc = launch_tiles<kEpiBf16, false, true>(px, false, s);
    if (rc != STQ1_OK) return rc;
  }
  return dW ? launch_tiles<kEpiBf16, true, true>(pw, false, s) : rc;
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
  const DenseProduct up = i8_product(xq, sx, gateup_q, gateup_scales, act, T, N / 2, H);
  const DenseProduct down = i8_product(aq, sa, down_q, down_scales, out, T, H, N / 2);
  FewPlan fg, fd;
  if (plan_few(&fg, T, N / 2, H, true) && plan_few(&fd, T, H, N / 2, false, true)) {
    // few tokens: each kernel asks for its weights while the one before it
    // still runs; the activation's maxima are kept by the kernel that writes
    // it, so that its codes are made inside the second product
    uint32_t* amax = reinterpret_cast<uint32_t*>(sa);
    DenseProduct dn = down;
    dn.a = act;
    int rc = launch_quant_i8(x, STQ1_TYPE_BF16, T, H, xq, sx, s, amax);
    if (rc == STQ1_OK) rc = launch_few<kEpiI8Glu, false>(fg, up, true, amax, s);
    return rc != STQ1_OK ? rc : launch_few<kEpiI8F32, true>(fd, dn, true, amax, s);
  }
  int rc = launch_quant_i8(x, STQ1_TYPE_BF16, T, H, xq, sx, s);
  if (rc != STQ1_OK) return rc;
  rc = launch_product<kEpiI8Glu>(up, true, s);
  if (rc != STQ1_OK) return rc;
  rc = launch_quant_i8(act, STQ1_TYPE_BF16, T, N / 2, aq, sa, s);
  if (rc != STQ1_OK) return rc;
  return launch_product<kEpiI8F32>(down, true, s);
}
