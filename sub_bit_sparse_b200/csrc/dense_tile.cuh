// Tensor-core products of the 8-bit integer and bf16 gated layers (sm_100a,
// tcgen05): C[m, n] = sum_k A(m, k) B(n, k), both operands from shared memory,
// fp32 (bf16 operands) or 32-bit integer (8-bit operands) sums in TMEM, and
// the layer's arithmetic on each finished sum before it is stored.
//
// Operands are K-major (rows of k, as x [T, K] and W [N, K] lie in the forward
// products) or MN-major (the contraction runs over the rows of the matrix, as
// in dX = dY W for W and in dW = dY^T x for both), so no transposed copy is
// ever made: the tensor copies bring 128-byte pieces of rows in both cases and
// only the descriptors of the MMAs differ.
#pragma once

#include "dense_math.cuh"
#include "tc_gemm.cuh"

namespace stq1 {

// What becomes of a finished sum.
enum DenseEpi {
  kEpiI8F32,      // int8: fp32 out[m, n]
  kEpiI8Bf16,     // int8: bf16 out[m, n]
  kEpiI8Glu,      // int8: bf16 act[m, n] of gate channel n and up channel N + n
  kEpiGlu,        // bf16: the same, and optionally the sums as bf16 y [m, 2N]
  kEpiBf16,       // bf16: bf16 out[m, n]
};
__host__ __device__ constexpr bool epi_i8(int e) { return e == kEpiI8F32 || e == kEpiI8Bf16 || e == kEpiI8Glu; }
__host__ __device__ constexpr bool epi_glu(int e) { return e == kEpiI8Glu || e == kEpiGlu; }

struct DenseArgs {
  long long M, N;                    // outputs; for the gated forms N is half of B's rows
  int n_k;                           // 128-byte steps of K
  int a_bytes;                       // bytes of A per step and CTA that a step waits for
  int tiles_m, tiles_n;
  const float *sx, *sw;              // int8: scales of A's rows and of B's rows
  void* out;                         // [M, N]
  uint16_t* y;                       // kEpiGlu: [M, 2N] or NULL
};

// What the pair kernel works through: one product, or two with the same
// epilogue as one list of tiles, the product with the longer K first.  Pair c of
// C takes of the `long_tiles` tiles c, c + C, ...; where that leaves the pairs
// from `late` on one tile short, those take `lead` rounds of the other product's
// tiles (as many as a long one weighs) before all pairs share out the rest.
// (Taken simply in turn, 1000 tokens by [4096, 7168] had pairs with 128 steps of
// K before the 16-step tiles began and others with 64: 91 us against 85; 700
// tokens 74 against 67.)
struct PairArgs {
  DenseArgs p[2];
  int long_prob, long_tiles;         // none with one product
  int late, lead;
  int full, units;                   // of the rest: tiles done whole, then the others as two halves of 128 columns
};

constexpr int kDnStepBytes = 128;    // bytes of K per step and row: one swizzle atom
constexpr int kDnRows = 128;         // rows of A and rows of B per CTA and step
constexpr int kDnOperandBytes = kDnRows * kDnStepBytes;
constexpr int kDnStageBytes = 2 * kDnOperandBytes;

// ---- PTX wrappers (pairs of CTAs) ----
template <int CG>
__device__ __forceinline__ void dn_tmem_alloc(uint32_t dst_smem, uint32_t cols) {
  if constexpr (CG == 2) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem), "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  } else {
    tmem_alloc(dst_smem, cols);
    tmem_relinquish();
  }
}
template <int CG>
__device__ __forceinline__ void dn_tmem_dealloc(uint32_t taddr, uint32_t cols) {
  if constexpr (CG == 2)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(cols) : "memory");
  else
    tmem_dealloc(taddr, cols);
}
// Arrives on the barrier at this offset in both CTAs of the pair once the
// MMAs issued so far are done.
__device__ __forceinline__ void dn_commit_pair(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
      "h"(static_cast<uint16_t>(3))
      : "memory");
}
__device__ __forceinline__ uint32_t dn_mapa(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void dn_arrive_remote(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
// As mbar_wait_bounded, for arrivals from the other CTA of the cluster.
__device__ __forceinline__ bool dn_wait_cluster(uint32_t bar, uint32_t parity) {
  for (uint32_t i = 0; i < (1u << 14); ++i) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.b32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(bar), "r"(parity), "r"(kWaitHintNs)
        : "memory");
    if (done) return true;
  }
  flag_error(STQ1_DEV_WAIT_LIMIT);
  return false;
}
// 2-D tensor copy into this CTA; in a pair the bytes are counted on the
// leader's barrier (bar is then a shared::cluster address).
template <int CG>
__device__ __forceinline__ void dn_load(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  if constexpr (CG == 2)
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::
            "r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
  else
    tma_load_2d(dst, map, x, y, bar);
}
template <bool I8, int CG>
__device__ __forceinline__ void dn_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
#define STQ1_DN_MMA(CGS, KIND)                                                                       \
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"                                      \
               "tcgen05.mma.cta_group::" CGS ".kind::" KIND " [%0], %1, %2, %3, p;\n\t}" ::"r"(d),    \
               "l"(a), "l"(b), "r"(idesc), "r"(accumulate)                                            \
               : "memory")
  if constexpr (I8 && CG == 2) STQ1_DN_MMA("2", "i8");
  else if constexpr (I8) STQ1_DN_MMA("1", "i8");
  else if constexpr (CG == 2) STQ1_DN_MMA("2", "f16");
  else STQ1_DN_MMA("1", "f16");
#undef STQ1_DN_MMA
}

// Shared-memory descriptors, 128-byte swizzle.  K-major: rows of 128 bytes,
// groups of 8 rows 1024 bytes apart; an MMA (32 bytes of K) advances the
// start by 32 bytes.  MN-major: blocks of 64 bf16 values along MN (8 KB: one
// 128-byte row per k, 64 of them), groups of 8 k 1024 bytes apart; an MMA (16
// values of k) advances the start by 2048 bytes.
template <bool MN>
__device__ __forceinline__ uint64_t dn_desc(uint32_t addr) {
  if constexpr (MN)
    return static_cast<uint64_t>((addr >> 4) & 0x3FFFu) | (static_cast<uint64_t>(8192 >> 4) << 16) |
           (static_cast<uint64_t>(1024 >> 4) << 32) | (static_cast<uint64_t>(1) << 46) |
           (static_cast<uint64_t>(2) << 61);
  else
    return smem_desc_sw128(addr);
}
template <bool MN>
constexpr uint32_t dn_advance() { return MN ? 2048u >> 4 : 32u >> 4; }

// Instruction descriptor: D fp32 or 32-bit integer (bits 4-5), A and B bf16 or
// signed 8-bit (bits 7-9, 10-12: 1 in both kinds), MN-major A and B (bits 15,
// 16), N >> 3 at bit 17, M >> 4 at bit 24.
template <bool I8, bool AMN, bool BMN>
constexpr uint32_t dn_idesc(int m, int n) {
  return (I8 ? 2u << 4 : 1u << 4) | (1u << 7) | (1u << 10) | (AMN ? 1u << 15 : 0u) | (BMN ? 1u << 16 : 0u) |
         (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(m >> 4) << 24);
}

// One step of an operand into shared memory: rows (K-major) or columns
// (MN-major) of 128 bytes of K, in `boxes` boxes of 64.
template <bool I8, bool MN, int CG>
__device__ __forceinline__ void dn_load_operand(uint32_t dst, const CUtensorMap* map, int step, int row, int boxes,
                                                uint32_t bar) {
  constexpr int kStep = I8 ? 128 : 64;      // values of K per step
  for (int i = 0; i < boxes; ++i) {
    if constexpr (MN) dn_load<CG>(dst + i * (kDnOperandBytes / 2), map, row + 64 * i, step * kStep, bar);
    else dn_load<CG>(dst + i * (kDnOperandBytes / 2), map, step * kStep, row + 64 * i, bar);
  }
}

__device__ __forceinline__ void dn_prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

template <bool I8>
__device__ __forceinline__ float dn_sum(uint32_t v, float sx, float sw) {
  if constexpr (I8) return i8_value(static_cast<int>(v), sx, sw);
  else return __uint_as_float(v);
}

// Position of a tile: groups of kDnGroup row tiles, column by column, so that
// the tiles in flight share rows of A and of B in L2.  (Groups of 8: 2-3% slower
// for the gradients of 4096 tokens by [4096, 7168], 1% faster for the gated form.)
constexpr int kDnGroup = 16;
__device__ __forceinline__ void dn_tile_pos(const DenseArgs& p, int tile, int& tm, int& tn) {
  const int per = kDnGroup * p.tiles_n;
  const int g = tile / per, in = tile - g * per;
  const int rows = min(kDnGroup, p.tiles_m - g * kDnGroup);
  tn = in / rows;
  tm = g * kDnGroup + in - tn * rows;
}

// ---------------------------------------------------------------------------
// Large products: pairs of CTAs on 256 x 256 tiles, one pair per two SMs, each
// working through its tiles.  Per 128-byte step of K a CTA copies 128 rows of A
// and 128 of B (32 KB) and the pair's four MMAs (M = N = 256) take 512 cycles,
// so that L2 has to deliver 64 bytes a clock and SM; a smaller tile would need
// more.  The sums of one tile are stored while the next one's are formed (two
// accumulators of 256 columns are all of TMEM).
//   warps 0-7   epilogue
//   warps 8, 10 producers of A and of B (one thread for both is too slow where
//               an operand takes four copies a step: 340 us became 372 for the
//               two gradients of 4096 tokens by [4096, 7168])
//   warp 9      MMAs of the pair (leader)
// Bound by the tensor pipe and, in a sustained loop, by the power limit: int8
// 4096 tokens by [4096, 7168] 78-82 us cold (3.0 PFLOP/s), 95 sustained at
// lower clocks, 70 with all codes zero; tensor pipe 76% of the active cycles,
// the rest start, last epilogue and an uneven last round.
// ---------------------------------------------------------------------------

// (Four stages are 5-9% slower; five with two result blocks per epilogue warp 1-4%.)
constexpr int kPairStages = 6;
constexpr int kPairEpi = 8;                         // epilogue warps: TMEM quadrants x column blocks in turn
constexpr int kPairSides = kPairEpi / 4;
constexpr int kPairWarpA = kPairEpi, kPairWarpMma = kPairEpi + 1, kPairWarpB = kPairEpi + 2;
constexpr int kPairThreads = 32 * (kPairEpi + 3);
constexpr int kPairOffStage = kPairStages * kDnStageBytes;
constexpr int kPairOffBar = kPairOffStage + kPairEpi * 4096;     // a block of results per epilogue warp
constexpr int kPairSmemBytes = 1024 + kPairOffBar + 256;
static_assert(kPairSmemBytes <= 232448, "shared memory per CTA is at most 227 KB");

// One warp's block of results: 32 rows (row = lane) of WORDS words, in shared
// memory as the tensor copies' swizzle wants it (rows of 128 bytes: 16-byte
// piece c at c ^ (row & 7); of 64: at c ^ ((row >> 1) & 3)), so that the
// row-wise stores do not meet on a bank, then by one tensor copy to global
// memory, which drops what lies past the edges.  The copy runs while the warp
// computes its next block.  (With reads of whole rows and 16-byte stores in its
// place the fp32 results of [4096, 512] x [512, 7168] took 50 us instead of 34.)
template <int WORDS>
__device__ __forceinline__ uint32_t dn_place(int row, int piece) {
  return row * (WORDS * 4) + ((piece ^ (WORDS == 32 ? row & 7 : (row >> 1) & 3)) << 4);
}
template <int WORDS>
__device__ __forceinline__ void dn_block_to_smem(const uint32_t* w, uint32_t buf) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int c = 0; c < WORDS / 4; ++c)
    asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(buf + dn_place<WORDS>(lane, c)), "r"(w[4 * c]),
                 "r"(w[4 * c + 1]), "r"(w[4 * c + 2]), "r"(w[4 * c + 3])
                 : "memory");
}
// REUSE: an earlier copy may still be reading the buffer.
template <int WORDS, bool REUSE>
__device__ __forceinline__ void dn_store_copy(const uint32_t* w, uint32_t buf, const CUtensorMap* map, int x, int y) {
  const int lane = threadIdx.x & 31;
  if constexpr (REUSE) {
    if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
    __syncwarp();
  }
  dn_block_to_smem<WORDS>(w, buf);
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(x), "r"(y), "r"(buf)
                 : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
  }
}
// The same (blocks of 32 words a row) for rows that tensor copies cannot
// address, because a row's bytes are no multiple of 16: a row at a time, a lane
// per word (4096 tokens by [2053, 2048]: 21.1 us with fp32 results, 21.6 with
// bf16; by copies, [2056, 2048], 18.6 and 17.2).
template <int ES>
__device__ __forceinline__ void dn_store_plain(const uint32_t* w, uint32_t buf, void* out, long long row0,
                                               long long rows, long long ld, long long col0, long long cols) {
  const int lane = threadIdx.x & 31;
  __syncwarp();                                     // the previous block's reads are done
  dn_block_to_smem<32>(w, buf);
  __syncwarp();
  const int n = static_cast<int>(min(32LL, rows - row0));
  const long long c = col0 + lane * (4 / ES);
  char* dst = static_cast<char*>(out) + (row0 * ld + c) * ES;
#pragma unroll 4
  for (int r = 0; r < n; ++r, dst += ld * ES) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(buf + dn_place<32>(r, lane >> 2) + 4 * (lane & 3)));
    if constexpr (ES == 4) {
      if (c < cols) *reinterpret_cast<uint32_t*>(dst) = v;
    } else if ((ld & 1) == 0) {
      if (c < cols) *reinterpret_cast<uint32_t*>(dst) = v;       // an even row length: both values or neither
    } else {
      if (c < cols) reinterpret_cast<uint16_t*>(dst)[0] = static_cast<uint16_t>(v);
      if (c + 1 < cols) reinterpret_cast<uint16_t*>(dst)[1] = static_cast<uint16_t>(v >> 16);
    }
  }
}

// One warp's block of finished sums: 32 rows by 64 columns of B at TMEM columns
// t0 (32) and t1 (32 more; gated: the 32 up sums of the same outputs), from sums
// to stored results.  scale: this lane's column scales of the two halves.
// loaded() runs once the sums are in registers.  my0, my1: maps of the gate and
// up halves of y.  REUSE: `buf` is one buffer for all of the warp's blocks; else
// there are three, used once.
template <int EPI, bool REUSE, typename F>
__device__ __forceinline__ void dn_block_epilogue(uint32_t t0, uint32_t t1, float sx, const float (&scale)[2],
                                                  const DenseArgs& p, const CUtensorMap* mo, const CUtensorMap* my0,
                                                  const CUtensorMap* my1, uint32_t buf, long long row0, long long col0,
                                                  F&& loaded) {
  constexpr bool I8 = epi_i8(EPI), GLU = epi_glu(EPI);
  constexpr int ES = EPI == kEpiI8F32 ? 4 : 2;
  const bool copies = p.N % (16 / ES) == 0, in = row0 < p.M && col0 < p.N;
  const int x = static_cast<int>(col0), y = static_cast<int>(row0);
  uint32_t v0[32], v1[32];
  STQ1_TMEM_LD32(t0, v0);
  STQ1_TMEM_LD32(t1, v1);
  tmem_wait_ld();
  loaded();
  if (!in) return;
  auto sum0 = [&](int j) { return dn_sum<I8>(v0[j], sx, I8 ? __shfl_sync(0xffffffffu, scale[0], j) : 0.f); };
  auto sum1 = [&](int j) { return dn_sum<I8>(v1[j], sx, I8 ? __shfl_sync(0xffffffffu, scale[1], j) : 0.f); };
  if constexpr (GLU) {
    // Rows and columns past the edges hold zeros or anything at all, which the
    // activation would take the long way round; they count as one instead.
    const bool row_in = row0 + (threadIdx.x & 31) < p.M;
    const int cols = static_cast<int>(min(32LL, p.N - col0));
    uint32_t act[16], kg[16], ku[16];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      float gv[16], uv[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const float gs = sum0(16 * c + j), us = sum1(16 * c + j);
        const bool is = row_in && 16 * c + j < cols;
        gv[j] = is ? gs : 1.f;
        uv[j] = is ? us : 1.f;
      }
      swiglu_bf16_pack<16>(gv, uv, act + 8 * c);
      if constexpr (EPI == kEpiGlu) {
#pragma unroll
        for (int j = 0; j < 16; j += 2) {
          kg[8 * c + j / 2] = bf16_bits_rn(gv[j]) | (bf16_bits_rn(gv[j + 1]) << 16);
          ku[8 * c + j / 2] = bf16_bits_rn(uv[j]) | (bf16_bits_rn(uv[j + 1]) << 16);
        }
      }
    }
    // N is a multiple of 8: rows are always whole pieces of 16 bytes
    dn_store_copy<16, REUSE>(act, buf, mo, x, y);
    if (EPI == kEpiGlu && p.y) {
      dn_store_copy<16, REUSE>(kg, REUSE ? buf : buf + 4096, my0, x, y);
      dn_store_copy<16, REUSE>(ku, REUSE ? buf : buf + 8192, my1, x, y);
    }
  } else if constexpr (ES == 4) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t w[32];
#pragma unroll
      for (int j = 0; j < 32; ++j) w[j] = __float_as_uint(h ? sum1(j) : sum0(j));
      if (col0 + 32 * h >= p.N) continue;
      if (copies) dn_store_copy<32, REUSE>(w, REUSE ? buf : buf + 4096 * h, mo, x + 32 * h, y);
      else dn_store_plain<4>(w, buf, p.out, row0, p.M, p.N, col0 + 32 * h, p.N);
    }
  } else {
    uint32_t w[32];
#pragma unroll
    for (int j = 0; j < 32; j += 2) {
      w[j / 2] = bf16_bits_rn(sum0(j)) | (bf16_bits_rn(sum0(j + 1)) << 16);
      w[16 + j / 2] = bf16_bits_rn(sum1(j)) | (bf16_bits_rn(sum1(j + 1)) << 16);
    }
    if (copies) dn_store_copy<32, REUSE>(w, buf, mo, x, y);
    else dn_store_plain<2>(w, buf, p.out, row0, p.M, p.N, col0, p.N);
  }
}
// The scales of a block's columns: of B's rows col0 + lane and, for the second
// half, 32 further (gated: of the up row of the same output).
template <bool GLU>
__device__ __forceinline__ void dn_block_scales(const DenseArgs& p, long long col0, float (&scale)[2]) {
  const long long c = col0 + (threadIdx.x & 31);
  scale[0] = c < p.N ? p.sw[c] : 0.f;
  if (GLU) scale[1] = c < p.N ? p.sw[p.N + c] : 0.f;
  else scale[1] = c + 32 < p.N ? p.sw[c + 32] : 0.f;
}

// A unit of the pair kernel's work: which product, the tile's place, and
// whether it is a whole tile or one half of its columns.
struct PairUnit {
  int prob, tm, tn, half;            // half: -1 whole, 0 / 1 the left / right 128 columns
};
// The i-th unit of this pair; false past its last one.
template <bool DUAL>
__device__ __forceinline__ bool pair_unit(const PairArgs& a, int i, PairUnit& u) {
  const int c = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  u.half = -1;
  u.prob = 0;
  int at = c + i * pairs;
  if constexpr (DUAL) {
    if (at < a.long_tiles) {
      u.prob = a.long_prob;
      dn_tile_pos(a.p[u.prob], at, u.tm, u.tn);
      return true;
    }
    u.prob = 1 - a.long_prob;
    i -= (a.long_tiles - c + pairs - 1) / pairs;     // the pair's long tiles are done
    if (c >= a.late) {
      if (i < a.lead) {
        dn_tile_pos(a.p[u.prob], i * (pairs - a.late) + c - a.late, u.tm, u.tn);
        return true;
      }
      i -= a.lead;
    }
    at = a.lead * (pairs - a.late) + c + i * pairs;
  }
  if (at >= a.units) return false;
  int tile = at;
  if (at >= a.full) {
    tile = a.full + ((at - a.full) >> 1);
    u.half = (at - a.full) & 1;
  }
  dn_tile_pos(a.p[u.prob], tile, u.tm, u.tn);
  return true;
}

// A place in the ring of stages: its index and the parity of its use.
struct RingPos {
  uint32_t s = 0, ph = 0;
  __device__ __forceinline__ void next() {
    if (++s == kPairStages) s = 0, ph ^= 1;
  }
};

// The MMAs of one unit: this thread waits for each step's operands (both
// CTAs'), issues four MMAs and hands the stage back.
template <bool I8, bool AMN, bool BMN>
__device__ __forceinline__ bool pair_mmas(uint32_t d, int n_k, uint32_t idesc, uint32_t sbase, uint32_t bar_full,
                                          uint32_t bar_empty, RingPos& r) {
  const uint64_t da0 = dn_desc<AMN>(sbase), db0 = dn_desc<BMN>(sbase + kDnOperandBytes);
  uint32_t acc = 0;
  for (int k = 0; k < n_k; ++k) {
    if (!dn_wait_cluster(bar_full + 8 * r.s, r.ph)) return false;
    tc_fence_after();
    const uint64_t da = da0 + r.s * (kDnStageBytes >> 4), db = db0 + r.s * (kDnStageBytes >> 4);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      dn_mma<I8, 2>(d, da + j * dn_advance<AMN>(), db + j * dn_advance<BMN>(), idesc, acc);
      acc = 1;
    }
    dn_commit_pair(bar_empty + 8 * r.s);
    r.next();
  }
  return true;
}

// This CTA's share of one operand for the steps of one unit.
template <bool I8, bool MN>
__device__ __forceinline__ bool pair_loads(const CUtensorMap* map, int n_k, int row, int boxes, uint32_t dst0,
                                           uint32_t bar_empty, uint32_t bar_full, uint32_t full0, uint32_t expect,
                                           RingPos& r) {
  for (int k = 0; k < n_k; ++k) {
    if (!mbar_wait_bounded(bar_empty + 8 * r.s, r.ph ^ 1)) return false;
    if (expect) mbar_arrive_expect_tx(bar_full + 8 * r.s, expect);
    dn_load_operand<I8, MN, 2>(dst0 + r.s * kDnStageBytes, map, k, row, boxes, full0 + 8 * r.s);
    r.next();
  }
  return true;
}

// DUAL: the second product's A is MN-major (dW beside dX).  map_o: the result;
// map_o1, map_o2: the second product's result (DUAL), or the gate and up halves
// of y (kEpiGlu).
template <int EPI, bool AMN, bool BMN, bool DUAL>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
dense_pair_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                  const __grid_constant__ CUtensorMap map_a1, const __grid_constant__ CUtensorMap map_b1,
                  const __grid_constant__ CUtensorMap map_o, const __grid_constant__ CUtensorMap map_o1,
                  const __grid_constant__ CUtensorMap map_o2, const __grid_constant__ PairArgs args) {
  constexpr bool I8 = epi_i8(EPI), GLU = epi_glu(EPI);
  static_assert(!(I8 && (AMN || BMN)), "8-bit operands are K-major");
  extern __shared__ __align__(16) uint8_t smem_raw[];
  const uint32_t sraw = smem_u32(smem_raw);
  const uint32_t sbase = (sraw + 1023u) & ~1023u;
  const uint32_t bar = sbase + kPairOffBar;
  const uint32_t bar_full = bar, bar_empty = bar + 64, bar_acc_full = bar + 128, bar_acc_empty = bar + 144,
                 bar_drain = bar + 160, s_tmem = bar + 176;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  if (threadIdx.x == 0) {
    for (int i = 0; i < kPairStages; ++i) {
      mbar_init(bar_full + 8 * i, 2);                // the leader's two producers
      mbar_init(bar_empty + 8 * i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar_acc_full + 8 * i, 1);
      mbar_init(bar_acc_empty + 8 * i, 2 * kPairEpi);   // the epilogue warps of both CTAs
    }
    mbar_init(bar_drain, 1);
    fence_mbar_init();
  }
  if (warp == kPairWarpMma) dn_tmem_alloc<2>(s_tmem, 512);
  if (threadIdx.x == 32 * kPairWarpA) dn_prefetch_map(&map_a);
  if (threadIdx.x == 32 * kPairWarpB) dn_prefetch_map(&map_b);
  tc_fence_before();
  cluster_sync_all();
  tc_fence_after();
  uint32_t tmem;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(tmem) : "r"(s_tmem));
  griddep_wait();
  griddep_launch_dependents();

  if (warp == kPairWarpA || warp == kPairWarpB) {
    // ---- producers: this CTA's 128 rows of A and 128 or 64 rows of B per step ----
    // A wait that runs out ends the role; it started after the last copy was
    // issued, so no copy is in flight any more by then.
    if (lane == 0) {
      const uint32_t full0 = dn_mapa(bar_full, 0);
      RingPos r;
      bool ok = true;
      PairUnit u;
      for (int i = 0; ok && pair_unit<DUAL>(args, i, u); ++i) {
        const DenseArgs& p = args.p[u.prob];
        const int boxes = warp == kPairWarpA || u.half < 0 ? 2 : 1;
        // bytes of both CTAs
        const uint32_t expect = rank != 0 ? 0 : (warp == kPairWarpA ? 2 * p.a_bytes : boxes * kDnOperandBytes);
        if (warp == kPairWarpA) {
          const int row = u.tm * 256 + static_cast<int>(rank) * kDnRows;
          if (DUAL && u.prob)
            ok = pair_loads<I8, true>(&map_a1, p.n_k, row, 2, sbase, bar_empty, bar_full, full0, expect, r);
          else
            ok = pair_loads<I8, AMN>(&map_a, p.n_k, row, 2, sbase, bar_empty, bar_full, full0, expect, r);
        } else {
          // gated: the leader loads the gate rows, its peer the up rows of the same outputs
          const int half = u.half > 0 ? 1 : 0;
          const int row = GLU ? static_cast<int>(rank * p.N) + u.tn * 128 + 64 * half
                              : u.tn * 256 + 128 * half + static_cast<int>(rank) * 64 * boxes;
          if (DUAL && u.prob)
            ok = pair_loads<I8, BMN>(&map_b1, p.n_k, row, boxes, sbase + kDnOperandBytes, bar_empty, bar_full, full0,
                                     expect, r);
          else
            ok = pair_loads<I8, BMN>(&map_b, p.n_k, row, boxes, sbase + kDnOperandBytes, bar_empty, bar_full, full0,
                                     expect, r);
        }
      }
    }
  } else if (warp == kPairWarpMma) {
    // ---- MMA issuer (leader only): both CTAs' operands, both CTAs' TMEM ----
    if (lane == 0 && rank == 0) {
      RingPos r;
      uint32_t t = 0;
      bool ok = true;
      PairUnit u;
      for (; ok && pair_unit<DUAL>(args, static_cast<int>(t), u); ++t) {
        const uint32_t buf = t & 1, use = t >> 1;
        ok = dn_wait_cluster(bar_acc_empty + 8 * buf, (use & 1) ^ 1);
        if (!ok) break;
        tc_fence_after();
        const int n_k = args.p[u.prob].n_k, n = u.half < 0 ? 256 : 128;
        const uint32_t d = tmem + 256 * buf;
        if (DUAL && u.prob)
          ok = pair_mmas<I8, true, BMN>(d, n_k, dn_idesc<I8, true, BMN>(256, n), sbase, bar_full, bar_empty, r);
        else
          ok = pair_mmas<I8, AMN, BMN>(d, n_k, dn_idesc<I8, AMN, BMN>(256, n), sbase, bar_full, bar_empty, r);
        // after a wait that ran out the sums are incomplete: the epilogue is not told of them,
        // gives up in its turn and stores nothing of this tile
        if (ok) dn_commit_pair(bar_acc_full + 8 * buf);
      }
      if (!ok) {
        // every MMA issued must be done before TMEM is freed (bounded)
        asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar_drain)
                     : "memory");
        mbar_wait_bounded(bar_drain, 0);
      }
    }
  } else {
    // ---- epilogue: warp w reads TMEM lanes 32 (w & 3).. and every kPairSides-th block of columns ----
    const int quad = warp & 3, side = warp >> 2;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(32 * quad) << 16);
    const uint32_t buf0 = sbase + kPairOffStage + warp * 4096;
    const uint32_t acc_empty0 = dn_mapa(bar_acc_empty, 0);
    constexpr int kMine = 4 / kPairSides;            // column blocks of a whole tile that are this warp's
    uint32_t t = 0;
    PairUnit un;
    for (; pair_unit<DUAL>(args, static_cast<int>(t), un); ++t) {
      const uint32_t buf = t & 1, use = t >> 1;
      const DenseArgs& p = args.p[un.prob];
      const CUtensorMap* mo = DUAL && un.prob ? &map_o1 : &map_o;
      const long long row0 = un.tm * 256LL + rank * kDnRows + 32 * quad;
      const float sx = I8 && row0 + lane < p.M ? p.sx[row0 + lane] : 0.f;
      // blocks of 64 columns of B: four of a whole tile, two of a half
      const int blocks = un.half < 0 ? 4 : 2;
      // the first output of a block, and the scales of its weight rows (fetched before the wait for the sums)
      auto first_col = [&](int blk) -> long long {
        if constexpr (GLU) return un.tn * 128LL + 32 * blk + (un.half > 0 ? 64 : 0);
        else return un.tn * 256LL + 64 * blk + (un.half > 0 ? 128 : 0);
      };
      float scale[kMine][2] = {};
      if constexpr (I8) {
#pragma unroll
        for (int i = 0; i < kMine; ++i) dn_block_scales<GLU>(p, first_col(side + i * kPairSides), scale[i]);
      }
      if (!__all_sync(0xffffffffu, mbar_wait_bounded(bar_acc_full + 8 * buf, use & 1))) break;
      tc_fence_after();
      const uint32_t acc = lanes + 256 * buf;
      auto release = [&]() {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) dn_arrive_remote(acc_empty0 + 8 * buf);
      };
#pragma unroll
      for (int i = 0; i < kMine; ++i) {
        const int blk = side + i * kPairSides;
        if (blk >= blocks) break;
        const bool last = blk + kPairSides >= blocks;
        const long long col0 = first_col(blk);
        dn_block_epilogue<EPI, true>(acc + (GLU ? 32 : 64) * blk,
                               acc + (GLU ? (un.half < 0 ? 128 : 64) + 32 * blk : 64 * blk + 32), sx, scale[i], p, mo,
                               &map_o1, &map_o2, buf0, row0, col0, [&]() {
                                 if (last) release();
                               });
      }
    }
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  }

  // all roles of both CTAs meet here (every wait above is bounded): the
  // barriers and shared memory a peer uses stay alive until it is done
  __syncwarp();
  tc_fence_before();
  cluster_sync_all();
  if (warp == kPairWarpMma) {
    tc_fence_after();
    dn_tmem_dealloc<2>(tmem, 512);
  }
}

// ---------------------------------------------------------------------------
// Products with few tiles: one CTA per 128 x 128 tile and piece of K.  Bound by
// the copies into shared memory: 32 KB per step in 436 cycles (75 bytes a clock)
// where the MMAs take 256; below about 128 tokens by the weights' way from HBM.
// [4096, 7168] int8: 9.1 us at 64 tokens, 10.1 at 128, 12.6 at 256, 17.1 at 512.
// (Prefetching the weights into L2 as well, from idle warps, is 5-18% slower.)
// ---------------------------------------------------------------------------

constexpr int kSplitStages = 6;
constexpr int kSplitThreads = 256;                  // warps 0-3 sums, 4 producer, 5 MMA; all store
constexpr int kSplitPitch = 132;                    // words per row of a finished piece
constexpr int kSplitOffBar = kSplitStages * kDnStageBytes;
constexpr int kSplitSmemBytes = 1024 + kSplitOffBar + 256;
static_assert(kDnRows * kSplitPitch * 4 <= kSplitOffBar, "a finished piece takes the place of the stages");
static_assert(kSplitThreads / 32 * 12288 <= kSplitOffBar, "and so do the blocks of results");

template <bool I8, bool AMN, bool BMN>
__device__ __forceinline__ bool split_mmas(uint32_t tmem, int steps, uint32_t sbase, uint32_t bar_full,
                                           uint32_t bar_empty) {
  constexpr uint32_t idesc = dn_idesc<I8, AMN, BMN>(128, 128);
  for (int it = 0; it < steps; ++it) {
    const uint32_t s = it % kSplitStages, ph = (it / kSplitStages) & 1;
    if (!mbar_wait_bounded(bar_full + 8 * s, ph)) return false;
    tc_fence_after();
    const uint64_t da = dn_desc<AMN>(sbase + s * kDnStageBytes);
    const uint64_t db = dn_desc<BMN>(sbase + s * kDnStageBytes + kDnOperandBytes);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      dn_mma<I8, 1>(tmem, da + j * dn_advance<AMN>(), db + j * dn_advance<BMN>(), idesc, (it | j) != 0);
    tc_commit(bar_empty + 8 * s);
  }
  return true;
}

struct SplitArgs {
  DenseArgs p[2];
  int tiles0;                        // 128 x 128 tiles of the first product
  int early;                         // B is not written by the kernel before: load it at once
};

// Each CTA of a cluster sums its piece of K in TMEM and lays the 128 x 128
// sums into its shared memory; each then adds up its share of the rows over
// all pieces, in the order of the pieces, and stores them: the result does not
// depend on which CTA comes first.  With one piece the sums go to the result
// as in the pair kernel.  DUAL, map_o...: as there.
template <int EPI, bool AMN, bool BMN, bool DUAL, int S>
__global__ void __launch_bounds__(kSplitThreads, 1)
dense_split_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                   const __grid_constant__ CUtensorMap map_a1, const __grid_constant__ CUtensorMap map_b1,
                   const __grid_constant__ CUtensorMap map_o, const __grid_constant__ CUtensorMap map_o1,
                   const __grid_constant__ CUtensorMap map_o2, const __grid_constant__ SplitArgs args) {
  constexpr bool I8 = epi_i8(EPI), GLU = epi_glu(EPI);
  extern __shared__ __align__(16) uint8_t smem_raw[];
  const uint32_t sraw = smem_u32(smem_raw);
  const uint32_t sbase = (sraw + 1023u) & ~1023u;
  const uint32_t bar = sbase + kSplitOffBar;
  const uint32_t bar_full = bar, bar_empty = bar + 64, bar_acc = bar + 128, bar_drain = bar + 136,
                 s_tmem = bar + 144, s_failed = bar + 148;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int piece = blockIdx.y;                      // the cluster of S runs along y
  const int prob = DUAL && static_cast<int>(blockIdx.x) >= args.tiles0 ? 1 : 0;
  const DenseArgs& p = args.p[prob];
  const CUtensorMap* ma = DUAL && prob ? &map_a1 : &map_a;
  const CUtensorMap* mb = DUAL && prob ? &map_b1 : &map_b;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kSplitStages; ++i) {
      mbar_init(bar_full + 8 * i, 1);
      mbar_init(bar_empty + 8 * i, 1);
    }
    mbar_init(bar_acc, 1);
    mbar_init(bar_drain, 1);
    fence_mbar_init();
    asm volatile("st.shared.u32 [%0], %1;" ::"r"(s_failed), "r"(0u) : "memory");
  }
  if (warp == 5) dn_tmem_alloc<1>(s_tmem, 128);
  if (warp == 4 && lane == 0) {
    dn_prefetch_map(ma);
    dn_prefetch_map(mb);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  uint32_t tmem;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(tmem) : "r"(s_tmem));
  int tm, tn;
  dn_tile_pos(p, static_cast<int>(blockIdx.x) - (prob ? args.tiles0 : 0), tm, tn);
  const int k0 = static_cast<int>(static_cast<long long>(p.n_k) * piece / S);
  const int k1 = static_cast<int>(static_cast<long long>(p.n_k) * (piece + 1) / S);
  constexpr int kOutCols = GLU ? 64 : 128;

  auto load_b = [&](int k, uint32_t dst, uint32_t b) {
    if constexpr (GLU) {
      // 64 gate rows and the 64 up rows of the same outputs
      dn_load_operand<I8, BMN, 1>(dst, mb, k, tn * 64, 1, b);
      dn_load_operand<I8, BMN, 1>(dst + kDnOperandBytes / 2, mb, k, static_cast<int>(p.N) + tn * 64, 1, b);
    } else {
      dn_load_operand<I8, BMN, 1>(dst, mb, k, tn * kDnRows, 2, b);
    }
  };
  // With `early` the stages' first weights are on their way while the kernel
  // before still runs (see dense_few_kernel for why that is sound).
  const int ahead = args.early ? min(kSplitStages, k1 - k0) : 0;
  if (warp == 4 && lane == 0) {
    for (int i = 0; i < ahead; ++i) {
      mbar_arrive_expect_tx(bar_full + 8 * i, p.a_bytes + kDnOperandBytes);
      load_b(k0 + i, sbase + i * kDnStageBytes + kDnOperandBytes, bar_full + 8 * i);
    }
  }
  __syncwarp();
  griddep_wait();
  griddep_launch_dependents();

  if (warp == 4) {
    if (lane == 0) {
      for (int k = k0; k < k1; ++k) {
        const uint32_t it = k - k0, s = it % kSplitStages, use = it / kSplitStages;
        const uint32_t dst = sbase + s * kDnStageBytes, b = bar_full + 8 * s;
        if (k - k0 >= ahead) {
          if (!mbar_wait_bounded(bar_empty + 8 * s, (use & 1) ^ 1)) break;
          mbar_arrive_expect_tx(b, p.a_bytes + kDnOperandBytes);
          load_b(k, dst + kDnOperandBytes, b);
        }
        if (AMN || (DUAL && prob)) {
          dn_load_operand<I8, true, 1>(dst, ma, k, tm * kDnRows, 2, b);
        } else {
          dn_load<1>(dst, ma, k * (I8 ? 128 : 64), tm * kDnRows, b);      // one box of as many rows as a tile has
        }
      }
    }
  } else if (warp == 5) {
    if (lane == 0) {
      bool ok;
      if (DUAL && prob) ok = split_mmas<I8, true, BMN>(tmem, k1 - k0, sbase, bar_full, bar_empty);
      else ok = split_mmas<I8, AMN, BMN>(tmem, k1 - k0, sbase, bar_full, bar_empty);
      // After a wait that ran out the sums are incomplete: who waits for them is not told, gives up
      // in its turn and stores nothing.  The MMAs issued must be done before TMEM is freed (bounded).
      tc_commit(ok ? bar_acc : bar_drain);
      if (!ok) mbar_wait_bounded(bar_drain, 0);
    }
  } else if (S > 1 && warp < 4) {
    // the sums to shared memory (the stages are free once the last MMA is done); an empty piece sums to zero
    const bool ok = __all_sync(0xffffffffu, mbar_wait_bounded(bar_acc, 0));
    tc_fence_after();
    const uint32_t lanes = tmem + (static_cast<uint32_t>(32 * warp) << 16);
    const uint32_t row = sbase + (32 * warp + lane) * (kSplitPitch * 4);
    if (!ok) {
      asm volatile("st.shared.u32 [%0], %1;" ::"r"(s_failed), "r"(1u) : "memory");
    } else if (tm * static_cast<long long>(kDnRows) + 32 * warp < p.M) {
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t v[32];
        STQ1_TMEM_LD32(lanes + 32 * c, v);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 32; i += 4)
          asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(row + 128 * c + 4 * i), "r"(k1 > k0 ? v[i] : 0u),
                       "r"(k1 > k0 ? v[i + 1] : 0u), "r"(k1 > k0 ? v[i + 2] : 0u), "r"(k1 > k0 ? v[i + 3] : 0u)
                       : "memory");
      }
    }
  }
  __syncwarp();
  if constexpr (S == 1) {
    // the whole of K: every warp takes 32 rows and half of the columns, from TMEM to the result
    // (by way of whole rows in shared memory, as with S > 1, 805 tokens by [544, 208] took 5.3 us, gated 7.0)
    const long long row0 = static_cast<long long>(tm) * kDnRows + 32 * (warp & 3);
    const long long col0 = static_cast<long long>(tn) * kOutCols + kOutCols / 2 * (warp >> 2);
    const float sx = I8 && row0 + lane < p.M ? p.sx[row0 + lane] : 0.f;
    float scale[2] = {};
    if constexpr (I8) dn_block_scales<GLU>(p, col0, scale);
    if (__all_sync(0xffffffffu, mbar_wait_bounded(bar_acc, 0))) {
      tc_fence_after();
      const uint32_t acc = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
      const int h = warp >> 2;
      dn_block_epilogue<EPI, false>(acc + (GLU ? 32 * h : 64 * h), acc + (GLU ? 64 + 32 * h : 64 * h + 32), sx, scale, p,
                             DUAL && prob ? &map_o1 : &map_o, &map_o1, &map_o2, sbase + warp * 12288, row0, col0, []() {});
      if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 5) {
      tc_fence_after();
      dn_tmem_dealloc<1>(tmem, 128);
    }
    return;
  }
  tc_fence_before();
  cluster_sync_all();                                // every piece lies in shared memory
  if (warp == 5) {
    tc_fence_after();
    dn_tmem_dealloc<1>(tmem, 128);
  }

  // this CTA's rows: piece, piece + S, ... ; a warp takes kRows of them at a time, so that their reads overlap, a
  // lane four sums of each (or two gate/up pairs)
  constexpr int kRows = S >= 8 ? 1 : 2;
  constexpr int kWarps = kSplitThreads / 32;
  const long long m0 = static_cast<long long>(tm) * kDnRows;
  const long long n0 = static_cast<long long>(tn) * kOutCols;
  const int rows = static_cast<int>(min(static_cast<long long>(kDnRows), p.M - m0));
  const int c0 = GLU ? 2 * lane : 4 * lane;          // first output column of this lane
  float swa[4] = {0.f, 0.f, 0.f, 0.f};
  if constexpr (I8) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const long long col = n0 + c0 + (GLU ? (i & 1) : i);
      if (col < p.N) swa[i] = p.sw[(GLU && i >= 2 ? p.N : 0) + col];
    }
  }
  // a piece without sums (lane q asks after piece q): none of the tile's rows is stored
  uint32_t failed = 0;
  if (lane < S) asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(failed) : "r"(dn_mapa(s_failed, lane)) : "memory");
  for (int r0 = piece + S * warp; r0 < rows; r0 += S * kWarps * kRows) {
    uint32_t w[kRows][S][4];
    float sxs[kRows];
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      const int r = min(r0 + j * S * kWarps, rows - 1);      // past the end: the last row again, not stored
      sxs[j] = I8 ? p.sx[m0 + r] : 0.f;
      const uint32_t at = sbase + r * (kSplitPitch * 4);
#pragma unroll
      for (int q = 0; q < S; ++q) {
        const uint32_t src = dn_mapa(at, q);
        uint32_t(&o)[4] = w[j][q];
        if constexpr (GLU) {
          asm volatile("ld.shared::cluster.v2.u32 {%0,%1}, [%2];" : "=r"(o[0]), "=r"(o[1]) : "r"(src + 8 * lane) : "memory");
          asm volatile("ld.shared::cluster.v2.u32 {%0,%1}, [%2];"
                       : "=r"(o[2]), "=r"(o[3])
                       : "r"(src + 256 + 8 * lane)
                       : "memory");
        } else {
          asm volatile("ld.shared::cluster.v4.u32 {%0,%1,%2,%3}, [%4];"
                       : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3])
                       : "r"(src + 16 * lane)
                       : "memory");
        }
      }
    }
    if (__any_sync(0xffffffffu, failed != 0)) break;
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      if (r0 + j * S * kWarps >= rows) break;
      const long long m = m0 + r0 + j * S * kWarps;
      float f[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t v = w[j][0][i];
#pragma unroll
        for (int q = 1; q < S; ++q) {
          if constexpr (I8) v += w[j][q][i];
          else v = __float_as_uint(__uint_as_float(v) + __uint_as_float(w[j][q][i]));
        }
        f[i] = dn_sum<I8>(v, sxs[j], swa[i]);
      }
      const long long col = n0 + c0;
      if constexpr (GLU) {
        // N is a multiple of 8 here and c0 even, so both columns exist or neither does
        if (col < p.N) {
          const uint32_t a = swiglu_bf16(f[0], f[2]) | (swiglu_bf16(f[1], f[3]) << 16);
          *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.out) + m * p.N + col) = a;
          if constexpr (EPI == kEpiGlu)
            if (p.y) {
              uint16_t* yr = p.y + m * 2 * p.N + col;
              *reinterpret_cast<uint32_t*>(yr) = bf16_bits_rn(f[0]) | (bf16_bits_rn(f[1]) << 16);
              *reinterpret_cast<uint32_t*>(yr + p.N) = bf16_bits_rn(f[2]) | (bf16_bits_rn(f[3]) << 16);
            }
        }
      } else if constexpr (EPI == kEpiI8F32) {
        float* dst = static_cast<float*>(p.out) + m * p.N + col;
        if (p.N % 4 == 0) {
          if (col < p.N) *reinterpret_cast<float4*>(dst) = make_float4(f[0], f[1], f[2], f[3]);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (col + i < p.N) dst[i] = f[i];
        }
      } else {
        uint16_t* dst = static_cast<uint16_t*>(p.out) + m * p.N + col;
        const uint32_t lo = bf16_bits_rn(f[0]) | (bf16_bits_rn(f[1]) << 16);
        const uint32_t hi = bf16_bits_rn(f[2]) | (bf16_bits_rn(f[3]) << 16);
        if (p.N % 4 == 0) {
          if (col < p.N) *reinterpret_cast<uint2*>(dst) = make_uint2(lo, hi);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (col + i < p.N) dst[i] = static_cast<uint16_t>((i < 2 ? lo : hi) >> (16 * (i & 1)));
        }
      }
    }
  }
  __syncwarp();
  cluster_sync_all();                                // a peer may still read this CTA's piece
}

}  // namespace stq1
