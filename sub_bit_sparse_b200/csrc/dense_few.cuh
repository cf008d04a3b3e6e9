// Products of the 8-bit integer and bf16 gated layers with up to 16 tokens:
// the weights are streamed once from HBM, everything else is kept small.
//
// A CTA owns a few weight rows (about N / SMs of them, so that every SM pulls
// its share) over the whole of K: no exchange between CTAs.  Its eight warps
// share out the 128-byte steps of K; each brings its own steps by tensor
// copies into slots of its own and contracts them with mma.sync.  (tcgen05
// is no help here: an MMA reads 64 or 128 rows of A whatever the tokens, and
// with 32 weight rows a step's four MMAs take longer than its bytes from HBM:
// 13 us against 6 on [4096, 7168] int8.)
//
// Bound by HBM and by what a launch cannot avoid, about 3 us from its start to
// the first bytes and from the last bytes to the stored sums: int8 [4096, 7168] at
// one token 7.1-8.6 us from HBM, 4.1 TB/s at best (29.4 MB alone would take 4.5),
// 5.2-6.4 where a part of the weights is in L2, and 8.0-9.3 and 6.8-7.4 at 16; bf16
// gated 10.8 us, 5.4 TB/s, 12.3 at 16.  (Loads straight into registers instead of
// copies through shared memory: 7.7 and 14.3 us at one token.)  The tokens' steps
// come beside the weights' as copies of their own: brought whole before the first
// step, 16 tokens took 7.2 (L2) and 14.1.
//
// A contraction may take its k in any order as long as both operands agree on
// it.  So a lane's share of an A fragment need not be the 4-byte pieces that
// mma.sync's layout spreads over a row: lane (g, t) takes the 16-byte pieces
// 2t and 2t + 1 of a step's rows g and g + 8 (words 0, 1 and 2, 3 of a piece
// feed one MMA each), and the same pieces of token g make the B fragments.
// In the copies' 128-byte swizzle the reads of a quarter warp (two rows, every
// second piece) fall on different banks.  8-bit and bf16 operands have the
// same word layout.
//
// For the gated forms a fragment's rows 0-7 are gate rows and its rows 8-15
// the up rows of the same outputs: a lane then holds g and u of one output.
#pragma once

#include "dense_math.cuh"
#include "dense_tile.cuh"
#include "quant_i8.cuh"

namespace stq1 {

constexpr int kFewMaxTokens = 16;
constexpr int kFewWarps = 8;
constexpr int kFewThreads = 32 * kFewWarps;
constexpr int kFewMaxSlots = 8;              // steps in flight per warp
constexpr int kFewHead = 1024;               // barriers and small arrays
static_assert(8 * kFewMaxSlots * kFewWarps + 3 * 4 * kFewMaxTokens <= kFewHead, "");

struct FewArgs {
  const void* x;               // MADE: [T, K] bf16 (else by tensor copies)
  const float *sx, *sw;
  void* out;
  uint16_t* y;
  long long N, K;              // outputs (for the gated forms half of the weight rows); values per row (MADE)
  int T;
  int rows;                    // outputs per CTA
  int pad;                     // weight rows of one step in shared memory (a multiple of 16)
  int n_k;                     // 128-byte steps of K
  int n_slots;
  int early;                   // the weights are not written by the kernel before: load them at once
  uint32_t* amax;              // fp32 bits of each token's largest magnitude: of x, read (MADE); of the
                               // output, raised (8-bit gated form), or NULL
};

// Bytes of a step of the tokens beside a slot: a lone token takes one plain row
// (all lanes read it), more take groups of eight rows in the copies' swizzle; none
// where their codes are made here.
__host__ __device__ constexpr int few_x_bytes(int T, bool made) {
  return made ? 0 : (T == 1 ? kDnStepBytes : (T + 7) / 8 * 8 * kDnStepBytes);
}
// Bytes between tokens whose codes are made here: whole steps and 16 more, so that two
// tokens' pieces (every second one of a step) fall on different banks.
__host__ __device__ constexpr long long few_pitch(int n_k) { return n_k * 128LL + 16; }

__device__ __forceinline__ void few_mma(int (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void few_mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// MADE: x is bf16 and its codes are made here, from each token's largest
// magnitude, which the kernel that wrote x kept (the down projection of the
// 8-bit layer).  For the first projection the magnitudes would have to be found
// by every CTA, which takes longer than a launch of its own (at four tokens of a
// [4096, 7168] layer by 2.5 us).
// MT: fragments of 16 weight rows (at most); NT: groups of 8 tokens.
template <int EPI, bool MADE, int MT, int NT>
__global__ void __launch_bounds__(kFewThreads, 2)
dense_few_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x, const FewArgs p) {
  constexpr bool I8 = epi_i8(EPI), GLU = epi_glu(EPI);
  static_assert(I8 || !MADE, "codes are made for 8-bit weights");
  using Acc = std::conditional_t<I8, int, float>;
  constexpr int ES = I8 ? 1 : 2;
  constexpr int kStep = kDnStepBytes / ES;
  extern __shared__ __align__(16) uint8_t smem_raw[];
  const uint32_t sraw = smem_u32(smem_raw);
  const uint32_t sbase = (sraw + 1023u) & ~1023u;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  // the warps' barriers, then 16 words each of scales, their inverses and largest outputs
  const uint32_t s_scale = sbase + 8 * kFewMaxSlots * kFewWarps, s_inv_at = s_scale + 64, s_amax_at = s_inv_at + 64;
  const uint32_t slot_bytes = p.pad * kDnStepBytes, x_bytes = few_x_bytes(p.T, MADE);
  const uint32_t s_w = sbase + kFewHead;                               // the warps' slots
  const uint32_t s_x = s_w + kFewWarps * p.n_slots * slot_bytes;       // the slots' tokens, or (MADE) their codes
  const uint32_t pitch = static_cast<uint32_t>(few_pitch(p.n_k));
  const uint32_t my_bar = sbase + 8 * kFewMaxSlots * warp;
  const uint32_t my_slots = s_w + warp * p.n_slots * slot_bytes, my_x = s_x + warp * p.n_slots * x_bytes;
  const long long n0 = static_cast<long long>(blockIdx.x) * p.rows;

  // ---- this warp's first steps ----
  const int y0 = static_cast<int>(n0), y1 = static_cast<int>(p.N + n0);
  const uint32_t step_bytes = ((GLU ? 2 : 1) * p.rows + (MADE ? 0 : p.T)) * kDnStepBytes;
  auto fetch = [&](int step, int slot) {                               // lane 0 only
    const uint32_t bar = my_bar + 8 * slot, dst = my_slots + slot * slot_bytes;
    mbar_arrive_expect_tx(bar, step_bytes);
    dn_load<1>(dst, &map_w, step * kStep, y0, bar);
    if constexpr (GLU) dn_load<1>(dst + slot_bytes / 2, &map_w, step * kStep, y1, bar);
  };
  auto fetch_x = [&](int step, int slot) {                             // and its tokens
    if constexpr (!MADE) dn_load<1>(my_x + slot * x_bytes, &map_x, step * kStep, 0, my_bar + 8 * slot);
  };
  if (threadIdx.x == 0) {
    dn_prefetch_map(&map_w);
    if constexpr (!MADE) dn_prefetch_map(&map_x);
  }
  if (lane == 0) {
    for (int i = 0; i < p.n_slots; ++i) mbar_init(my_bar + 8 * i, 1);
    fence_mbar_init();
  }
  __syncwarp();
  // With `early` the weights are fetched while the kernel before still runs:
  // what ran before that one is complete (its CTAs passed their own wait
  // before they let this kernel start), and the weights are not its output.
  if (!p.early) griddep_wait();
  if (lane == 0)
    for (int i = 0; i < p.n_slots && warp + kFewWarps * i < p.n_k; ++i) fetch(warp + kFewWarps * i, i);
  if (p.early) griddep_wait();
  griddep_launch_dependents();
  if (lane == 0)
    for (int i = 0; i < p.n_slots && warp + kFewWarps * i < p.n_k; ++i) fetch_x(warp + kFewWarps * i, i);

  if constexpr (MADE) {
    // 16 values a piece, the CTA's pieces dealt out to all threads, eight loads
    // of each thread in flight (a warp per token took 0.5 us more at 16 tokens)
    constexpr int kMany = 4;
    const int nv = static_cast<int>(p.K / 16), total = nv * p.T;
    float* s_inv = reinterpret_cast<float*>(smem_raw + (s_inv_at - sraw));
    if (threadIdx.x < p.T) {
      const I8Scale sc = i8_scale(__ldcg(p.amax + threadIdx.x));
      s_inv[threadIdx.x] = sc.inv;
      asm volatile("st.shared.f32 [%0], %1;" ::"r"(s_scale + 4 * threadIdx.x), "f"(sc.scale) : "memory");
    }
    for (int i0 = threadIdx.x; i0 < total + static_cast<int>(threadIdx.x); i0 += kMany * kFewThreads) {
      Row8<false> a[kMany], b[kMany];
#pragma unroll
      for (int j = 0; j < kMany; ++j) {
        const int i = i0 + j * kFewThreads;
        if (i < total) {                             // (the tokens' rows lie one after another)
          a[j].load(p.x, 2 * i);
          b[j].load(p.x, 2 * i + 1);
        }
      }
      if (i0 == static_cast<int>(threadIdx.x)) __syncthreads();   // the scales
#pragma unroll
      for (int j = 0; j < kMany; ++j) {
        const int i = i0 + j * kFewThreads;
        if (i < total) {
          const int tok = i / nv;
          const float inv = s_inv[tok];
          const uint2 lo = a[j].codes(inv), hi = b[j].codes(inv);
          asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(s_x + tok * pitch + 16 * (i - tok * nv)), "r"(lo.x),
                       "r"(lo.y), "r"(hi.x), "r"(hi.y)
                       : "memory");
        }
      }
    }
    // K past its end within the last step: the weights read as zero there, and so must the tokens
    const int tail = p.n_k * 8 - nv;
    for (int i = threadIdx.x; i < tail * p.T; i += kFewThreads)
      asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(s_x + (i / tail) * pitch + 16 * (nv + i % tail)), "r"(0u)
                   : "memory");
    __syncthreads();
  }
  bool ok = true;

  // ---- this warp's steps ----
  const int mt = p.pad >> 4;
  Acc acc[MT][NT][4] = {};
  // rows of a fragment in a slot, and this lane's pieces of them
  const uint32_t up = GLU ? slot_bytes / 2 : 8 * kDnStepBytes;         // from row g to the row of fragment row g + 8
  const uint32_t frag = (GLU ? 8 : 16) * kDnStepBytes;
  const uint32_t off0 = g * kDnStepBytes + (((2 * t) ^ g) << 4), off1 = g * kDnStepBytes + (((2 * t + 1) ^ g) << 4);
  int slot = 0;
  uint32_t ph = 0;
  for (int step = warp; step < p.n_k; step += kFewWarps) {
    if (!mbar_wait_bounded(my_bar + 8 * slot, ph)) {
      ok = false;
      break;                                         // (its own copies have had that wait to land)
    }
    const uint32_t base = my_slots + slot * slot_bytes;
    uint4 x0[NT], x1[NT];                            // (what stands for a token past the last is not stored)
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      if constexpr (MADE) {
        const bool token = 8 * n + g < p.T;
        const uint32_t at = s_x + (8 * n + g) * pitch + step * kDnStepBytes + 32 * t;
        x0[n] = token ? lds_v4(at) : make_uint4(0, 0, 0, 0);
        x1[n] = token ? lds_v4(at + 16) : make_uint4(0, 0, 0, 0);
      } else {
        const uint32_t at = my_x + slot * x_bytes + n * 8 * kDnStepBytes;
        x0[n] = lds_v4(at + (p.T == 1 ? 32 * t : off0));
        x1[n] = lds_v4(at + (p.T == 1 ? 32 * t + 16 : off1));
      }
    }
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      if (i < mt) {
        const uint32_t b = base + i * frag;
        const uint4 a0 = lds_v4(b + off0), a1 = lds_v4(b + up + off0);
        const uint4 c0 = lds_v4(b + off1), c1 = lds_v4(b + up + off1);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          few_mma(acc[i][n], a0.x, a1.x, a0.y, a1.y, x0[n].x, x0[n].y);
          few_mma(acc[i][n], a0.z, a1.z, a0.w, a1.w, x0[n].z, x0[n].w);
          few_mma(acc[i][n], c0.x, c1.x, c0.y, c1.y, x1[n].x, x1[n].y);
          few_mma(acc[i][n], c0.z, c1.z, c0.w, c1.w, x1[n].z, x1[n].w);
        }
      }
    }
    __syncwarp();                                    // every lane has read the slot
    const int next = step + kFewWarps * p.n_slots;
    if (lane == 0 && next < p.n_k) {
      fetch(next, slot);
      fetch_x(next, slot);
    }
    if (++slot == p.n_slots) slot = 0, ph ^= 1;
  }
  __syncthreads();                                   // the slots are free: the warps' sums take their place
  const uint32_t red = s_w + (warp * MT * NT * 32 + lane) * 16;
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int n = 0; n < NT; ++n)
      asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(red + (i * NT + n) * 512),
                   "r"(*reinterpret_cast<const uint32_t*>(&acc[i][n][0])), "r"(*reinterpret_cast<const uint32_t*>(&acc[i][n][1])),
                   "r"(*reinterpret_cast<const uint32_t*>(&acc[i][n][2])), "r"(*reinterpret_cast<const uint32_t*>(&acc[i][n][3]))
                   : "memory");
  // the CTA's largest outputs of each token (8-bit gated form)
  uint32_t* s_amax = reinterpret_cast<uint32_t*>(smem_raw + (s_amax_at - sraw));
  if (EPI == kEpiI8Glu && threadIdx.x < kFewMaxTokens) s_amax[threadIdx.x] = 0u;
  if (__syncthreads_or(!ok)) return;                 // a wait ran out (flagged): nothing is stored

  // sums over the warps, in their order; consecutive threads take consecutive outputs of one token
  const int count = static_cast<int>(min(static_cast<long long>(p.rows), p.N - n0));
  for (int e = threadIdx.x; e < count * p.T; e += kFewThreads) {
    const int tok = e / count, r = e - tok * count;
    const int i = GLU ? r >> 3 : r >> 4;
    const uint32_t at = s_w + ((i * NT + (tok >> 3)) * 32 + (r & 7) * 4 + ((tok & 7) >> 1)) * 16 + 4 * (tok & 1);
    auto total = [&](int reg) {
      Acc v;
#pragma unroll
      for (int q = 0; q < kFewWarps; ++q) {
        uint32_t w;
        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w) : "r"(at + 4 * reg + q * MT * NT * 512));
        const Acc a = *reinterpret_cast<const Acc*>(&w);
        if (q == 0) v = a;
        else v += a;
      }
      return v;
    };
    const long long n = n0 + r;
    float sx = 0.f;
    if constexpr (MADE) asm volatile("ld.shared.f32 %0, [%1];" : "=f"(sx) : "r"(s_scale + 4 * tok));
    else if constexpr (I8) sx = p.sx[tok];
    auto value = [&](Acc v, long long row) -> float {
      if constexpr (I8) return i8_value(v, sx, p.sw[row]);
      else return v;
    };
    if constexpr (GLU) {
      const float gv = value(total(0), n), uv = value(total(2), p.N + n);
      const uint32_t bits = swiglu_bf16(gv, uv);
      static_cast<uint16_t*>(p.out)[tok * p.N + n] = static_cast<uint16_t>(bits);
      if constexpr (EPI == kEpiI8Glu)
        if (p.amax) atomicMax(s_amax + tok, (bits & 0x7FFFu) << 16);
      if constexpr (EPI == kEpiGlu)
        if (p.y) {
          p.y[tok * 2 * p.N + n] = static_cast<uint16_t>(bf16_bits_rn(gv));
          p.y[tok * 2 * p.N + p.N + n] = static_cast<uint16_t>(bf16_bits_rn(uv));
        }
    } else {
      const float v = value(total((r & 8) ? 2 : 0), n);
      if constexpr (EPI == kEpiI8F32) static_cast<float*>(p.out)[tok * p.N + n] = v;
      else static_cast<uint16_t*>(p.out)[tok * p.N + n] = static_cast<uint16_t>(bf16_bits_rn(v));
    }
  }
  if constexpr (EPI == kEpiI8Glu) {
    // one update per token and CTA: one per output took 9 us at 16 tokens.  (A
    // maximum does not depend on the order of its updates.)
    if (p.amax) {
      __syncthreads();
      if (threadIdx.x < p.T) atomicMax(p.amax + threadIdx.x, s_amax[threadIdx.x]);
    }
  }
}

}  // namespace stq1
