// linear_tc.cuh -- the layer's projections on sm_100a tensor cores.
//
//   out[t][n] = residual + mul * act(sum_k x[t][k] W[n][k] + bias[n])
//
// Both kernels compute the transposed product D[n][t]: W's rows are the MMA's M side (128
// a CTA), the tokens its N side. One token then still fills the M side, so a decode step's
// few tokens cost no idle rows, only the 16-token minimum of the N side; and a thread of the
// epilogue owns one feature (its TMEM lane), so a warp's store of one token covers 32
// neighbouring features. x and W are both K-major: TMA streams 128-byte-wide K blocks (64
// bf16 or 128 E4M3 elements, 128-byte swizzle) and one elected lane issues the MMAs, fp32 in
// TMEM. Rows and columns past T, N and K arrive as zeros and are not stored.
//
// linear_split_kernel (few tokens): bound by the bytes of W. One CTA per 128 features x NT
// tokens x K slice; the slices of a tile are a cluster, which adds its fp32 partial sums
// through distributed shared memory in slice order. One launch, no workspace, and the same
// sum in every run.
//
// linear_pair_kernel (many tokens): bound by the tensor cores. Persistent pairs of CTAs
// (tcgen05 cta_group::2), 256 features x NT tokens a tile, with two accumulators in TMEM so
// that a tile's epilogue runs under the next tile's main loop.
#pragma once

#include "common.cuh"
#include "linear.cuh"
#include "ptx.cuh"

namespace mla {
namespace lin {

constexpr int kM = 128;              // features (MMA rows) per CTA
constexpr int kKBytes = 128;         // bytes of a K block of one row
constexpr int kABytes = kM * kKBytes;

template <bool F8> __host__ __device__ constexpr int kb_elems() { return F8 ? 128 : 64; }

// Epilogue of CNT consecutive tokens t0 + j of feature n, one feature per thread; tokens
// past `tokens` and features past N are computed on zeros and not stored. Every load is
// issued before the arithmetic that waits for it.
template <bool F8, int CNT>
__device__ __forceinline__ void finish_tokens(const Params& p, float (&v)[CNT], int64_t t0, int tokens, int32_t n,
                                              float bias, float ws) {
  if (n >= p.N) return;
  const int64_t at = t0 * p.N + n;
  __nv_bfloat16 m[CNT], r[CNT];
  if (p.mul) {
#pragma unroll
    for (int j = 0; j < CNT; ++j)
      if (j < tokens) m[j] = p.mul[at + (int64_t)j * p.N];
  }
  if (p.res) {
#pragma unroll
    for (int j = 0; j < CNT; ++j)
      if (j < tokens) r[j] = p.res[at + (int64_t)j * p.N];
  }
  if (F8) {
#pragma unroll
    for (int j = 0; j < CNT; ++j)
      if (j < tokens) v[j] = v[j] * ws * scale_of(p.xs[t0 + j]);
  }
#pragma unroll
  for (int j = 0; j < CNT; ++j) v[j] += bias;
  if (p.act != kActNone) {
#pragma unroll
    for (int j = 0; j < CNT; ++j) v[j] = activate(v[j], p.act);
  }
#pragma unroll
  for (int j = 0; j < CNT; ++j)
    if (j < tokens) {
      float y = v[j];
      if (p.mul) y *= __bfloat162float(m[j]);
      if (p.res) y += __bfloat162float(r[j]);
      p.out[at + (int64_t)j * p.N] = __float2bfloat16_rn(y);
    }
}

// ------------------------------------------------------------------ few tokens: K slices
template <bool F8, int NT, int STAGES>
struct SplitCfg {
  static constexpr int kBBytes = NT * kKBytes;
  static constexpr int kStageBytes = kABytes + kBBytes;
  static constexpr int kPartBytes = kM * NT * 4;
  static constexpr int kPipeBytes = STAGES * kStageBytes > kPartBytes ? STAGES * kStageBytes : kPartBytes;
  static constexpr int kOffBar = kPipeBytes;
  static constexpr int kSmemBytes = kOffBar + 256 + 1024;      // barriers + alignment slack
  static constexpr uint32_t kCols = NT < 32 ? 32 : NT;
  static constexpr uint32_t kIdesc = F8 ? ptx::idesc_e4m3_f32(kM, NT, 0, 0) : ptx::idesc_bf16_f32(kM, NT, 0, 0);
  static_assert(NT % 16 == 0 && NT <= 256 && kStageBytes % 1024 == 0, "tile");
};

// grid (slices, feature tiles, token tiles), clusters of `slices` CTAs.
template <bool F8, int NT, int STAGES>
__global__ void __launch_bounds__(128) linear_split_kernel(const __grid_constant__ CUtensorMap tmW,
                                                           const __grid_constant__ CUtensorMap tmX, const Params p) {
  using C = SplitCfg<F8, NT, STAGES>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = ptx::smem_u32(smem);
  auto bar = [&](int i) { return sbase + C::kOffBar + 8u * i; };   // [0,S) full, [S,2S) empty, 2S done
  const uint32_t tmem_holder = sbase + C::kOffBar + 8u * (2 * STAGES + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffBar + 8 * (2 * STAGES + 3));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int slices = gridDim.x, slice = blockIdx.x;
  const int n0 = blockIdx.y * kM;
  const int64_t t0 = (int64_t)blockIdx.z * NT;
  const int kblk = (p.K + kb_elems<F8>() - 1) / kb_elems<F8>();
  const int kb0 = (int)((int64_t)kblk * slice / slices), kb1 = (int)((int64_t)kblk * (slice + 1) / slices);
  const int nkb = kb1 - kb0;      // at least one: the host cuts no more slices than K blocks

  if (tid == 0) {
    *abort_flag = 0;
    for (int s = 0; s < STAGES; ++s) {
      ptx::mbar_init(bar(s), 1);
      ptx::mbar_init(bar(STAGES + s), 1);
    }
    ptx::mbar_init(bar(2 * STAGES), 1);
    ptx::fence_mbar_init();
  }
  if (warp == 2) {
    ptx::tmem_alloc(tmem_holder, C::kCols);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tbase = *reinterpret_cast<volatile uint32_t*>(smem + C::kOffBar + 8 * (2 * STAGES + 2));
  auto wait_all = [&](uint32_t b, uint32_t parity) -> bool {
    return __all_sync(0xffffffffu, ptx::mbar_wait_bounded(b, parity, abort_flag, p.timeout_ns));
  };
  auto give_up = [&]() {
    if (lane == 0) {
      raise_status(kStatusTimeout);
      *abort_flag = 1;
    }
  };
  bool ok = true;

  if (warp == 0) {
    // ---------------------------------------------------------------- loads
    const bool leader = ptx::elect_one();
    int issued = 0;
    for (int i = 0; i < nkb; ++i) {
      const int s = i % STAGES, use = i / STAGES;
      if (!wait_all(bar(STAGES + s), (use & 1) ^ 1)) { give_up(); ok = false; break; }
      if (leader) {
        const uint32_t sa = sbase + s * C::kStageBytes, sb = sa + kABytes;
        ptx::mbar_arrive_expect_tx(bar(s), C::kStageBytes);
        ptx::tma_load_2d(sa, &tmW, bar(s), (kb0 + i) * kb_elems<F8>(), n0);
        ptx::tma_load_2d(sb, &tmX, bar(s), (kb0 + i) * kb_elems<F8>(), (int32_t)t0);
      }
      issued = i + 1;
    }
    // copies in flight land in this CTA's shared memory: wait (bounded) for the last ones
    for (int i = issued > STAGES ? issued - STAGES : 0; i < issued; ++i) wait_all(bar(i % STAGES), (i / STAGES) & 1);
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issuer
    const bool leader = ptx::elect_one();
    for (int i = 0; i < nkb; ++i) {
      const int s = i % STAGES, use = i / STAGES;
      if (!wait_all(bar(s), use & 1)) { give_up(); ok = false; break; }
      ptx::tc_fence_after();
      const uint32_t sa = sbase + s * C::kStageBytes, sb = sa + kABytes;
      const uint64_t dA = ptx::sdesc_sw128(sa, 16, 1024), dB = ptx::sdesc_sw128(sb, 16, 1024);
      if (leader) {
#pragma unroll
        for (int kk = 0; kk < kKBytes / 32; ++kk) {
          const uint64_t o = (uint64_t)((kk * 32) >> 4);
          if (F8) ptx::umma_f8_ss(tbase, dA + o, dB + o, C::kIdesc, (i | kk) ? 1u : 0u);
          else ptx::umma_f16_ss(tbase, dA + o, dB + o, C::kIdesc, (i | kk) ? 1u : 0u);
        }
        ptx::umma_commit(bar(STAGES + s));
        if (i == nkb - 1) ptx::umma_commit(bar(2 * STAGES));
      }
      __syncwarp();
    }
  }

  // ---------------------------------------------------------------- epilogue (all warps)
  const bool done = ok && wait_all(bar(2 * STAGES), 0);
  if (!done) give_up();
  ptx::tc_fence_after();
  const int tokens = (int)min((int64_t)NT, p.T - t0);
  const int32_t n = n0 + tid;
  const float bias = p.bias && n < p.N ? __bfloat162float(p.bias[n]) : 0.f;
  const float ws = F8 && n < p.N ? scale_of(p.ws[n]) : 1.f;
  const uint32_t trow = tbase + ((32u * warp) << 16);
  if (slices == 1) {
    if (done) {
#pragma unroll 1
      for (int c = 0; c < tokens; c += 16) {
        float v[16];
        ptx::tmem_ld_32x32b_x16(trow + c, v);
        ptx::tmem_wait_ld();
        finish_tokens<F8, 16>(p, v, t0 + c, tokens - c, n, bias, ws);
      }
    }
  } else {
    // the slice's sums into this CTA's shared memory, [token][feature]: every load of this
    // CTA has landed and every MMA has read its operands (the done barrier), so the stages
    // are free
    float* part = reinterpret_cast<float*>(smem);
    if (done) {
#pragma unroll 1
      for (int c = 0; c < tokens; c += 16) {
        float v[16];
        ptx::tmem_ld_32x32b_x16(trow + c, v);
        ptx::tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < 16; ++j) part[(c + j) * kM + tid] = v[j];
      }
    }
    __syncthreads();
    ptx::cluster_sync();
    if (done) {
      // CTA `slice` adds tokens slice, slice + slices, ..
      for (int t = slice; t < tokens; t += slices) {
        float v[1] = {0.f};
        for (int s = 0; s < slices; ++s)
          v[0] += ptx::ld_cluster_f32(ptx::map_peer(sbase + 4u * (t * kM + tid), s));
        finish_tokens<F8, 1>(p, v, t0 + t, 1, n, bias, ws);
      }
    }
    __syncthreads();
    ptx::cluster_sync();   // no CTA leaves while another reads its partial sums
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tbase, C::kCols);
  }
}

// ------------------------------------------------------------------ many tokens: SM pairs
template <bool F8, int NT, int STAGES>
struct PairCfg {
  static constexpr int kHalf = NT / 2;                 // tokens whose rows a CTA loads
  static constexpr int kBBytes = kHalf * kKBytes;
  static constexpr int kStageBytes = kABytes + kBBytes;
  static constexpr int kOffBar = STAGES * kStageBytes;
  static constexpr int kEpiWarps = 4;
  static constexpr int kThreads = 32 * (4 + kEpiWarps);
  static constexpr int kSmemBytes = kOffBar + 256 + 1024;
  static constexpr uint32_t kCols = 2 * NT;            // two accumulators
  static constexpr uint32_t kIdesc =
      F8 ? ptx::idesc_e4m3_f32(2 * kM, NT, 0, 0) : ptx::idesc_bf16_f32(2 * kM, NT, 0, 0);
  static_assert(kStageBytes % 1024 == 0 && kABytes % 1024 == 0, "stage alignment");
  static_assert(8 * (2 * STAGES + 4) + 16 <= 256, "barriers");
};

constexpr int kGroupT = 8;   // token tiles that share a sweep over the feature tiles

// Tile `i` of tiles_n x tiles_t: groups of kGroupT token tiles, within a group the token
// tile fastest, so the pairs at work at one time share feature and token tiles in L2.
__device__ __forceinline__ void tile_of(int64_t i, int tiles_n, int tiles_t, int& tn, int& tt) {
  const int64_t per = (int64_t)kGroupT * tiles_n;
  const int g = (int)(i / per);
  const int first = g * kGroupT, width = min(kGroupT, tiles_t - first);
  const int64_t rem = i - (int64_t)g * per;
  tn = (int)(rem / width);
  tt = first + (int)(rem % width);
}

template <bool F8, int NT, int STAGES>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(PairCfg<F8, NT, STAGES>::kThreads, 1)
linear_pair_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX, const Params p) {
  using C = PairCfg<F8, NT, STAGES>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = ptx::smem_u32(smem);
  // [0,S) full (even CTA: both CTAs' loads), [S,2S) empty (each CTA), 2S.. accumulator full
  // (each CTA), 2S+2.. accumulator free (even CTA: both CTAs' epilogue warps)
  auto bar = [&](int i) { return sbase + C::kOffBar + 8u * i; };
  constexpr int kFull = 0, kEmpty = STAGES, kAccFull = 2 * STAGES, kAccFree = 2 * STAGES + 2;
  constexpr int kOffMisc = C::kOffBar + 8 * (2 * STAGES + 4);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kOffMisc + 8);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = ptx::cluster_rank();
  const bool even = rank == 0;
  auto lead = [&](uint32_t a) { return ptx::map_peer(a, 0); };
  const int tiles_n = (p.N + 2 * kM - 1) / (2 * kM), tiles_t = (int)(((int64_t)p.T + NT - 1) / NT);
  const int64_t tiles = (int64_t)tiles_n * tiles_t;
  const int pairs = gridDim.x / 2, pair = blockIdx.x / 2;
  const int kblk = (p.K + kb_elems<F8>() - 1) / kb_elems<F8>();

  if (tid == 0) {
    *abort_flag = 0;
    for (int s = 0; s < STAGES; ++s) {
      ptx::mbar_init(bar(kFull + s), 1);
      ptx::mbar_init(bar(kEmpty + s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      ptx::mbar_init(bar(kAccFull + b), 1);
      ptx::mbar_init(bar(kAccFree + b), 2 * C::kEpiWarps);
    }
    ptx::fence_mbar_init();
  }
  if (warp == 2) {
    ptx::tmem_alloc_pair(sbase + kOffMisc, C::kCols);
    ptx::tmem_relinquish_pair();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::cluster_sync();   // both CTAs' barriers exist before anyone arrives, loads or issues
  ptx::tc_fence_after();
  const uint32_t tbase = *reinterpret_cast<volatile uint32_t*>(smem + kOffMisc);
  auto wait_all = [&](uint32_t b, uint32_t parity) -> bool {
    return __all_sync(0xffffffffu, ptx::mbar_wait_cluster_bounded(b, parity, abort_flag, p.timeout_ns));
  };
  auto give_up = [&]() {
    if (lane == 0) {
      raise_status(kStatusTimeout);
      *abort_flag = 1;
      ptx::st_cluster_u32(ptx::map_peer(sbase + kOffMisc + 8, rank ^ 1), 1u);
    }
  };

  if (warp == 0) {
    // ---------------------------------------------------------------- loads
    const bool leader = ptx::elect_one();
    int64_t g = 0;       // K blocks of this pair so far
    bool ok = true;
    for (int64_t i = pair; i < tiles && ok; i += pairs) {
      int tn, tt;
      tile_of(i, tiles_n, tiles_t, tn, tt);
      const int32_t nrow = tn * 2 * kM + kM * (int)rank, trow = tt * NT + C::kHalf * (int)rank;
      for (int kb = 0; kb < kblk; ++kb, ++g) {
        const int s = (int)(g % STAGES);
        if (!wait_all(bar(kEmpty + s), (uint32_t)((g / STAGES) & 1) ^ 1u)) { give_up(); ok = false; break; }
        if (leader) {
          const uint32_t sa = sbase + s * C::kStageBytes, sb = sa + kABytes;
          if (even) ptx::mbar_arrive_expect_tx(bar(kFull + s), 2 * C::kStageBytes);
          ptx::tma_load_2d_pair(sa, &tmW, lead(bar(kFull + s)), kb * kb_elems<F8>(), nrow);
          ptx::tma_load_2d_pair(sb, &tmX, lead(bar(kFull + s)), kb * kb_elems<F8>(), trow);
        }
      }
    }
    // the loads in flight land before the pair may exit (both CTAs' count on these barriers)
    if (even)
      for (int64_t i = g > STAGES ? g - STAGES : 0; i < g; ++i)
        __all_sync(0xffffffffu, ptx::mbar_wait_cluster_timed(bar(kFull + (int)(i % STAGES)),
                                                             (uint32_t)((i / STAGES) & 1), p.timeout_ns));
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issuer (even CTA)
    if (even) {
      const bool leader = ptx::elect_one();
      int64_t g = 0;
      int u = 0;         // tiles of this pair so far
      bool ok = true;
      for (int64_t i = pair; i < tiles && ok; i += pairs, ++u) {
        const int b = u & 1;
        if (!wait_all(bar(kAccFree + b), (uint32_t)((u >> 1) & 1) ^ 1u)) { give_up(); break; }
        ptx::tc_fence_after();
        for (int kb = 0; kb < kblk; ++kb, ++g) {
          const int s = (int)(g % STAGES);
          if (!wait_all(bar(kFull + s), (uint32_t)((g / STAGES) & 1))) { give_up(); ok = false; break; }
          ptx::tc_fence_after();
          const uint32_t sa = sbase + s * C::kStageBytes, sb = sa + kABytes;
          const uint64_t dA = ptx::sdesc_sw128(sa, 16, 1024), dB = ptx::sdesc_sw128(sb, 16, 1024);
          if (leader) {
#pragma unroll
            for (int kk = 0; kk < kKBytes / 32; ++kk) {
              const uint64_t o = (uint64_t)((kk * 32) >> 4);
              if (F8) ptx::umma_pair_ss_f8(tbase + b * NT, dA + o, dB + o, C::kIdesc, (kb | kk) ? 1u : 0u);
              else ptx::umma_pair_ss(tbase + b * NT, dA + o, dB + o, C::kIdesc, (kb | kk) ? 1u : 0u);
            }
            ptx::umma_commit_pair(bar(kEmpty + s), 3);
            if (kb == kblk - 1) ptx::umma_commit_pair(bar(kAccFull + b), 3);
          }
          __syncwarp();
        }
      }
    }
  } else if (warp >= 4) {
    // ---------------------------------------------------------------- epilogue
    const int q = warp - 4;          // TMEM lanes 32q ..
    int u = 0;
    for (int64_t i = pair; i < tiles; i += pairs, ++u) {
      const int b = u & 1;
      int tn, tt;
      tile_of(i, tiles_n, tiles_t, tn, tt);
      const int32_t n = tn * 2 * kM + kM * (int)rank + 32 * q + lane;
      const int64_t t0 = (int64_t)tt * NT;
      const int tokens = (int)min((int64_t)NT, p.T - t0);
      const float bias = p.bias && n < p.N ? __bfloat162float(p.bias[n]) : 0.f;
      const float ws = F8 && n < p.N ? scale_of(p.ws[n]) : 1.f;
      if (!wait_all(bar(kAccFull + b), (uint32_t)((u >> 1) & 1))) { give_up(); break; }
      ptx::tc_fence_after();
      const uint32_t trow = tbase + ((32u * q) << 16) + b * NT;
#pragma unroll 1
      for (int c = 0; c < tokens; c += 32) {
        uint32_t raw[32];
        ptx::tmem_ld_32x32b_x32(trow + c, raw);
        ptx::tmem_wait_ld();
        if (c + 32 >= tokens) {
          // this warp has read its part of the accumulator
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive_cluster_relaxed(lead(bar(kAccFree + b)));
        }
        float v[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(raw[j]);
        finish_tokens<F8, 32>(p, v, t0 + c, tokens - c, n, bias, ws);
      }
    }
  }
  __syncthreads();
  ptx::cluster_sync();   // the even CTA's MMAs, commits and loads for both CTAs are done
  if (warp == 2) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc_pair(tbase, C::kCols);
  }
  ptx::cluster_sync();
}

}  // namespace lin
}  // namespace mla
