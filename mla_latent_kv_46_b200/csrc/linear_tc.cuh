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
constexpr int kMaxSlices = 4;        // pairs of CTAs of a portable cluster

template <bool F8> __host__ __device__ constexpr int kb_elems() { return F8 ? 128 : 64; }

// mul and residual of CNT consecutive tokens of one feature, from element `at` on (one
// feature per thread; tokens past `tokens` are not read).
template <int CNT>
struct Operands {
  __nv_bfloat16 m[CNT], r[CNT];
  __device__ __forceinline__ void load(const Params& p, int64_t at, int tokens) {
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
  }
};

// Epilogue of those tokens, t0 first, of a feature below N.
template <bool F8, int CNT>
__device__ __forceinline__ void finish_tokens(const Params& p, float (&v)[CNT], const Operands<CNT>& o, int64_t at,
                                              int64_t t0, int tokens, float bias, float ws) {
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
  if (p.mul) {
#pragma unroll
    for (int j = 0; j < CNT; ++j) v[j] *= __bfloat162float(o.m[j]);
  }
  if (p.res) {
#pragma unroll
    for (int j = 0; j < CNT; ++j) v[j] += __bfloat162float(o.r[j]);
  }
#pragma unroll
  for (int j = 0; j < CNT; ++j)
    if (j < tokens) p.out[at + (int64_t)j * p.N] = __float2bfloat16_rn(v[j]);
}

__device__ __forceinline__ void unpack4(const uint2& w, float (&f)[4]) {
  f[0] = __uint_as_float(w.x << 16);
  f[1] = __uint_as_float(w.x & 0xFFFF0000u);
  f[2] = __uint_as_float(w.y << 16);
  f[3] = __uint_as_float(w.y & 0xFFFF0000u);
}

// The epilogue of `items` quads (features n .. n + 3 of one token; the thread's n is the same
// for all of its items), items tid, tid + threads, ..: token(i) is item i's token, sums(i, v)
// its fp32 sums, c the constants of the features. kQuadBatch items at a time: their mul and residual are all loaded before the
// first is used (out may be either's buffer, so the compiler may not move a load above an
// earlier item's store).
constexpr int kQuadBatch = 4;
template <bool F8>
struct QuadConstants {
  float bias[4], ws[4];
  __device__ __forceinline__ QuadConstants(const Params& p, int32_t n) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      bias[j] = p.bias && n + j < p.N ? __bfloat162float(p.bias[n + j]) : 0.f;
      ws[j] = F8 && n + j < p.N ? scale_of(p.ws[n + j]) : 1.f;
    }
  }
};
template <bool F8, class Token, class Sums>
__device__ __forceinline__ void finish_quads(const Params& p, int items, int tid, int threads, int32_t n,
                                             const QuadConstants<F8>& c, const Token& token, const Sums& sums) {
  if (n >= p.N) return;
  for (int i0 = tid; i0 < items; i0 += kQuadBatch * threads) {
    int64_t at[kQuadBatch];
    uint2 m[kQuadBatch], r[kQuadBatch];
    float xs[kQuadBatch];
#pragma unroll
    for (int b = 0; b < kQuadBatch; ++b) {
      const int i = i0 + b * threads;
      if (i < items) {
        const int64_t t = token(i);
        at[b] = t * p.N + n;
        if (F8) xs[b] = scale_of(p.xs[t]);
        if (p.quads && p.mul) m[b] = *reinterpret_cast<const uint2*>(p.mul + at[b]);
        if (p.quads && p.res) r[b] = *reinterpret_cast<const uint2*>(p.res + at[b]);
      }
    }
#pragma unroll
    for (int b = 0; b < kQuadBatch; ++b) {
      const int i = i0 + b * threads;
      if (i >= items) break;
      float v[4];
      sums(i, v);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = activate((F8 ? v[j] * c.ws[j] * xs[b] : v[j]) + c.bias[j], p.act);
      if (p.quads) {
        float f[4];
        if (p.mul) {
          unpack4(m[b], f);
#pragma unroll
          for (int j = 0; j < 4; ++j) v[j] *= f[j];
        }
        if (p.res) {
          unpack4(r[b], f);
#pragma unroll
          for (int j = 0; j < 4; ++j) v[j] += f[j];
        }
        const __nv_bfloat162 lo = __floats2bfloat162_rn(v[0], v[1]), hi = __floats2bfloat162_rn(v[2], v[3]);
        *reinterpret_cast<uint2*>(p.out + at[b]) =
            make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (n + j < p.N) {
            if (p.mul) v[j] *= __bfloat162float(p.mul[at[b] + j]);
            if (p.res) v[j] += __bfloat162float(p.res[at[b] + j]);
            p.out[at[b] + j] = __float2bfloat16_rn(v[j]);
          }
      }
    }
  }
}

__device__ __forceinline__ void prefetch_l2(const void* q) { asm volatile("prefetch.global.L2 [%0];" ::"l"(q)); }

// Asks L2 for `count` rows of `width` elements of mul and residual, from row t0 and column n0
// on (32 lanes of a warp; `w` of `warps` warps): they come from HBM under the main loop.
__device__ __forceinline__ void prefetch_rows(const Params& p, int64_t t0, int count, int32_t n0, int width, int w,
                                              int warps, int lane) {
  const int cols = min(width, p.N - n0);
  if (cols <= 0) return;
  const int lines = (cols * 2 + 127) / 128 + 1;      // 128-byte lines a row may touch
  for (int i = w * 32 + lane; i < count * lines; i += warps * 32) {
    const int64_t at = (t0 + i / lines) * p.N + n0 + min(64 * (i % lines), cols - 1);
    if (p.mul) prefetch_l2(p.mul + at);
    if (p.res) prefetch_l2(p.res + at);
  }
}

// ------------------------------------------------------------------ shared by both kernels
constexpr int kMaxStages = 12;
constexpr int kBarBytes = 256;       // barriers and two words behind the ring
constexpr int kSmemSlack = kBarBytes + 1024;
static_assert(8 * (2 * kMaxStages + 4) + 16 <= kBarBytes, "barriers");

template <bool F8> __host__ __device__ constexpr uint32_t instr_desc(int m, int n) {
  return F8 ? ptx::idesc_e4m3_f32(m, n, 0, 0) : ptx::idesc_bf16_f32(m, n, 0, 0);
}
__host__ __device__ constexpr uint32_t tmem_cols(int cols) {
  return cols <= 32 ? 32 : cols <= 64 ? 64 : cols <= 128 ? 128 : cols <= 256 ? 256 : 512;
}

// ------------------------------------------------------------------ few tokens: K slices
// grid (2 slices, feature tiles, token tiles), clusters of 2 slices CTAs: pair after pair.
// Warp 0 loads, warp 1 of the even CTA issues the MMAs, warps 3.. fetch the epilogue's operands into L2 meanwhile, and all warps
// run the epilogue. p.nt tokens a tile (a multiple of 16, at most 256), p.stages stages.
constexpr int kSplitThreads = 256;
__host__ __device__ constexpr int stage_bytes_of(int nt) { return kABytes + nt / 2 * kKBytes; }
// the ring, and in the same place the slices' sums of the CTA's own tokens (chunks of
// kChunk tokens are dealt to the CTAs of a cluster in turn)
constexpr int kChunk = 16;
__host__ __device__ constexpr int split_chunk_slots(int nt, int slices) {
  return slices * ((nt / kChunk + slices - 1) / slices);
}
__host__ __device__ constexpr int split_ring(int nt, int stages, int slices) {
  return stages * stage_bytes_of(nt) > split_chunk_slots(nt, slices) * kChunk * kM * 4
             ? stages * stage_bytes_of(nt)
             : split_chunk_slots(nt, slices) * kChunk * kM * 4;
}
__host__ __device__ constexpr int split_smem(int nt, int stages, int slices) {
  return split_ring(nt, stages, slices) + kSmemSlack;
}

template <bool F8>
__global__ void __launch_bounds__(kSplitThreads) linear_split_kernel(const __grid_constant__ CUtensorMap tmW,
                                                                     const __grid_constant__ CUtensorMap tmX,
                                                                     const Params p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = ptx::smem_u32(smem);
  const int nt = p.nt, stages = p.stages;
  const uint32_t stage_bytes = (uint32_t)stage_bytes_of(nt);
  const int slices = gridDim.x / 2, slice = blockIdx.x / 2;
  const uint32_t r = blockIdx.x & 1;      // CTA of its pair; cluster rank 2 slice + r
  const bool even = r == 0;
  const int off_bar = split_ring(nt, stages, slices);
  // barriers: full (even CTA: both CTAs' loads), empty and done (each CTA)
  auto bar = [&](int i) { return sbase + off_bar + 8u * i; };
  const int kFull = 0, kEmpty = stages, kDone = 2 * stages, off_misc = off_bar + 8 * (2 * stages + 2);
  auto lead = [&](uint32_t a) { return ptx::map_peer(a, 2 * slice); };
  const uint16_t both = (uint16_t)(3u << (2 * slice));
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + off_misc + 8);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int n0 = blockIdx.y * 2 * kM + kM * (int)r;
  const int64_t t0 = (int64_t)blockIdx.z * nt;
  const int kblk = (p.K + kb_elems<F8>() - 1) / kb_elems<F8>();
  const int kb0 = (int)((int64_t)kblk * slice / slices), kb1 = (int)((int64_t)kblk * (slice + 1) / slices);
  const int nkb = kb1 - kb0;      // at least one: the host cuts no more slices than K blocks

  if (tid == 0) {
    *abort_flag = 0;
    for (int s = 0; s < stages; ++s) {
      ptx::mbar_init(bar(kFull + s), 1);
      ptx::mbar_init(bar(kEmpty + s), 1);
    }
    ptx::mbar_init(bar(kDone), 1);
    ptx::fence_mbar_init();
    ptx::prefetch_tmap(&tmW);
    ptx::prefetch_tmap(&tmX);
  }
  if (warp == 2) {
    ptx::tmem_alloc_pair(sbase + off_misc, tmem_cols(nt));
    ptx::tmem_relinquish_pair();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::cluster_sync();   // the pair's barriers exist before anyone loads or issues
  ptx::tc_fence_after();
  const uint32_t tbase = *reinterpret_cast<volatile uint32_t*>(smem + off_misc);
  ptx::grid_launch_next();
  ptx::grid_wait();      // from here on this kernel reads and writes global memory
  auto wait_all = [&](uint32_t b, uint32_t parity) -> bool {
    return __all_sync(0xffffffffu, ptx::mbar_wait_cluster_bounded(b, parity, abort_flag, p.timeout_ns));
  };
  auto give_up = [&]() {
    if (lane == 0) {
      raise_status(kStatusTimeout);
      *abort_flag = 1;
      ptx::st_cluster_u32(ptx::map_peer(sbase + off_misc + 8, (2 * slice + r) ^ 1), 1u);
    }
  };
  bool ok = true;

  if (warp == 0) {
    // ---------------------------------------------------------------- loads
    const bool leader = ptx::elect_one();
    const int32_t trow = (int32_t)t0 + nt / 2 * (int)r;
    // with one token tile W is read once and by this pair alone: it should not push the
    // epilogue's operands, fetched early, out of L2
    const uint64_t w_policy = gridDim.z == 1 ? ptx::policy_evict_first() : ptx::policy_evict_normal();
    int s = 0, issued = 0;
    uint32_t parity = 1;
    for (int i = 0; i < nkb; ++i) {
      if (!wait_all(bar(kEmpty + s), parity)) { give_up(); ok = false; break; }
      if (leader) {
        const uint32_t sa = sbase + s * stage_bytes, sb = sa + kABytes;
        if (even) ptx::mbar_arrive_expect_tx(bar(kFull + s), 2 * stage_bytes);
        ptx::tma_load_2d_pair_hint(sa, &tmW, lead(bar(kFull + s)), (kb0 + i) * kb_elems<F8>(), n0, w_policy);
        ptx::tma_load_2d_pair(sb, &tmX, lead(bar(kFull + s)), (kb0 + i) * kb_elems<F8>(), trow);
      }
      issued = i + 1;
      if (++s == stages) {
        s = 0;
        parity ^= 1;
      }
    }
    // the loads in flight land before the pair may exit (both CTAs' count on these barriers)
    if (even)
      for (int i = issued > stages ? issued - stages : 0; i < issued; ++i)
        __all_sync(0xffffffffu, ptx::mbar_wait_cluster_timed(bar(kFull + i % stages), (i / stages) & 1, p.timeout_ns));
  } else if (warp == 1 && even) {
    // ---------------------------------------------------------------- MMA issuer
    const bool leader = ptx::elect_one();
    const uint32_t idesc = instr_desc<F8>(2 * kM, nt);
    int s = 0;
    uint32_t parity = 0;
    for (int i = 0; i < nkb; ++i) {
      if (!wait_all(bar(kFull + s), parity)) { give_up(); ok = false; break; }
      ptx::tc_fence_after();
      const uint32_t sa = sbase + s * stage_bytes, sb = sa + kABytes;
      const uint64_t dA = ptx::sdesc_sw128(sa, 16, 1024), dB = ptx::sdesc_sw128(sb, 16, 1024);
      if (leader) {
#pragma unroll
        for (int kk = 0; kk < kKBytes / 32; ++kk) {
          const uint64_t o = (uint64_t)((kk * 32) >> 4);
          if (F8) ptx::umma_pair_ss_f8(tbase, dA + o, dB + o, idesc, (i | kk) ? 1u : 0u);
          else ptx::umma_pair_ss(tbase, dA + o, dB + o, idesc, (i | kk) ? 1u : 0u);
        }
        ptx::umma_commit_pair(bar(kEmpty + s), both);
        if (i == nkb - 1) ptx::umma_commit_pair(bar(kDone), both);
      }
      __syncwarp();
      if (++s == stages) {
        s = 0;
        parity ^= 1;
      }
    }
  }

  // ---------------------------------------------------------------- epilogue (all warps)
  const int tokens = (int)min((int64_t)nt, p.T - t0);
  if (warp >= 3 && (p.mul || p.res) && slice == 0)
    prefetch_rows(p, t0, tokens, n0, kM, warp - 3, kSplitThreads / 32 - 3, lane);
  if (F8 && warp == 2 && lane <= tokens / 128) prefetch_l2(p.xs + t0 + min(128 * lane, tokens - 1));
  const int32_t n = n0 + 4 * (tid % (kM / 4));
  const QuadConstants<F8> constants(p, n);
  const bool done = ok && wait_all(bar(kDone), 0);
  if (!done) give_up();
  ptx::tc_fence_after();
  // Chunk c of the tokens is finished by CTA c % slices: every CTA stores its sums straight
  // from TMEM into that CTA's shared memory, [slice][c / slices][token][feature]. Remote
  // stores need no answer; reading the peers' sums instead, a round trip per four tokens,
  // took ~10 us more at T = 128 (five slices). The stages they land in are free once every
  // CTA of the cluster has passed its done barrier.
  __syncthreads();
  if (slices > 1) ptx::cluster_sync();
  const int chunks = (tokens + kChunk - 1) / kChunk, per = (chunks + slices - 1) / slices;
  if (done) {
    // warps w and w + 4 reach the same TMEM lanes and take every other chunk
    const int feat = tid % kM;
    const uint32_t trow = tbase + ((32u * (warp % 4)) << 16);
#pragma unroll 1
    for (int c = warp / 4; c < chunks; c += kSplitThreads / 128) {
      float v[kChunk];
      ptx::tmem_ld_32x32b_x16(trow + kChunk * c, v);
      ptx::tmem_wait_ld();
      const uint32_t at =
          ptx::map_peer(sbase + 4u * ((slice * per + c / slices) * (kChunk * kM) + feat), 2 * (c % slices) + r);
#pragma unroll
      for (int j = 0; j < kChunk; ++j)
        if (kChunk * c + j < tokens) ptx::st_cluster_u32(at + 4u * j * kM, __float_as_uint(v[j]));
    }
  }
  __syncthreads();
  if (slices > 1) ptx::cluster_sync();   // every slice's sums are here; nothing remote is touched from now on
  if (done && slice < chunks) {
    // four neighbouring features of a token per thread, added in slice order
    const float4* part = reinterpret_cast<const float4*>(smem);
    constexpr int kQuads = kM / 4, kItems = kChunk * kQuads;
    // this CTA's tokens: whole chunks, but for the last of all
    const int mine = (chunks - slice + slices - 1) / slices;
    const bool has_last = (chunks - 1) % slices == slice;
    const int items = mine * kItems - (has_last ? (chunks * kChunk - tokens) * kQuads : 0);
    finish_quads<F8>(
        p, items, tid, kSplitThreads, n, constants,
        [&](int i) { return t0 + (int64_t)(i / kItems * slices + slice) * kChunk + i % kItems / kQuads; },
        [&](int i, float (&v)[4]) {
          v[0] = v[1] = v[2] = v[3] = 0.f;
#pragma unroll
          for (int s = 0; s < kMaxSlices; ++s)
            if (s < slices) {
              const float4 w = part[s * per * kItems + i];
              v[0] += w.x;
              v[1] += w.y;
              v[2] += w.z;
              v[3] += w.w;
            }
        });
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::cluster_sync();   // the even CTAs' MMAs, commits and loads for both CTAs are done
  if (warp == 2) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc_pair(tbase, tmem_cols(nt));
  }
  ptx::cluster_sync();
}

// ------------------------------------------------------------------ many tokens: SM pairs
// p.nt tokens a tile (a multiple of 16, at most 256; two accumulators in TMEM), p.stages
// stages. Warp 0 loads, warp 1 issues the MMAs (even CTA), warps 2 and 3 fetch the epilogue's
// operands into L2, warps 4.. run the epilogue (two per 32 TMEM lanes, on alternate chunks).
constexpr int kEpiWarps = 8;
constexpr int kPairThreads = 32 * (4 + kEpiWarps);
__host__ __device__ constexpr int pair_smem(int nt, int stages) { return stages * stage_bytes_of(nt) + kSmemSlack; }

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

template <bool F8>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
linear_pair_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX, const Params p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = ptx::smem_u32(smem);
  // barriers: full (even CTA: both CTAs' loads), empty (each CTA), accumulator full (each
  // CTA), accumulator free (even CTA: both CTAs' epilogue warps)
  const int nt = p.nt, stages = p.stages;
  const uint32_t stage_bytes = (uint32_t)stage_bytes_of(nt);
  const int off_bar = stages * (int)stage_bytes, kOffMisc = off_bar + 8 * (2 * stages + 4);
  auto bar = [&](int i) { return sbase + off_bar + 8u * i; };
  const int kFull = 0, kEmpty = stages, kAccFull = 2 * stages, kAccFree = 2 * stages + 2;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kOffMisc + 8);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = ptx::cluster_rank();
  const bool even = rank == 0;
  auto lead = [&](uint32_t a) { return ptx::map_peer(a, 0); };
  const int tiles_n = (p.N + 2 * kM - 1) / (2 * kM), tiles_t = (int)(((int64_t)p.T + nt - 1) / nt);
  const int64_t tiles = (int64_t)tiles_n * tiles_t;
  const int pairs = gridDim.x / 2, pair = blockIdx.x / 2;
  const int kblk = (p.K + kb_elems<F8>() - 1) / kb_elems<F8>();

  if (tid == 0) {
    *abort_flag = 0;
    for (int s = 0; s < stages; ++s) {
      ptx::mbar_init(bar(kFull + s), 1);
      ptx::mbar_init(bar(kEmpty + s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      ptx::mbar_init(bar(kAccFull + b), 1);
      ptx::mbar_init(bar(kAccFree + b), 2 * kEpiWarps);
    }
    ptx::fence_mbar_init();
    ptx::prefetch_tmap(&tmW);
    ptx::prefetch_tmap(&tmX);
  }
  const uint32_t cols = tmem_cols(2 * nt);
  if (warp == 2) {
    ptx::tmem_alloc_pair(sbase + kOffMisc, cols);
    ptx::tmem_relinquish_pair();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::cluster_sync();   // both CTAs' barriers exist before anyone arrives, loads or issues
  ptx::tc_fence_after();
  const uint32_t tbase = *reinterpret_cast<volatile uint32_t*>(smem + kOffMisc);
  ptx::grid_launch_next();
  ptx::grid_wait();      // from here on this kernel reads and writes global memory
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
    int s = 0;
    uint32_t parity = 1;
    bool ok = true;
    for (int64_t i = pair; i < tiles && ok; i += pairs) {
      int tn, tt;
      tile_of(i, tiles_n, tiles_t, tn, tt);
      const int32_t nrow = tn * 2 * kM + kM * (int)rank, trow = tt * nt + nt / 2 * (int)rank;
      for (int kb = 0; kb < kblk; ++kb, ++g) {
        if (!wait_all(bar(kEmpty + s), parity)) { give_up(); ok = false; break; }
        if (leader) {
          const uint32_t sa = sbase + s * stage_bytes, sb = sa + kABytes;
          if (even) ptx::mbar_arrive_expect_tx(bar(kFull + s), 2 * stage_bytes);
          ptx::tma_load_2d_pair(sa, &tmW, lead(bar(kFull + s)), kb * kb_elems<F8>(), nrow);
          ptx::tma_load_2d_pair(sb, &tmX, lead(bar(kFull + s)), kb * kb_elems<F8>(), trow);
        }
        if (++s == stages) {
          s = 0;
          parity ^= 1;
        }
      }
    }
    // the loads in flight land before the pair may exit (both CTAs' count on these barriers)
    if (even)
      for (int64_t i = g > stages ? g - stages : 0; i < g; ++i)
        __all_sync(0xffffffffu, ptx::mbar_wait_cluster_timed(bar(kFull + (int)(i % stages)),
                                                             (uint32_t)((i / stages) & 1), p.timeout_ns));
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issuer (even CTA)
    if (even) {
      const bool leader = ptx::elect_one();
      const uint32_t idesc = instr_desc<F8>(2 * kM, nt);
      int s = 0, u = 0;  // u: tiles of this pair so far
      uint32_t parity = 0;
      bool ok = true;
      for (int64_t i = pair; i < tiles && ok; i += pairs, ++u) {
        const int b = u & 1;
        if (!wait_all(bar(kAccFree + b), (uint32_t)((u >> 1) & 1) ^ 1u)) { give_up(); break; }
        ptx::tc_fence_after();
        for (int kb = 0; kb < kblk; ++kb) {
          if (!wait_all(bar(kFull + s), parity)) { give_up(); ok = false; break; }
          ptx::tc_fence_after();
          const uint32_t sa = sbase + s * stage_bytes, sb = sa + kABytes;
          const uint64_t dA = ptx::sdesc_sw128(sa, 16, 1024), dB = ptx::sdesc_sw128(sb, 16, 1024);
          if (leader) {
#pragma unroll
            for (int kk = 0; kk < kKBytes / 32; ++kk) {
              const uint64_t o = (uint64_t)((kk * 32) >> 4);
              if (F8) ptx::umma_pair_ss_f8(tbase + b * nt, dA + o, dB + o, idesc, (kb | kk) ? 1u : 0u);
              else ptx::umma_pair_ss(tbase + b * nt, dA + o, dB + o, idesc, (kb | kk) ? 1u : 0u);
            }
            ptx::umma_commit_pair(bar(kEmpty + s), 3);
            if (kb == kblk - 1) ptx::umma_commit_pair(bar(kAccFull + b), 3);
          }
          __syncwarp();
          if (++s == stages) {
            s = 0;
            parity ^= 1;
          }
        }
      }
    }
  } else if (warp < 4) {
    // ---------------------------------------------------------------- the epilogue's operands into L2
    if (p.mul || p.res) {
      int u = 0;
      for (int64_t i = pair; i < tiles; i += pairs, ++u) {
        // a tile's own main loop is the time to fetch its operands: wait for the one before it
        if (u > 0 && !wait_all(bar(kAccFull + ((u - 1) & 1)), (uint32_t)(((u - 1) >> 1) & 1))) break;
        int tn, tt;
        tile_of(i, tiles_n, tiles_t, tn, tt);
        const int64_t t0 = (int64_t)tt * nt;
        prefetch_rows(p, t0, (int)min((int64_t)nt, p.T - t0), tn * 2 * kM + kM * (int)rank, kM, warp - 2, 2, lane);
      }
    }
  } else {
    // ---------------------------------------------------------------- epilogue
    const int q = warp % 4, half = (warp - 4) / 4;          // TMEM lanes 32q ..
    int u = 0;
    for (int64_t i = pair; i < tiles; i += pairs, ++u) {
      const int b = u & 1;
      int tn, tt;
      tile_of(i, tiles_n, tiles_t, tn, tt);
      const int32_t n = tn * 2 * kM + kM * (int)rank + 32 * q + lane;
      const int64_t t0 = (int64_t)tt * nt;
      const int tokens = (int)min((int64_t)nt, p.T - t0);
      const float bias = p.bias && n < p.N ? __bfloat162float(p.bias[n]) : 0.f;
      const float ws = F8 && n < p.N ? scale_of(p.ws[n]) : 1.f;
      // a chunk's operands are loaded before the chunk before it is finished
      const int64_t at = t0 * p.N + n;
      Operands<kChunk> ops, next;
      int c = kChunk * half;
      if (c < tokens && n < p.N) ops.load(p, at + (int64_t)c * p.N, tokens - c);
      if (!wait_all(bar(kAccFull + b), (uint32_t)((u >> 1) & 1))) { give_up(); break; }
      ptx::tc_fence_after();
      const uint32_t trow = tbase + ((32u * q) << 16) + b * nt;
#pragma unroll 1
      for (; c < tokens; c += 2 * kChunk) {
        float v[kChunk];
        ptx::tmem_ld_32x32b_x16(trow + c, v);
        const int after = c + 2 * kChunk;
        if (after < tokens && n < p.N) next.load(p, at + (int64_t)after * p.N, tokens - after);
        ptx::tmem_wait_ld();
        if (n < p.N) finish_tokens<F8, kChunk>(p, v, ops, at + (int64_t)c * p.N, t0 + c, tokens - c, bias, ws);
        ops = next;
        __syncwarp();
      }
      // this warp has read its part of the accumulator
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive_cluster_relaxed(lead(bar(kAccFree + b)));
    }
  }
  __syncthreads();
  ptx::cluster_sync();   // the even CTA's MMAs, commits and loads for both CTAs are done
  if (warp == 2) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc_pair(tbase, cols);
  }
  ptx::cluster_sync();
}

}  // namespace lin
}  // namespace mla
