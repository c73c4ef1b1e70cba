// linear_tc.cuh -- the layer's projections on sm_100a tensor cores.
//
//   out[t][n] = residual + mul * act(sum_k x[t][k] W[n][k] + bias[n])
//
// Both kernels compute the transposed product D[n][t]: W's rows are the MMA's M side, the
// tokens its N side. One token then still fills the M side, so a decode step's
// few tokens cost no idle rows, only the 16-token minimum of the N side; and a thread of the
// epilogue owns one feature (its TMEM lane), so a warp's store of one token covers 32
// neighbouring features. x and W are both K-major: TMA streams 128-byte-wide K blocks (64
// bf16 or 128 E4M3 elements, 128-byte swizzle) and one elected lane issues the MMAs, fp32 in
// TMEM. Rows and columns past T, N and K arrive as zeros and are not stored.
//
// Both run on pairs of CTAs (tcgen05 cta_group::2): 256 features x nt tokens a tile, each CTA
// loading its 128 rows of W and half of the tokens' rows of x, which halves what an SM takes in
// of x. nt is chosen per call.
//
// linear_split_kernel (few tokens): bound by the bytes of W. One pair per tile and K slice; the
// slices of a tile are a cluster, which adds its fp32 partial sums through distributed shared
// memory in slice order. One launch, no workspace, and the same sum in every run. (128 x 7168 x
// 16384 bf16 with a residual: 45 us in a short run, 49 in a long one, against 36 for W's bytes; 8
// bits: 31 against 18.)
//
// linear_pair_kernel (many tokens): bound by the tensor cores. Persistent pairs, with two
// accumulators in TMEM so that a tile's epilogue runs under the next tile's main loop (16384 x
// 8192 x 7168 bf16: 1.24 ms, 1.56 PFLOP/s, in a short run; 1.45 ms under the power cap). It also
// serves few tokens where there are feature tiles for most pairs and one wave of them streams W
// as fast as slices would (one token, 16384 x 7168: 38 us, 8 bits 21, against 36 and 18).
#pragma once

#include "common.cuh"
#include "linear.cuh"
#include "ptx.cuh"

namespace mla {
namespace lin {

constexpr int kM = 128;              // features (MMA rows) per CTA
constexpr int kKBytes = 128;         // bytes of a K block of one row
constexpr int kABytes = kM * kKBytes;
constexpr int kMaxSlices = 8;        // pairs of CTAs of the largest cluster

template <bool F8> __host__ __device__ constexpr int kb_elems() { return F8 ? 128 : 64; }

// mul and residual of CNT consecutive tokens of one feature, from element `at` on (one
// feature per thread; tokens past `tokens` are not read).
template <int CNT>
struct Operands {
  __nv_bfloat16 m[CNT], r[CNT];
  __device__ __forceinline__ void load(const Params& p, int64_t at, int tokens) {
    if (p.mul) column(m, p.mul + at, p.N, tokens);
    if (p.res) column(r, p.res + at, p.N, tokens);
  }
  static __device__ __forceinline__ void column(__nv_bfloat16 (&v)[CNT], const __nv_bfloat16* q, int32_t N, int tokens) {
    if (tokens >= CNT) {
#pragma unroll
      for (int j = 0; j < CNT; ++j, q += N) v[j] = *q;
    } else {
#pragma unroll
      for (int j = 0; j < CNT; ++j, q += N)
        if (j < tokens) v[j] = *q;
    }
  }
};

// Epilogue of those tokens for a feature below N; ws, sx: the feature's and the tokens' scales
// (8-bit operands). Two tokens' results are converted at once, and a whole chunk is stored
// without a test per token: single conversions and the tests were most of this function's time.
template <bool F8, int CNT>
__device__ __forceinline__ void finish_tokens(const Params& p, float (&v)[CNT], const Operands<CNT>& o, int64_t at,
                                              int tokens, float bias, float ws, const float (&sx)[CNT]) {
  if (F8) {
#pragma unroll
    for (int j = 0; j < CNT; ++j) v[j] = v[j] * ws * sx[j];
  }
#pragma unroll
  for (int j = 0; j < CNT; ++j) v[j] += bias;
  activate(v, p.act);
  if (p.mul) {
#pragma unroll
    for (int j = 0; j < CNT; ++j) v[j] *= __bfloat162float(o.m[j]);
  }
  if (p.res) {
#pragma unroll
    for (int j = 0; j < CNT; ++j) v[j] += __bfloat162float(o.r[j]);
  }
  __nv_bfloat16* out = p.out + at;
  __nv_bfloat162 two[CNT / 2];
#pragma unroll
  for (int j = 0; j < CNT / 2; ++j) two[j] = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
  if (tokens >= CNT) {
#pragma unroll
    for (int j = 0; j < CNT; ++j, out += p.N) *out = j % 2 ? two[j / 2].y : two[j / 2].x;
  } else {
#pragma unroll
    for (int j = 0; j < CNT; ++j, out += p.N)
      if (j < tokens) *out = j % 2 ? two[j / 2].y : two[j / 2].x;
  }
}

// Where N and every pointer allow it (p.octs), the few-token kernel's epilogue, whose sums lie
// in shared memory, moves eight neighbouring features of one token at a time, 16 bytes.
template <bool F8>
struct OctConstants {   // as they lie in memory: unpacked where they are used
  uint4 bias;
  uint2 ws;
  __device__ __forceinline__ void load(const Params& p, int32_t n) {
    bias = make_uint4(0, 0, 0, 0);
    if (p.bias && n < p.N) bias = *reinterpret_cast<const uint4*>(p.bias + n);
    if (F8 && n < p.N) ws = *reinterpret_cast<const uint2*>(p.ws + n);
  }
};
template <bool F8>
__device__ __forceinline__ void finish_oct(const Params& p, float (&v)[8], const uint4& mul, const uint4& res, float xs,
                                           const OctConstants<F8>& c, int64_t at) {
  float f[8];
  if (F8) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = v[j] * scale_of((uint8_t)((j < 4 ? c.ws.x : c.ws.y) >> (8 * (j % 4)))) * xs;
  }
  if (p.bias) {
    f8::unpack8(c.bias, f);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] += f[j];
  }
  activate(v, p.act);
  if (p.mul) {
    f8::unpack8(mul, f);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] *= f[j];
  }
  if (p.res) {
    f8::unpack8(res, f);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] += f[j];
  }
  uint32_t o[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
    o[j] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p.out + at) = make_uint4(o[0], o[1], o[2], o[3]);
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

// Two bf16 values.
__device__ __forceinline__ ptx::F2 halves(uint32_t two) {
  return ptx::f2(__uint_as_float(two << 16), __uint_as_float(two & 0xFFFF0000u));
}

// ------------------------------------------------------------------ shared by both kernels
constexpr int kMaxStages = 12;
// How long a kernel that gave up waits for its own copies and MMAs in flight, which land
// within microseconds, however short the caller's bound on waits is.
__device__ __forceinline__ uint64_t drain_ns(const Params& p) {
  return p.timeout_ns > 10000000ull ? p.timeout_ns : 10000000ull;
}
constexpr uint64_t kSettleNs = 100000;
// The even CTA's loader: the last `stages` armed phases of the full barriers complete (both
// CTAs' loads), or, if the peer gave up before its share, time out once.
template <class Bar>
__device__ __forceinline__ void drain_loads(int64_t armed, int stages, const Bar& full, uint64_t ns) {
  for (int64_t i = armed > stages ? armed - stages : 0; i < armed; ++i)
    if (!__all_sync(0xffffffffu, ptx::mbar_wait_cluster_timed(full((int)(i % stages)), (uint32_t)((i / stages) & 1), ns)))
      break;
}
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
// Warp 0 loads, warp 1 of the even CTA issues the MMAs, warps 3.. fetch the epilogue's
// operands into L2 meanwhile, and all warps run the epilogue. p.nt tokens a tile (a multiple of 16, at most 256), p.stages stages.
constexpr int kSplitThreads = 256;
__host__ __device__ constexpr int stage_bytes_of(int nt) { return kABytes + nt / 2 * kKBytes; }
// the ring, and in the same place the slices' sums of the CTA's own tokens (chunks of
// kChunk tokens are dealt to the pairs of a cluster in turn)
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
__global__ void __launch_bounds__(kSplitThreads, 2) linear_split_kernel(const __grid_constant__ CUtensorMap tmW,
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
  // barriers: full (even CTA: both CTAs' loads), empty and done (each CTA), drain (even CTA)
  auto bar = [&](int i) { return sbase + off_bar + 8u * i; };
  const int kFull = 0, kEmpty = stages, kDone = 2 * stages, kDrain = 2 * stages + 1;
  const int off_misc = off_bar + 8 * (2 * stages + 2);
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
    ptx::mbar_init(bar(kDrain), 1);
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
    if (even) drain_loads(issued, stages, [&](int s) { return bar(kFull + s); }, drain_ns(p));
    if (!ok) ptx::delay_ns(kSettleNs);
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
    if (!ok) {      // the MMAs issued so far end before the pair's memory goes
      if (leader) ptx::umma_commit_pair(bar(kDrain), (uint16_t)(1u << (2 * slice)));
      __all_sync(0xffffffffu, ptx::mbar_wait_cluster_timed(bar(kDrain), 0, drain_ns(p)));
    }
  }

  // ---------------------------------------------------------------- epilogue (all warps)
  const int tokens = (int)min((int64_t)nt, p.T - t0);
  if (warp >= 3 && (p.mul || p.res) && slice == 0)
    prefetch_rows(p, t0, tokens, n0, kM, warp - 3, kSplitThreads / 32 - 3, lane);
  if (F8 && warp == 2 && lane <= tokens / 128) prefetch_l2(p.xs + t0 + min(128 * lane, tokens - 1));
  // this thread's features in the last step: eight, or one
  constexpr int kOcts = kM / 8;
  const int32_t n = p.octs ? n0 + 8 * (tid % kOcts) : n0 + tid % kM;
  OctConstants<F8> constants;
  float bias = 0.f, ws = 1.f;
  if (p.octs) {
    constants.load(p, n);
  } else if (n < p.N) {
    if (p.bias) bias = __bfloat162float(p.bias[n]);
    if (F8) ws = scale_of(p.ws[n]);
  }
  const bool done = ok && wait_all(bar(kDone), 0);
  if (!done) give_up();
  ptx::tc_fence_after();
  // Chunk c of the tokens is finished by pair c % slices: every CTA stores its sums straight
  // from TMEM into the shared memory of that pair's CTA for the same features, [slice][c / slices][token][feature]. Remote
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
  // Every slice's sums are here, no MMA, commit or load of the pair is under way and TMEM is
  // read: it is given back, and nothing remote is touched from now on but by that. The last
  // barrier's arrival is here, so that its wait, after the last step, has nothing to wait for.
  ptx::tc_fence_before();
  __syncthreads();
  ptx::cluster_sync();
  if (warp == 2) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc_pair(tbase, tmem_cols(nt));
  }
  __syncwarp();
  ptx::cluster_arrive();
  if (done && slice < chunks && n < p.N && p.octs) {
    // the slices' sums added in their order, for this CTA's tokens: whole chunks, but for the
    // last of all
    const float* part = reinterpret_cast<const float*>(smem);
    const int stride = per * kChunk * kM;       // from one slice's sums to the next's
    const int mine = (chunks - slice + slices - 1) / slices;
    const int held = mine * kChunk - ((chunks - 1) % slices == slice ? chunks * kChunk - tokens : 0);
    auto token_of = [&](int i) { return t0 + (int64_t)(i / kChunk * slices + slice) * kChunk + i % kChunk; };
    constexpr int kBatch = 4;   // tokens whose operands are loaded before the first is finished: out may
                                // be mul's or residual's buffer, so no load moves above an earlier store
    constexpr int kStep = kSplitThreads / kOcts;
    for (int i0 = tid / kOcts; i0 < held; i0 += kBatch * kStep) {
      uint4 m[kBatch], r[kBatch];
      float xs[kBatch];
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int i = i0 + b * kStep;
        if (i < held) {
          const int64_t t = token_of(i), at = t * p.N + n;
          if (F8) xs[b] = scale_of(p.xs[t]);
          if (p.mul) m[b] = *reinterpret_cast<const uint4*>(p.mul + at);
          if (p.res) r[b] = *reinterpret_cast<const uint4*>(p.res + at);
        }
      }
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int i = i0 + b * kStep;
        if (i < held) {
          float v[8] = {};
#pragma unroll
          for (int s = 0; s < kMaxSlices; ++s)
            if (s < slices) {
              const float4* w = reinterpret_cast<const float4*>(part + s * stride + i * kM + 8 * (tid % kOcts));
              const float4 lo = w[0], hi = w[1];
              v[0] += lo.x;
              v[1] += lo.y;
              v[2] += lo.z;
              v[3] += lo.w;
              v[4] += hi.x;
              v[5] += hi.y;
              v[6] += hi.z;
              v[7] += hi.w;
            }
          finish_oct<F8>(p, v, m[b], r[b], xs[b], constants, token_of(i) * p.N + n);
        }
      }
    }
  }
  if (done && slice < chunks && !p.octs) {
    // one feature and a chunk of tokens per thread, a chunk's operands all in flight at once
    const float* part = reinterpret_cast<const float*>(smem);
    for (int k = tid / kM; slice + k * slices < chunks; k += kSplitThreads / kM) {
      const int64_t t = t0 + (int64_t)(slice + k * slices) * kChunk;
      const int left = (int)min((int64_t)kChunk, t0 + tokens - t);
      const int64_t at = t * p.N + n;
      Operands<kChunk> ops;
      if (n < p.N) ops.load(p, at, left);
      float sx[kChunk];
      if (F8) {
        const float mine = lane < left ? scale_of(p.xs[t + lane]) : 0.f;
#pragma unroll
        for (int j = 0; j < kChunk; ++j) sx[j] = __shfl_sync(0xffffffffu, mine, j);
      }
      float v[kChunk] = {};
      for (int s = 0; s < slices; ++s)
#pragma unroll
        for (int j = 0; j < kChunk; ++j) v[j] += part[((s * per + k) * kChunk + j) * kM + tid % kM];
      if (n < p.N) finish_tokens<F8, kChunk>(p, v, ops, at, left, bias, ws, sx);
    }
  }
  __syncwarp();
  ptx::cluster_wait();
}

// ------------------------------------------------------------------ many tokens: SM pairs
// p.nt tokens a tile (a multiple of 16, at most 256; two accumulators in TMEM), p.stages
// stages. Warp 0 loads, warp 1 issues the MMAs (even CTA), warp 2 holds TMEM, warps 4.. run the
// epilogue. Where K is short (below ~1000 for a bare output, ~2000 with a gate and a residual, more for
// gelu) the epilogue is what a tile takes: its instructions and its few warps' latencies
// count. Two forms:
//   WIDE, where N and the pointers let rows move in 16-byte parts: sixteen warps, each 32
//   features and every fourth piece of 8 tokens. The sums are read in the matrix fragment's shape
//   (16 lanes x 256 bits), two tokens of a feature side by side, so that paired fp32 instructions
//   serve both and the transposing matrix store turns them into rows of shared memory; mul and
//   residual come the other way, by the thread's asynchronous copies and the transposing matrix
//   load.
//   otherwise: eight warps, two per 32 TMEM lanes on alternate chunks of 16 tokens, a feature a
//   lane: every access is 2 bytes a lane, 64 a warp and token, at any alignment.
// (8192 x 8192 x 64 bf16, us, otherwise -> WIDE: bare 64 -> 41, with a residual 95 -> 72, with residual
// and sigmoid 107 -> 79, gelu 143 -> 96, all of it and gelu 188 -> 132. Of that the wide accesses
// with eight warps gave 49 / 86 / 102 / 123 / 162. 12 and 20 warps were slower, and so was asking
// L2 for the next tile's operands, which the narrow form wants: 8192 x 8192 x 1024 with residual
// and sigmoid 114 against 102. Eight slots a warp for one stage of the ring less: 67 us with a
// residual, but 92 against 88 at K = 1024 bare.)
__host__ __device__ constexpr int epi_warps(bool wide) { return wide ? 16 : 8; }
__host__ __device__ constexpr int pair_threads(bool wide) { return 32 * (4 + epi_warps(wide)); }
// Behind the ring, per epilogue warp: its tile's token scales (8-bit operands); in the WIDE kernel
// kSlots places for an 8 token x 32 feature piece of mul, residual or the results.
constexpr int kOctTokens = 8, kSlotBytes = kOctTokens * 32 * 2, kSlots = 4;
__host__ __device__ constexpr int epi_bytes(bool wide) { return epi_warps(wide) * (wide ? kSlots * kSlotBytes : 256 * 4); }
__host__ __device__ constexpr int pair_smem(int nt, int stages, bool wide) {
  return stages * stage_bytes_of(nt) + epi_bytes(wide) + kSmemSlack;
}
static_assert(8 * (2 * kMaxStages + 5) + 16 <= kBarBytes, "barriers");

// Token tiles that share a sweep over the feature tiles (16384 x 8192 x 7168 bf16: 1.27 ms; 4, 16 and
// 32 give 1.30, 1.31 and 1.39).
constexpr int kGroupT = 8;

// Tile `i` of tiles_n x tiles_t: groups of kGroupT token tiles, within a group the token
// tile fastest, so the pairs at work at one time share feature and token tiles in L2.
// (32-bit division: 64-bit ones took a microsecond a tile.)
struct TileAt {
  int tn, tt;
};
__device__ __forceinline__ TileAt tile_of(uint32_t i, uint32_t tiles_n, uint32_t tiles_t) {
  const uint32_t per = kGroupT * tiles_n, g = i / per, rem = i - g * per;
  const uint32_t first = g * kGroupT, width = min((uint32_t)kGroupT, tiles_t - first);
  return TileAt{(int)(rem / width), (int)(first + rem % width)};
}

template <bool F8, bool WIDE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(pair_threads(WIDE), 1)
linear_pair_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX, const Params p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = ptx::smem_u32(smem);
  // barriers: full (even CTA: both CTAs' loads), empty (each CTA), accumulator full (each
  // CTA), accumulator free (even CTA: both CTAs' epilogue warps)
  const int nt = p.nt, stages = p.stages;
  const uint32_t stage_bytes = (uint32_t)stage_bytes_of(nt);
  const int off_epi = stages * (int)stage_bytes, off_bar = off_epi + epi_bytes(WIDE);
  constexpr int kEpiWarps = epi_warps(WIDE), kEpiSets = kEpiWarps / 4;
  auto bar = [&](int i) { return sbase + off_bar + 8u * i; };
  const int kFull = 0, kEmpty = stages, kAccFull = 2 * stages, kAccFree = 2 * stages + 2;
  const int kDrain = 2 * stages + 4, kOffMisc = off_bar + 8 * (kDrain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kOffMisc + 8);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = ptx::cluster_rank();
  const bool even = rank == 0;
  auto lead = [&](uint32_t a) { return ptx::map_peer(a, 0); };
  const int tiles_n = (p.N + 2 * kM - 1) / (2 * kM), tiles_t = (int)(((int64_t)p.T + nt - 1) / nt);
  const int tiles = tiles_n * tiles_t;      // below 2^31 - pairs: the host checks
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
    ptx::mbar_init(bar(kDrain), 1);
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
    const uint64_t w_policy = tiles_t == 1 ? ptx::policy_evict_first() : ptx::policy_evict_normal();   // as above
    int64_t g = 0;       // K blocks of this pair so far
    int s = 0;
    uint32_t parity = 1;
    bool ok = true;
    for (int i = pair; i < tiles && ok; i += pairs) {
      const TileAt at = tile_of(i, tiles_n, tiles_t);
      const int32_t nrow = at.tn * 2 * kM + kM * (int)rank, trow = at.tt * nt + nt / 2 * (int)rank;
      for (int kb = 0; kb < kblk; ++kb, ++g) {
        if (!wait_all(bar(kEmpty + s), parity)) { give_up(); ok = false; break; }
        if (leader) {
          const uint32_t sa = sbase + s * stage_bytes, sb = sa + kABytes;
          if (even) ptx::mbar_arrive_expect_tx(bar(kFull + s), 2 * stage_bytes);
          ptx::tma_load_2d_pair_hint(sa, &tmW, lead(bar(kFull + s)), kb * kb_elems<F8>(), nrow, w_policy);
          ptx::tma_load_2d_pair(sb, &tmX, lead(bar(kFull + s)), kb * kb_elems<F8>(), trow);
        }
        if (++s == stages) {
          s = 0;
          parity ^= 1;
        }
      }
    }
    // the loads in flight land before the pair may exit (both CTAs' count on these barriers)
    if (even) drain_loads(g, stages, [&](int s) { return bar(kFull + s); }, drain_ns(p));
    if (!ok) ptx::delay_ns(kSettleNs);
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issuer (even CTA)
    if (even) {
      const bool leader = ptx::elect_one();
      const uint32_t idesc = instr_desc<F8>(2 * kM, nt);
      int s = 0, u = 0;  // u: tiles of this pair so far
      uint32_t parity = 0;
      bool ok = true;
      for (int i = pair; i < tiles && ok; i += pairs, ++u) {
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
      // after a wait that ran out: the MMAs issued so far end before the pair's memory goes
      if (__any_sync(0xffffffffu, *abort_flag != 0)) {
        if (leader) ptx::umma_commit_pair(bar(kDrain), 1);
        __all_sync(0xffffffffu, ptx::mbar_wait_cluster_timed(bar(kDrain), 0, drain_ns(p)));
      }
    }
  } else if (warp >= 4) {
    // ---------------------------------------------------------------- epilogue
    const int q = warp % 4, set = (warp - 4) / 4;          // TMEM lanes 32q ..; every kEpiSets-th chunk
    struct Tile {
      int64_t t0;
      int32_t nw;      // the warp's first feature
      int tokens;
    };
    auto tile_at = [&](int i) {
      const TileAt at = tile_of(i, tiles_n, tiles_t);
      const int64_t t0 = (int64_t)at.tt * nt;
      return Tile{t0, at.tn * 2 * kM + kM * (int)rank + 32 * q, (int)min((int64_t)nt, p.T - t0)};
    };
    // this warp has read its part of accumulator b
    auto release = [&](int b) {
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive_cluster_relaxed(lead(bar(kAccFree + b)));
    };
    // this warp's share of a tile's operands into L2, a tile ahead (not WIDE)
    auto prefetch = [&](const Tile& t) {
      if (p.mul || p.res) prefetch_rows(p, t.t0, t.tokens, t.nw, 32, set, kEpiSets, lane);
    };
    float* scale = reinterpret_cast<float*>(smem + off_epi) + (warp - 4) * 256;      // not WIDE
    // WIDE: a piece lies [token][feature] in its place, 64 bytes a token, whose 16-byte parts are
    // turned by the token so that neither access has a bank conflict: lane / 4 is the token and lane %
    // 4 the part of the 16-byte accesses, lane % 8 and lane / 8 those of the matrix ones. The results
    // take the place of the piece's operand. With one operand three pieces are on their way behind
    // the one at work, with two one.
    const uint32_t slots = sbase + off_epi + (warp - 4) * (kSlots * kSlotBytes);
    const bool operands = p.mul || p.res, both = p.mul && p.res;
    const int ahead = both ? kSlots / 2 - 1 : kSlots - 1;
    const uint32_t piece_bytes = both ? 2 * kSlotBytes : kSlotBytes, res_off = both ? kSlotBytes : 0;
    auto place = [](int token, int piece) { return (uint32_t)(64 * token + 16 * (piece ^ (token / 2 % 4))); };
    const uint32_t vec_off = place(lane / 4, lane % 4), mat_off = place(lane % 8, lane / 8);
    // WIDE: scale bytes of the tokens of the warp's piece lane / 4 whose sums lane % 4 has, two each
    auto scales_of = [&](const Tile& t) {
      static_assert(!WIDE || 256 <= 8 * kEpiSets * kOctTokens, "a lane per two tokens");
      const int j = kOctTokens * (set + kEpiSets * (lane / 4)) + 2 * (lane % 4);
      uint32_t two = 0;
      if (j < t.tokens) two = p.xs[t.t0 + j];
      if (j + 1 < t.tokens) two |= (uint32_t)p.xs[t.t0 + j + 1] << 8;
      return two;
    };
    int u = 0;
    Tile t = tile_at(min(pair, tiles - 1)), after = t;
    uint32_t scales_after = WIDE && F8 ? scales_of(t) : 0;
    if (!WIDE) prefetch(t);
    for (int i = pair; i < tiles; i += pairs, ++u) {
      const int b = u & 1;
      t = after;
      if (i + pairs < tiles) after = tile_at(i + pairs);
      if constexpr (WIDE) {
        const int tok = lane / 4;
        const int32_t n = t.nw + 8 * (lane % 4);
        float bias[4], ws[4];      // of features nw + lane / 4 + 8 m
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          const int32_t f = t.nw + lane / 4 + 8 * m;
          bias[m] = p.bias && f < p.N ? __bfloat162float(p.bias[f]) : 0.f;
          ws[m] = F8 && f < p.N ? scale_of(p.ws[f]) : 1.f;
        }
        const uint32_t trow = tbase + ((32u * q) << 16) + b * nt;
        constexpr int kSweep = kEpiSets * kOctTokens;
        int c = kOctTokens * set, k = 0;
        const int64_t step = (int64_t)kSweep * p.N;
        int64_t at = (t.t0 + c + tok) * p.N + n;
        // operands of the piece from token c on, one group of copies (empty past the tile's tokens)
        const int own = n < p.N ? t.tokens - tok : 0;      // pieces before it have this thread's token
        auto fetch = [&](int c, int64_t at, int into) {
          const uint32_t dst = slots + (into & ahead) * piece_bytes + vec_off;
          if (c < own) {
            if (p.mul) ptx::copy16_async(dst, p.mul + at);
            if (p.res) ptx::copy16_async(dst + res_off, p.res + at);
          }
          ptx::copy_commit();
        };
        const uint32_t scales = scales_after;      // of this tile
        if (F8 && i + pairs < tiles) scales_after = scales_of(after);
        __syncwarp();      // the tile before is read
        if (operands)
          for (int far = 0; far < ahead; ++far) fetch(c + far * kSweep, at + far * step, far);
        const int64_t far = ahead * step;
        if (!wait_all(bar(kAccFull + b), (uint32_t)((u >> 1) & 1))) { give_up(); break; }
        ptx::tc_fence_after();
#pragma unroll 1
        for (; c < t.tokens; c += kSweep, at += step, ++k) {
          float v[8];      // feature lane / 4 + 8 m, tokens c + 2 (lane % 4) + {0, 1}: v[2 m ..]
          ptx::tmem_ld_16x256b_x1(trow + c, v);
          ptx::tmem_ld_16x256b_x1(trow + (16u << 16) + c, v + 4);
          const uint32_t piece = slots + (k & ahead) * piece_bytes;
          if (operands) {
            if (both) ptx::copy_wait<kSlots / 2 - 2>();
            else ptx::copy_wait<kSlots - 2>();
            __syncwarp();      // and every lane has read the results from the place that is filled next
            fetch(c + ahead * kSweep, at + far, k + ahead);
          }
          const uint32_t sx = F8 ? __shfl_sync(0xffffffffu, scales, 4 * k + lane % 4) : 0;
          const ptx::F2 x = ptx::f2(scale_of((uint8_t)sx), scale_of((uint8_t)(sx >> 8)));
          ptx::tmem_wait_ld();
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            ptx::F2 two = ptx::f2(v[2 * m], v[2 * m + 1]);
            if (F8) two = ptx::mul2(ptx::mul2(two, ptx::f2(ws[m], ws[m])), x);
            ptx::split(ptx::add2(two, ptx::f2(bias[m], bias[m])), v[2 * m], v[2 * m + 1]);
          }
          activate(v, p.act);
          uint32_t w[4];
          if (p.mul) {
            ptx::ldmatrix_x4_trans(piece + mat_off, w);
#pragma unroll
            for (int m = 0; m < 4; ++m)
              ptx::split(ptx::mul2(ptx::f2(v[2 * m], v[2 * m + 1]), halves(w[m])), v[2 * m], v[2 * m + 1]);
          }
          if (p.res) {
            ptx::ldmatrix_x4_trans(piece + res_off + mat_off, w);
#pragma unroll
            for (int m = 0; m < 4; ++m)
              ptx::split(ptx::add2(ptx::f2(v[2 * m], v[2 * m + 1]), halves(w[m])), v[2 * m], v[2 * m + 1]);
          }
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * m], v[2 * m + 1]);
            w[m] = *reinterpret_cast<const uint32_t*>(&h);
          }
          if (operands) __syncwarp();      // the operand is read: its place takes the results
          ptx::stmatrix_x4_trans(piece + mat_off, w);
          __syncwarp();
          if (c < own) *reinterpret_cast<uint4*>(p.out + at) = ptx::ld_shared_v4(piece + vec_off);
        }
      } else {
        if (F8) {
          __syncwarp();      // the tile before is read
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int j = 32 * k + lane;
            scale[j] = j < t.tokens ? scale_of(p.xs[t.t0 + j]) : 0.f;
          }
          __syncwarp();
        }
        const int32_t n = t.nw + lane;
        const float bias = p.bias && n < p.N ? __bfloat162float(p.bias[n]) : 0.f;
        const float ws = F8 && n < p.N ? scale_of(p.ws[n]) : 1.f;
        const uint32_t trow = tbase + ((32u * q) << 16) + b * nt;
        const int64_t step = (int64_t)kEpiSets * kChunk * p.N;
        int c = kChunk * set;
        int64_t at = (t.t0 + c) * p.N + n;
        // a chunk's operands are loaded before the chunk before it is finished
        Operands<kChunk> ops, next;
        if (c < t.tokens && n < p.N) ops.load(p, at, t.tokens - c);
        if (!wait_all(bar(kAccFull + b), (uint32_t)((u >> 1) & 1))) { give_up(); break; }
        ptx::tc_fence_after();
        if (i + pairs < tiles) prefetch(after);      // its main loop is beginning
#pragma unroll 2
        for (; c < t.tokens; c += kEpiSets * kChunk, at += step) {
          float v[kChunk];
          ptx::tmem_ld_32x32b_x16(trow + c, v);
          const int left = t.tokens - c, then = left - kEpiSets * kChunk;
          if (then > 0 && n < p.N) next.load(p, at + step, then);
          float sx[kChunk];
          if (F8) {
#pragma unroll
            for (int j = 0; j < kChunk; j += 4)
              *reinterpret_cast<float4*>(sx + j) = *reinterpret_cast<const float4*>(scale + c + j);
          }
          ptx::tmem_wait_ld();
          if (n < p.N) finish_tokens<F8, kChunk>(p, v, ops, at, left, bias, ws, sx);
          ops = next;
          __syncwarp();
        }
      }
      release(b);
    }
    if (WIDE) ptx::copy_wait<0>();      // (after a wait that ran out)
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
