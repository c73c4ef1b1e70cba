// add_rmsnorm.cuh -- the residual stream's addition and RMS norm, with a bf16, fp32 or
// 8-bit output, and the 8-bit row quantiser at any width.
//
// Per row t of x [T][M]:  s = x + r (r optional),  r' = round(s),
//   y = (s g) / sqrt(mean(s^2) + eps)
// and y is written in the rows' type, or as E4M3 codes with one power-of-two scale 2^k (the
// byte k + 127), or both. The norm and y are taken from the fp32 sum s, not from the stored
// r': the one rounding of each output is its store. With no norm (the quantiser) y = x.
//
// The scale needs max |y| before any code is written. y is computed as (s g) inv with one
// row-wide inv > 0, and rounding is monotonic, so max |y| is exactly (max |s g|) inv: the
// sum of squares and max |s g| are reduced together, in one exchange, and a row is read
// once and stays in registers. Bound by HBM (each input read once, each output written once).
//
// Rows of any width are moved in granules, the aligned 16-byte pieces (VE elements) of the
// whole tensor: row t covers elements tM .. tM + M, which begin `shift` elements into
// granule tM / VE. x, r, r' and y share that layout; the codes of a granule are VE aligned
// bytes, for tM - shift is a multiple of VE. A row's first and last granule may hold a
// neighbour's elements: those are read and ignored, and never written. Only the gain is
// out of step with a shifted row; its VE elements come out of two of its granules.
// (With 2-byte accesses instead, a bf16 row of odd width moved at a quarter of the rate.)
#pragma once

#include "common.cuh"
#include "fp8_kernels.cuh"
#include "ptx.cuh"

namespace mla {
namespace rms {

struct Params {
  const void* x;
  const void* r;          // or null
  const void* gain;       // null: no norm (y = x)
  void* r_out;            // or null
  void* y;                // or null
  uint8_t* codes;         // [T][M] or null
  uint8_t* scales;        // [T], with codes
  int32_t T, M;
  float eps;
};

constexpr int kWarpRows = 8;      // rows (warps) of a block when one warp holds a row

template <typename T> __host__ __device__ constexpr int granule() { return 16 / (int)sizeof(T); }

// The scale exponent of a row whose largest magnitude is amax: the smallest k in
// [-126, 7] with amax <= 448 2^k. 448 = 1.75 * 2^8, so an amax of mantissa up to 1.75
// takes its own exponent - 8, a larger one exponent - 7. An infinite amax gives 7, a zero
// or subnormal one -126.
__device__ __forceinline__ int scale_exponent(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int e = (int)(u >> 23) - 127;
  const int k = (u & 0x7FFFFFu) <= 0x600000u ? e - 8 : e - 7;
  return min(max(k, f8::kKMin), f8::kKMax);
}

template <typename T>
__device__ __forceinline__ void unpack(const uint4& w, float (&v)[granule<T>()]) {
  if constexpr (sizeof(T) == 2) {
    f8::unpack8(w, v);
  } else {
    v[0] = __uint_as_float(w.x);
    v[1] = __uint_as_float(w.y);
    v[2] = __uint_as_float(w.z);
    v[3] = __uint_as_float(w.w);
  }
}
template <typename T>
__device__ __forceinline__ uint4 pack(const float (&v)[granule<T>()]) {
  uint4 w;
  T* e = reinterpret_cast<T*>(&w);
#pragma unroll
  for (int i = 0; i < granule<T>(); ++i) e[i] = from_f32<T>(v[i]);
  return w;
}
// Granule i of a tensor of n elements; one that reaches past the tensor (or before it) is
// filled element by element, zeros outside.
template <typename T>
__device__ __forceinline__ uint4 load_granule(const void* base, int64_t i, int64_t n) {
  constexpr int VE = granule<T>();
  if (i >= 0 && (i + 1) * VE <= n) return static_cast<const uint4*>(base)[i];
  uint4 w = make_uint4(0, 0, 0, 0);
  T* e = reinterpret_cast<T*>(&w);
#pragma unroll
  for (int k = 0; k < VE; ++k)
    if (i * VE + k >= 0 && i * VE + k < n) e[k] = static_cast<const T*>(base)[i * VE + k];
  return w;
}
// The VE elements that start VE - shift elements into granules lo, hi (shift < VE, the same
// for the whole warp).
template <typename T>
__device__ __forceinline__ uint4 window(const uint4& lo, const uint4& hi, int shift) {
  constexpr int VE = granule<T>(), kPerWord = 4 / (int)sizeof(T);
  const uint32_t w[9] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w, 0u};
  const int p = VE - shift;
  uint32_t r[5];
  switch (p / kPerWord) {
#define MLA_RMS_CASE(K)                       \
  case K:                                     \
    for (int i = 0; i < 5; ++i) r[i] = w[K + i]; \
    break;
    MLA_RMS_CASE(0)
    MLA_RMS_CASE(1)
    MLA_RMS_CASE(2)
    MLA_RMS_CASE(3)
    default:
      for (int i = 0; i < 5; ++i) r[i] = w[4 + i];
#undef MLA_RMS_CASE
  }
  if (p % kPerWord != 0) {
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = __funnelshift_r(r[i], r[i + 1], 16);
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}
// Granule i of a row-shaped output, elements [first, last) of it only.
template <typename T>
__device__ __forceinline__ void store_granule(void* base, int64_t i, const float (&v)[granule<T>()], int first,
                                              int last) {
  constexpr int VE = granule<T>();
  if (first <= 0 && last >= VE) {
    static_cast<uint4*>(base)[i] = pack<T>(v);
  } else {
#pragma unroll
    for (int k = 0; k < VE; ++k)
      if (k >= first && k < last) static_cast<T*>(base)[i * VE + k] = from_f32<T>(v[k]);
  }
}
// The codes of v * up, elements [first, last) of granule i.
template <int VE>
__device__ __forceinline__ void store_codes(uint8_t* base, int64_t i, const float (&v)[VE], float up, int first,
                                            int last) {
  uint32_t c[VE / 4];
#pragma unroll
  for (int k = 0; k < VE; k += 4)
    c[k / 4] = f8::to_e4m3x2(v[k] * up, v[k + 1] * up) | (f8::to_e4m3x2(v[k + 2] * up, v[k + 3] * up) << 16);
  if (first <= 0 && last >= VE) {
    if constexpr (VE == 8) reinterpret_cast<uint2*>(base)[i] = make_uint2(c[0], c[1]);
    else reinterpret_cast<uint32_t*>(base)[i] = c[0];
  } else {
#pragma unroll
    for (int k = 0; k < VE; ++k)
      if (k >= first && k < last) base[i * VE + k] = (uint8_t)(c[k / 4] >> (8 * (k % 4)));
  }
}

// Sum of ss and maximum of am (>= 0) over a warp.
__device__ __forceinline__ void warp_reduce(float& ss, float& am) {
  ss = warp_sum(ss);
  am = f8::warp_max_abs(am);
}
// ... and over the block, in the same fixed order in every thread.
__device__ __forceinline__ void block_reduce(float& ss, float& am, float (&red)[2][32]) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, n = blockDim.x >> 5;
  warp_reduce(ss, am);
  if (lane == 0) {
    red[0][warp] = ss;
    red[1][warp] = am;
  }
  __syncthreads();
  ss = lane < n ? red[0][lane] : 0.f;
  am = lane < n ? red[1][lane] : 0.f;
  warp_reduce(ss, am);
}

// Where row `row` lies among the granules. SHIFTED = false: M is a multiple of VE.
template <int VE, bool SHIFTED>
struct Row {
  int64_t g0;      // its first granule
  int shift;       // its first element within that granule
  int count;       // granules it touches
  __device__ __forceinline__ Row(int64_t row, int M) {
    const int64_t e0 = row * M;
    g0 = e0 / VE;
    shift = SHIFTED ? (int)(e0 % VE) : 0;
    count = SHIFTED ? (shift + M + VE - 1) / VE : M / VE;
  }
  // elements [first, last) of its granule c are the row's
  __device__ __forceinline__ int first(int c) const { return SHIFTED && c == 0 ? shift : 0; }
  __device__ __forceinline__ int last(int c, int M) const { return SHIFTED ? min(VE, shift + M - c * VE) : VE; }
};

// s and its statistics, in the order every kernel here uses: v becomes s * gain.
template <int VE>
__device__ __forceinline__ void accumulate(float (&v)[VE], const float (&g)[VE], bool norm, int first, int last,
                                           float& ss, float& am) {
#pragma unroll
  for (int e = 0; e < VE; ++e)
    if (e >= first && e < last) {
      ss += v[e] * v[e];
      if (norm) v[e] *= g[e];
      am = fmaxf(am, fabsf(v[e]));
    }
}

// Few rows, or short ones: one row per warp (WARP: blocks of kWarpRows rows) or per block,
// ITEMS granules a thread, granule c of the row in thread c % threads. Straight loads: with
// as many threads as the row has granules a call of a few rows is one round trip to memory,
// and a thread's loads are all in flight before the first is used. A thread keeps its
// elements and their gains, so blocks of 1024 threads hold up to 16 elements a thread.
template <typename T, int ITEMS, bool WARP, bool SHIFTED>
__global__ void __launch_bounds__(WARP ? 32 * kWarpRows : 1024) add_rmsnorm_kernel(const Params p) {
  constexpr int VE = granule<T>();
  __shared__ float red[2][32];
  const int nthr = WARP ? 32 : blockDim.x;
  const int tid = WARP ? (threadIdx.x & 31) : threadIdx.x;
  const int64_t row = WARP ? (int64_t)blockIdx.x * kWarpRows + (threadIdx.x >> 5) : blockIdx.x;
  if (WARP && row >= p.T) return;
  const Row<VE, SHIFTED> at(row, p.M);
  const int64_t n = (int64_t)p.T * p.M;
  uint4 xw[ITEMS], rw[ITEMS], gw[ITEMS];
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const int c = tid + i * nthr;
    if (c < at.count) xw[i] = load_granule<T>(p.x, at.g0 + c, n);
  }
  if (p.r) {
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const int c = tid + i * nthr;
      if (c < at.count) rw[i] = load_granule<T>(p.r, at.g0 + c, n);
    }
  }
  if (p.gain) {
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const int c = tid + i * nthr;
      if (c < at.count) {
        gw[i] = load_granule<T>(p.gain, c, p.M);
        if (SHIFTED && at.shift) gw[i] = window<T>(load_granule<T>(p.gain, c - 1, p.M), gw[i], at.shift);
      }
    }
  }
  float v[ITEMS][VE];
  float ss = 0.f, am = 0.f;
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const int c = tid + i * nthr;
    if (c < at.count) {
      unpack<T>(xw[i], v[i]);
      if (p.r) {
        float r[VE];
        unpack<T>(rw[i], r);
#pragma unroll
        for (int e = 0; e < VE; ++e) v[i][e] += r[e];
      }
      const int first = at.first(c), last = at.last(c, p.M);
      if (p.r_out) store_granule<T>(p.r_out, at.g0 + c, v[i], first, last);
      float g[VE] = {};
      if (p.gain) unpack<T>(gw[i], g);
      accumulate<VE>(v[i], g, p.gain != nullptr, first, last, ss, am);
    }
  }
  if (WARP) warp_reduce(ss, am);
  else block_reduce(ss, am, red);
  const float inv = p.gain ? 1.f / sqrtf(ss / (float)p.M + p.eps) : 1.f;
  const int k = scale_exponent(am * inv);
  const float up = f8::pow2(-k);
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const int c = tid + i * nthr;
    if (c < at.count) {
#pragma unroll
      for (int e = 0; e < VE; ++e) v[i][e] *= inv;
      const int first = at.first(c), last = at.last(c, p.M);
      if (p.y) store_granule<T>(p.y, at.g0 + c, v[i], first, last);
      if (p.codes) store_codes<VE>(p.codes, at.g0 + c, v[i], up, first, last);
    }
  }
  if (p.codes && tid == 0) p.scales[row] = (uint8_t)(k + 127);
}

// Many rows: persistent blocks, each with a ring of kStages row buffers in shared memory
// that bulk copies keep full while the block works on the oldest row. ITEMS granules a
// thread. One barrier per row: once it has passed, every thread holds its part of the row
// in registers and the buffer is loaded again. The inputs are read once, so they are loaded
// with evict-first priority, which leaves L2 to the writes (T = 16384, M = 7168, bf16 with a
// residual: 160 us against 169 without, and 204 for the kernel above; two buffers and
// four granules a thread beat three buffers, or two or eight granules).
constexpr int kStages = 2;
constexpr int kStreamThreads = 512;

// Shared memory of a block, after the alignment of each part: the ring, then the gain with
// a granule of zeros on either side.
template <typename T>
__host__ __device__ constexpr int64_t stream_row_bytes(int64_t M) {
  return (M + granule<T>() - 1 + granule<T>() - 1) / granule<T>() * 16;   // touched at the worst shift
}
template <typename T>
__host__ __device__ constexpr int64_t stream_smem(int64_t M, bool residual) {
  return stream_row_bytes<T>(M) * (residual ? 2 : 1) * kStages + stream_row_bytes<T>(M) + 32;
}

template <typename T, int ITEMS, bool SHIFTED>
__global__ void __launch_bounds__(kStreamThreads) add_rmsnorm_stream_kernel(const Params p, uint64_t timeout_ns) {
  constexpr int VE = granule<T>();
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ __align__(8) uint64_t full_bar[kStages];
  __shared__ float red[2][2][kStreamThreads / 32];
  __shared__ int abort_word;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, nthr = blockDim.x, warps = nthr >> 5;
  const int64_t n = (int64_t)p.T * p.M;
  const uint32_t row_bytes = (uint32_t)stream_row_bytes<T>(p.M), stage_bytes = p.r ? 2 * row_bytes : row_bytes;
  const int grid = gridDim.x;
  auto bar = [&](int s) { return ptx::smem_u32(&full_bar[s]); };
  // one thread: the row's granules that lie wholly inside the tensor
  auto fetch = [&](int s, int64_t row) {
    const Row<VE, SHIFTED> at(row, p.M);
    const int whole = SHIFTED && (at.g0 + at.count) * VE > n ? at.count - 1 : at.count;
    const uint32_t bytes = (uint32_t)whole * 16u;
    const uint32_t dst = ptx::smem_u32(smem + (size_t)s * stage_bytes);
    const uint64_t policy = ptx::policy_evict_first();
    ptx::mbar_arrive_expect_tx(bar(s), p.r ? 2 * bytes : bytes);
    if (bytes) {
      ptx::bulk_load_g2s_hint(dst, static_cast<const uint4*>(p.x) + at.g0, bytes, bar(s), policy);
      if (p.r) ptx::bulk_load_g2s_hint(dst + row_bytes, static_cast<const uint4*>(p.r) + at.g0, bytes, bar(s), policy);
    }
  };
  if (tid == 0) {
    abort_word = 0;
    for (int s = 0; s < kStages; ++s) ptx::mbar_init(bar(s), 1);
    ptx::fence_mbar_init();
    for (int s = 0; s < kStages; ++s)
      if (blockIdx.x + (int64_t)s * grid < p.T) fetch(s, blockIdx.x + (int64_t)s * grid);
  }
  // the gain: in registers where every row has the same columns, else in shared memory
  uint4 gw[ITEMS];
  uint4* sg = reinterpret_cast<uint4*>(smem + (size_t)kStages * stage_bytes);   // granule -1 first
  if (SHIFTED) {
    for (int i = tid; i < p.M / VE + 3; i += nthr) sg[i] = load_granule<T>(p.gain, i - 1, p.M);
  } else {
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const int c = tid + i * nthr;
      if (c < p.M / VE) gw[i] = static_cast<const uint4*>(p.gain)[c];
    }
  }
  __syncthreads();
  int s = 0, it = 0;
  uint32_t parity = 0;
  for (int64_t row = blockIdx.x; row < p.T; row += grid, ++it) {
    const Row<VE, SHIFTED> at(row, p.M);
    const bool ok = ptx::mbar_wait_bounded(bar(s), parity, &abort_word, timeout_ns);
    const uint4* sx = reinterpret_cast<const uint4*>(smem + (size_t)s * stage_bytes);
    const uint4* sr = reinterpret_cast<const uint4*>(smem + (size_t)s * stage_bytes + row_bytes);
    float v[ITEMS][VE];
    float ss = 0.f, am = 0.f;
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const int c = tid + i * nthr;
      if (c < at.count) {
        // the tensor's last granule, if partial, was not copied
        const bool tail = SHIFTED && (at.g0 + c + 1) * VE > n;
        unpack<T>(tail ? load_granule<T>(p.x, at.g0 + c, n) : sx[c], v[i]);
        if (p.r) {
          float r[VE];
          unpack<T>(tail ? load_granule<T>(p.r, at.g0 + c, n) : sr[c], r);
#pragma unroll
          for (int e = 0; e < VE; ++e) v[i][e] += r[e];
        }
      }
    }
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const int c = tid + i * nthr;
      if (c < at.count) {
        const int first = at.first(c), last = at.last(c, p.M);
        if (p.r_out) store_granule<T>(p.r_out, at.g0 + c, v[i], first, last);
        float g[VE];
        if (SHIFTED) unpack<T>(at.shift ? window<T>(sg[c], sg[c + 1], at.shift) : sg[c + 1], g);
        else unpack<T>(gw[i], g);
        accumulate<VE>(v[i], g, true, first, last, ss, am);
      }
    }
    warp_reduce(ss, am);
    if (lane == 0) {
      red[it & 1][0][warp] = ss;
      red[it & 1][1][warp] = am;
    }
    if (!__syncthreads_and(ok)) {
      // the wait ran out: report, let the copies in flight land (bounded), leave
      if (tid == 0) {
        raise_status(kStatusTimeout);
        for (int k = 0; k < kStages; ++k) {
          const int b = (s + k) % kStages;
          if (row + (int64_t)k * grid < p.T)
            ptx::mbar_wait_cluster_timed(bar(b), b < s ? parity ^ 1u : parity, timeout_ns);
        }
      }
      return;
    }
    if (tid == 0 && row + (int64_t)kStages * grid < p.T) fetch(s, row + (int64_t)kStages * grid);
    ss = lane < warps ? red[it & 1][0][lane] : 0.f;
    am = lane < warps ? red[it & 1][1][lane] : 0.f;
    warp_reduce(ss, am);
    const float inv = 1.f / sqrtf(ss / (float)p.M + p.eps);
    const int k = scale_exponent(am * inv);
    const float up = f8::pow2(-k);
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const int c = tid + i * nthr;
      if (c < at.count) {
#pragma unroll
        for (int e = 0; e < VE; ++e) v[i][e] *= inv;
        const int first = at.first(c), last = at.last(c, p.M);
        if (p.y) store_granule<T>(p.y, at.g0 + c, v[i], first, last);
        if (p.codes) store_codes<VE>(p.codes, at.g0 + c, v[i], up, first, last);
      }
    }
    if (p.codes && tid == 0) p.scales[row] = (uint8_t)(k + 127);
    if (++s == kStages) {
      s = 0;
      parity ^= 1;
    }
  }
}

// Any width and alignment: one block per row, two passes over it (the second reads again
// what the first summed; r_out and y are written in the second, element by element by the
// thread that read them, so they may be r's and x's own buffers). For operands that are not
// 16-byte aligned, and rows too wide for the registers of a block.
template <typename T>
__global__ void __launch_bounds__(1024) add_rmsnorm_any_kernel(const Params p) {
  __shared__ float red[2][32];
  const int64_t at = (int64_t)blockIdx.x * p.M;
  const T* x = static_cast<const T*>(p.x) + at;
  const T* r = p.r ? static_cast<const T*>(p.r) + at : nullptr;
  const T* g = static_cast<const T*>(p.gain);
  float ss = 0.f, am = 0.f;
  for (int c = threadIdx.x; c < p.M; c += blockDim.x) {
    const float s = to_f32<T>(x[c]) + (r ? to_f32<T>(r[c]) : 0.f);
    ss += s * s;
    am = fmaxf(am, fabsf(g ? s * to_f32<T>(g[c]) : s));
  }
  block_reduce(ss, am, red);
  const float inv = g ? 1.f / sqrtf(ss / (float)p.M + p.eps) : 1.f;
  const int k = scale_exponent(am * inv);
  const float up = f8::pow2(-k);
  for (int c = threadIdx.x; c < p.M; c += blockDim.x) {
    const float s = to_f32<T>(x[c]) + (r ? to_f32<T>(r[c]) : 0.f);
    if (p.r_out) static_cast<T*>(p.r_out)[at + c] = from_f32<T>(s);
    const float y = g ? (s * to_f32<T>(g[c])) * inv : s;
    if (p.y) static_cast<T*>(p.y)[at + c] = from_f32<T>(y);
    if (p.codes) p.codes[at + c] = (uint8_t)f8::to_e4m3x2(y * up, 0.f);
  }
  if (p.codes && threadIdx.x == 0) p.scales[blockIdx.x] = (uint8_t)(k + 127);
}

}  // namespace rms
}  // namespace mla
