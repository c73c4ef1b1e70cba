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
// out of step with a shifted row. (16384 x 1111 bf16: 31 us with a residual, 26 without; with
// 2-byte accesses instead, as the row's own alignment allows, about 100.)
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
  float inv_m;            // 1 / M
  float eps;
};

constexpr int kWarpRows = 8;      // rows (warps) of a block when one warp holds a row

template <typename T> __host__ __device__ constexpr int granule() { return 16 / (int)sizeof(T); }

// The scale exponent of a row whose largest magnitude is amax: the smallest k in
// [-126, 7] with amax <= 448 2^k. 448 = 1.75 * 2^8, so an amax of mantissa up to 1.75
// takes its own exponent - 8, a larger one exponent - 7. An infinite amax gives 7, a zero
// or subnormal one -126. So does a NaN, max |s g| times a 1 / sqrt that is NaN, or infinity
// times zero either way round: then every value of the row is a NaN, which does not count, or 0.
__device__ __forceinline__ int scale_exponent(float amax) {
  const uint32_t u = __float_as_uint(fmaxf(amax, 0.f));
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
// Granule i of a row or tensor, of which elements [0, have) exist (VE: all of them); the
// others are zeros.
template <typename T>
__device__ __forceinline__ uint4 load_granule(const void* base, int64_t i, int have = granule<T>()) {
  constexpr int VE = granule<T>();
  if (have >= VE) return static_cast<const uint4*>(base)[i];
  uint4 w = make_uint4(0, 0, 0, 0);
  T* e = reinterpret_cast<T*>(&w);
#pragma unroll
  for (int k = 0; k < VE; ++k)
    if (k < have) e[k] = static_cast<const T*>(base)[i * VE + k];
  return w;
}
// Elements [first, last) of granule i of a row-shaped output (WHOLE: all of them).
template <typename T, bool WHOLE>
__device__ __forceinline__ void store_granule(void* base, int64_t i, const float (&v)[granule<T>()], int first,
                                              int last) {
  constexpr int VE = granule<T>();
  if (WHOLE) {
    static_cast<uint4*>(base)[i] = pack<T>(v);
  } else {
#pragma unroll
    for (int k = 0; k < VE; ++k)
      if (k >= first && k < last) static_cast<T*>(base)[i * VE + k] = from_f32<T>(v[k]);
  }
}
// The codes of v * up, elements [first, last) of granule i.
template <int VE, bool WHOLE>
__device__ __forceinline__ void store_codes(uint8_t* base, int64_t i, const float (&v)[VE], float up, int first,
                                            int last) {
  uint32_t c[VE / 4];
#pragma unroll
  for (int k = 0; k < VE; k += 4)
    c[k / 4] = f8::to_e4m3x2(v[k] * up, v[k + 1] * up) | (f8::to_e4m3x2(v[k + 2] * up, v[k + 3] * up) << 16);
  if (WHOLE) {
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
  int have;        // the row's and its neighbours' elements up to its end in its last granule (0: all)
  int tail;        // the granule that reaches past the tensor's end (-1: none; with M < VE any of
                   // the last rows' can), ..
  int inside;      // .. and its elements inside
  __device__ __forceinline__ Row(int64_t row, int T, int M) {
    const int64_t e0 = row * M;
    g0 = e0 / VE;
    shift = SHIFTED ? (int)(e0 % VE) : 0;
    count = SHIFTED ? (shift + M + VE - 1) / VE : M / VE;
    have = (shift + M) % VE;
    const int64_t over = (g0 + count) * VE - (int64_t)T * M;      // elements past the end, below VE
    tail = SHIFTED && over > 0 ? count - 1 : -1;
    inside = VE - (int)(over > 0 ? over : 0);
  }
  // elements [first, last) of its granule c are the row's
  __device__ __forceinline__ int first(int c) const { return c == 0 ? shift : 0; }
  __device__ __forceinline__ int last(int c, int M) const { return min(VE, shift + M - c * VE); }
  __device__ __forceinline__ bool whole(int c) const {
    return !SHIFTED || ((c > 0 || shift == 0) && (c < count - 1 || have == 0));
  }
  // granule c of x or r
  template <typename T>
  __device__ __forceinline__ uint4 load(const void* base, int c) const {
    return load_granule<T>(base, g0 + c, SHIFTED && c == tail ? inside : VE);
  }
};

// The gains of the row's granule c, columns c VE - shift ..: a shifted row's are not aligned,
// and come one by one (from L1; zeros outside the row).
template <typename T, bool SHIFTED>
__device__ __forceinline__ void gains_of(const void* gain, const Row<granule<T>(), SHIFTED>& at, int c, int M,
                                         float (&g)[granule<T>()]) {
  constexpr int VE = granule<T>();
  if (!SHIFTED) {
    unpack<T>(static_cast<const uint4*>(gain)[c], g);
  } else {
    const T* gp = static_cast<const T*>(gain) + (c * VE - at.shift);
    if (at.whole(c)) {
#pragma unroll
      for (int e = 0; e < VE; ++e) g[e] = to_f32<T>(gp[e]);
    } else {
      const int first = at.first(c), last = at.last(c, M);
#pragma unroll
      for (int e = 0; e < VE; ++e) g[e] = e >= first && e < last ? to_f32<T>(gp[e]) : 0.f;
    }
  }
}

// s into its statistics, in the order every kernel here uses: v becomes s * gain.
template <int VE>
__device__ __forceinline__ void accumulate(float (&v)[VE], const float (&g)[VE], bool norm, float& ss, float& am) {
#pragma unroll
  for (int e = 0; e < VE; ++e) {
    ss += v[e] * v[e];
    if (norm) v[e] *= g[e];
    am = fmaxf(am, fabsf(v[e]));
  }
}

// The two steps of a granule: its s stored and summed (a neighbour's elements count as
// zeros from here on); its y stored.
template <typename T, bool SHIFTED>
__device__ __forceinline__ void first_step(const Params& p, const Row<granule<T>(), SHIFTED>& at, int c,
                                           float (&v)[granule<T>()], const float (&g)[granule<T>()], bool norm,
                                           float& ss, float& am) {
  constexpr int VE = granule<T>();
  if (at.whole(c)) {
    if (p.r_out) store_granule<T, true>(p.r_out, at.g0 + c, v, 0, VE);
  } else {
    const int first = at.first(c), last = at.last(c, p.M);
    if (p.r_out) store_granule<T, false>(p.r_out, at.g0 + c, v, first, last);
#pragma unroll
    for (int e = 0; e < VE; ++e)
      if (e < first || e >= last) v[e] = 0.f;
  }
  accumulate<VE>(v, g, norm, ss, am);
}
template <typename T, bool SHIFTED>
__device__ __forceinline__ void second_step(const Params& p, const Row<granule<T>(), SHIFTED>& at, int c,
                                            float (&v)[granule<T>()], float inv, float up) {
  constexpr int VE = granule<T>();
#pragma unroll
  for (int e = 0; e < VE; ++e) v[e] *= inv;
  if (at.whole(c)) {
    if (p.y) store_granule<T, true>(p.y, at.g0 + c, v, 0, VE);
    if (p.codes) store_codes<VE, true>(p.codes, at.g0 + c, v, up, 0, VE);
  } else {
    const int first = at.first(c), last = at.last(c, p.M);
    if (p.y) store_granule<T, false>(p.y, at.g0 + c, v, first, last);
    if (p.codes) store_codes<VE, false>(p.codes, at.g0 + c, v, up, first, last);
  }
}

// Few rows, or short ones: one row per warp (WARP: blocks of kWarpRows rows) or per block,
// ITEMS granules a thread, granule c of the row in thread c % threads. Straight loads: with
// as many threads as the row has granules a call of a few rows is one round trip to memory,
// and a thread's loads are all in flight before the first is used. One row a block: blocks
// that stay and load the next row's granules under this row's exchange were slower (16384 x
// 1111 bf16 45 us against 37 for this kernel's form of then, which now takes 31; 8000 x 1112 fp32
// 17.5 against 14.8). A thread keeps its
// elements and their gains, so blocks of 1024 threads hold up to 16 elements a thread, and
// kWideThreads up to 32.
constexpr int kWideThreads = 544;   // 16384 elements and a shifted row's one granule more
__host__ __device__ constexpr int max_threads(int elems) { return elems <= 16 ? 1024 : kWideThreads; }

template <typename T, int ITEMS, bool WARP, bool SHIFTED>
__global__ void __launch_bounds__(WARP ? 32 * kWarpRows : max_threads(granule<T>() * ITEMS))
add_rmsnorm_kernel(const Params p) {
  constexpr int VE = granule<T>();
  __shared__ float red[2][32];
  const int nthr = WARP ? 32 : blockDim.x;
  const int tid = WARP ? (threadIdx.x & 31) : threadIdx.x;
  const int64_t row = WARP ? (int64_t)blockIdx.x * kWarpRows + (threadIdx.x >> 5) : blockIdx.x;
  ptx::grid_launch_next();
  ptx::grid_wait();      // from here on this kernel reads and writes global memory
  if (WARP && row >= p.T) return;
  const Row<VE, SHIFTED> at(row, p.T, p.M);
  uint4 xw[ITEMS], rw[ITEMS];
  float g[ITEMS][VE];
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const int c = tid + i * nthr;
    if (c < at.count) xw[i] = at.template load<T>(p.x, c);
  }
  if (p.r) {
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const int c = tid + i * nthr;
      if (c < at.count) rw[i] = at.template load<T>(p.r, c);
    }
  }
  if (p.gain) {
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const int c = tid + i * nthr;
      if (c < at.count) gains_of<T, SHIFTED>(p.gain, at, c, p.M, g[i]);
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
      first_step<T, SHIFTED>(p, at, c, v[i], g[i], p.gain != nullptr, ss, am);
    }
  }
  if (WARP) warp_reduce(ss, am);
  else block_reduce(ss, am, red);
  const float inv = p.gain ? rsqrtf(ss * p.inv_m + p.eps) : 1.f;
  const int k = scale_exponent(am * inv);
  const float up = f8::pow2(-k);
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const int c = tid + i * nthr;
    if (c < at.count) second_step<T, SHIFTED>(p, at, c, v[i], inv, up);
  }
  if (p.codes && tid == 0) p.scales[row] = (uint8_t)(k + 127);
}

// Many rows of whole granules: persistent blocks, each with a ring of kStages row buffers in
// shared memory that bulk copies keep full while the block works on the oldest row. ITEMS
// granules a thread, whose gains it keeps for every row. One barrier per row: once it has
// passed, every thread holds its part of the row in registers and the buffer is loaded
// again. The inputs are read once, so they are loaded with evict-first priority, which
// leaves L2 to the writes (T = 16384, M = 7168, bf16 with a residual: 155 us, 6.05 TB/s,
// against 169 us without, and 204 for the kernel above; two buffers and four granules a
// thread beat three buffers, or two or eight granules). Shifted rows gained nothing here.
// It is not instantiated for the quantiser, which has a block a row (16384 x 8192 bf16: 114 us,
// 61 for the bytes).
constexpr int kStages = 2;
constexpr int kStreamThreads = 512;

template <typename T, int ITEMS>
__global__ void __launch_bounds__(kStreamThreads) add_rmsnorm_stream_kernel(const Params p, uint64_t timeout_ns) {
  constexpr int VE = granule<T>();
  extern __shared__ __align__(16) uint8_t smem[];     // [kStages][x row, r row]
  __shared__ __align__(8) uint64_t full_bar[kStages];
  __shared__ float red[2][2][kStreamThreads / 32];
  __shared__ int abort_word;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, nthr = blockDim.x, warps = nthr >> 5;
  const int count = p.M / VE;
  const uint32_t row_bytes = (uint32_t)count * 16u, stage_bytes = p.r ? 2 * row_bytes : row_bytes;
  const int grid = gridDim.x;
  auto bar = [&](int s) { return ptx::smem_u32(&full_bar[s]); };
  auto fetch = [&](int s, int64_t row) {       // one thread
    const uint32_t dst = ptx::smem_u32(smem + (size_t)s * stage_bytes);
    const uint64_t policy = ptx::policy_evict_first();
    ptx::mbar_arrive_expect_tx(bar(s), stage_bytes);
    ptx::bulk_load_g2s_hint(dst, static_cast<const uint4*>(p.x) + row * count, row_bytes, bar(s), policy);
    if (p.r)
      ptx::bulk_load_g2s_hint(dst + row_bytes, static_cast<const uint4*>(p.r) + row * count, row_bytes, bar(s), policy);
  };
  if (tid == 0) {
    abort_word = 0;
    for (int s = 0; s < kStages; ++s) ptx::mbar_init(bar(s), 1);
    ptx::fence_mbar_init();
  }
  ptx::grid_launch_next();
  ptx::grid_wait();      // from here on this kernel reads and writes global memory
  if (tid == 0) {
    for (int s = 0; s < kStages; ++s)
      if (blockIdx.x + (int64_t)s * grid < p.T) fetch(s, blockIdx.x + (int64_t)s * grid);
  }
  uint4 gw[ITEMS];
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const int c = tid + i * nthr;
    if (c < count) gw[i] = static_cast<const uint4*>(p.gain)[c];
  }
  __syncthreads();
  int s = 0, it = 0;
  uint32_t parity = 0;
  for (int64_t row = blockIdx.x; row < p.T; row += grid, ++it) {
    const Row<VE, false> at(row, p.T, p.M);
    const bool ok = ptx::mbar_wait_bounded(bar(s), parity, &abort_word, timeout_ns);
    const uint4* sx = reinterpret_cast<const uint4*>(smem + (size_t)s * stage_bytes);
    const uint4* sr = sx + count;
    float v[ITEMS][VE];
    float ss = 0.f, am = 0.f;
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const int c = tid + i * nthr;
      if (c < count) {
        unpack<T>(sx[c], v[i]);
        if (p.r) {
          float r[VE];
          unpack<T>(sr[c], r);
#pragma unroll
          for (int e = 0; e < VE; ++e) v[i][e] += r[e];
        }
      }
    }
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const int c = tid + i * nthr;
      if (c < count) {
        float g[VE];
        unpack<T>(gw[i], g);
        first_step<T, false>(p, at, c, v[i], g, true, ss, am);
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
            ptx::mbar_wait_cluster_timed(bar(b), b < s ? parity ^ 1u : parity,
                                         timeout_ns > 10000000ull ? timeout_ns : 10000000ull);
        }
      }
      return;
    }
    if (tid == 0 && row + (int64_t)kStages * grid < p.T) fetch(s, row + (int64_t)kStages * grid);
    ss = lane < warps ? red[it & 1][0][lane] : 0.f;
    am = lane < warps ? red[it & 1][1][lane] : 0.f;
    warp_reduce(ss, am);
    const float inv = rsqrtf(ss * p.inv_m + p.eps);
    const int k = scale_exponent(am * inv);
    const float up = f8::pow2(-k);
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const int c = tid + i * nthr;
      if (c < count) second_step<T, false>(p, at, c, v[i], inv, up);
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
// 16-byte aligned, and rows too wide for the registers of a block (above 17,408 elements).
// Element by element and twice over the row: 2048 x 18432 bf16 with a residual 131 us, where
// 2048 x 16384 takes 47; 2048 x 7168 one element off 56 us, aligned 21.
template <typename T>
__global__ void __launch_bounds__(1024) add_rmsnorm_any_kernel(const Params p) {
  __shared__ float red[2][32];
  ptx::grid_launch_next();
  ptx::grid_wait();      // from here on this kernel reads and writes global memory
  const int64_t at = (int64_t)blockIdx.x * p.M;
  const T* x = static_cast<const T*>(p.x) + at;
  const T* r = p.r ? static_cast<const T*>(p.r) + at : nullptr;
  const T* g = static_cast<const T*>(p.gain);
  auto sum = [&](int c) {      // (not x + 0 without r: that would lose the sign of -0)
    const float v = to_f32<T>(x[c]);
    return r ? v + to_f32<T>(r[c]) : v;
  };
  float ss = 0.f, am = 0.f;
  for (int c = threadIdx.x; c < p.M; c += blockDim.x) {
    const float s = sum(c);
    ss += s * s;
    am = fmaxf(am, fabsf(g ? s * to_f32<T>(g[c]) : s));
  }
  block_reduce(ss, am, red);
  const float inv = g ? rsqrtf(ss * p.inv_m + p.eps) : 1.f;
  const int k = scale_exponent(am * inv);
  const float up = f8::pow2(-k);
  for (int c = threadIdx.x; c < p.M; c += blockDim.x) {
    const float s = sum(c);
    if (p.r_out) static_cast<T*>(p.r_out)[at + c] = from_f32<T>(s);
    const float y = g ? (s * to_f32<T>(g[c])) * inv : s;
    if (p.y) static_cast<T*>(p.y)[at + c] = from_f32<T>(y);
    if (p.codes) p.codes[at + c] = (uint8_t)f8::to_e4m3x2(y * up, 0.f);
  }
  if (p.codes && threadIdx.x == 0) p.scales[blockIdx.x] = (uint8_t)(k + 127);
}

}  // namespace rms
}  // namespace mla
