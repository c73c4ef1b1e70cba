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
#pragma once

#include "common.cuh"
#include "fp8_kernels.cuh"

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

// VE consecutive elements of a row (VE * sizeof(T) bytes, aligned to that) <-> fp32.
template <int BYTES> struct Word;
template <> struct Word<16> { using type = uint4; };
template <> struct Word<8> { using type = uint2; };
template <> struct Word<4> { using type = uint32_t; };
template <> struct Word<2> { using type = uint16_t; };
template <> struct Word<1> { using type = uint8_t; };

template <typename T, int VE>
__device__ __forceinline__ void load(const void* base, int64_t chunk, float (&v)[VE]) {
  using W = typename Word<VE * (int)sizeof(T)>::type;
  const W w = reinterpret_cast<const W*>(base)[chunk];
  const T* e = reinterpret_cast<const T*>(&w);
#pragma unroll
  for (int i = 0; i < VE; ++i) v[i] = to_f32<T>(e[i]);
}
template <typename T, int VE>
__device__ __forceinline__ void store(void* base, int64_t chunk, const float (&v)[VE]) {
  using W = typename Word<VE * (int)sizeof(T)>::type;
  W w;
  T* e = reinterpret_cast<T*>(&w);
#pragma unroll
  for (int i = 0; i < VE; ++i) e[i] = from_f32<T>(v[i]);
  reinterpret_cast<W*>(base)[chunk] = w;
}
// VE codes of v * up (VE a power of two up to 8).
template <int VE>
__device__ __forceinline__ void store_codes(uint8_t* base, int64_t chunk, const float (&v)[VE], float up) {
  using W = typename Word<VE>::type;
  W w;
  uint8_t* e = reinterpret_cast<uint8_t*>(&w);
  if constexpr (VE == 1) {
    e[0] = (uint8_t)f8::to_e4m3x2(v[0] * up, 0.f);
  } else {
#pragma unroll
    for (int i = 0; i < VE; i += 2) reinterpret_cast<uint16_t*>(e)[i / 2] = (uint16_t)f8::to_e4m3x2(v[i] * up, v[i + 1] * up);
  }
  reinterpret_cast<W*>(base)[chunk] = w;
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

// One row per warp (WARP: blocks of kWarpRows rows) or per block; every thread holds ITEMS
// chunks of VE elements, chunk c of the row in thread c % threads. A thread keeps its
// elements and their gains (2 ITEMS VE registers), so blocks of 1024 threads hold up to 16
// elements a thread and blocks of 512 up to 32.
__host__ __device__ constexpr int max_threads(int ept) { return ept <= 16 ? 1024 : 512; }

template <typename T, int VE, int ITEMS, bool WARP>
__global__ void __launch_bounds__(WARP ? 32 * kWarpRows : max_threads(VE * ITEMS))
add_rmsnorm_kernel(const Params p) {
  __shared__ float red[2][32];
  const int nthr = WARP ? 32 : blockDim.x;
  const int tid = WARP ? (threadIdx.x & 31) : threadIdx.x;
  const int64_t row = WARP ? (int64_t)blockIdx.x * kWarpRows + (threadIdx.x >> 5) : blockIdx.x;
  if (WARP && row >= p.T) return;
  const int chunks = p.M / VE;
  const int64_t base = row * chunks;
  float v[ITEMS][VE], g[ITEMS][VE];
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const int c = tid + i * nthr;
    if (c < chunks) load<T, VE>(p.x, base + c, v[i]);
  }
  if (p.r) {
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const int c = tid + i * nthr;
      if (c < chunks) {
        float r[VE];
        load<T, VE>(p.r, base + c, r);
#pragma unroll
        for (int e = 0; e < VE; ++e) v[i][e] += r[e];
      }
    }
  }
  if (p.gain) {
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const int c = tid + i * nthr;
      if (c < chunks) load<T, VE>(p.gain, c, g[i]);
    }
  }
  float ss = 0.f, am = 0.f;
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const int c = tid + i * nthr;
    if (c < chunks) {
      if (p.r_out) store<T, VE>(p.r_out, base + c, v[i]);
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        ss += v[i][e] * v[i][e];
        if (p.gain) v[i][e] *= g[i][e];
        am = fmaxf(am, fabsf(v[i][e]));
      }
    }
  }
  if (WARP) warp_reduce(ss, am);
  else block_reduce(ss, am, red);
  if (p.gain) {
    const float inv = 1.f / sqrtf(ss / (float)p.M + p.eps);
    am *= inv;
#pragma unroll
    for (int i = 0; i < ITEMS; ++i)
#pragma unroll
      for (int e = 0; e < VE; ++e) v[i][e] *= inv;
  }
  const int k = scale_exponent(am);
  const float up = f8::pow2(-k);
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const int c = tid + i * nthr;
    if (c < chunks) {
      if (p.y) store<T, VE>(p.y, base + c, v[i]);
      if (p.codes) store_codes<VE>(p.codes, base + c, v[i], up);
    }
  }
  if (p.codes && tid == 0) p.scales[row] = (uint8_t)(k + 127);
}

// Any width and alignment: one block per row, two passes over it (the second reads again
// what the first summed; r_out and y are written in the second, element by element by the
// thread that read them, so they may be r's and x's own buffers). For rows too wide for the
// registers of a block.
template <typename T>
__global__ void __launch_bounds__(1024) add_rmsnorm_wide_kernel(const Params p) {
  __shared__ float red[2][32];
  const T* x = static_cast<const T*>(p.x) + (int64_t)blockIdx.x * p.M;
  const T* r = p.r ? static_cast<const T*>(p.r) + (int64_t)blockIdx.x * p.M : nullptr;
  const T* g = static_cast<const T*>(p.gain);
  const int64_t at = (int64_t)blockIdx.x * p.M;
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
