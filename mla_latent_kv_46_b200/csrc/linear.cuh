// linear.cuh -- the layer's projections: out = residual + mul * act(x W^T + bias), with
// W stored out x in. The epilogue every kernel shares, and the CUDA-core kernel for
// geometries the tensor-core kernels (linear_tc.cuh) do not take.
//
// Sums are fp32; bias, activation, mul and residual are applied to the fp32 sum and the
// result is rounded once, to bf16. 8-bit operands are E4M3 codes with one power-of-two
// scale per row of x and of W (see fp8_kernels.cuh): the codes' products are summed and the
// two scales multiply the sum, W's first: exact, but where that first product is subnormal (below
// 2^-126) and off by up to 2^-150, 2^-143 behind x's scale of at most 2^7: half a step of a bf16
// result is 2^-134 there or more.
#pragma once

#include "common.cuh"
#include "fp8_kernels.cuh"
#include "ptx.cuh"

namespace mla {
namespace lin {

enum : int { kActNone = 0, kActSigmoid = 1, kActSilu = 2, kActGelu = 3 };

struct Params {
  const __nv_bfloat16* bias;   // [N] or null
  const __nv_bfloat16* mul;    // [T][N] or null
  const __nv_bfloat16* res;    // [T][N] or null
  __nv_bfloat16* out;          // [T][N]
  const uint8_t* xs;           // [T] scale bytes (8-bit operands)
  const uint8_t* ws;           // [N]
  int32_t T, N, K, act;
  bool octs;                   // eight neighbouring features can be moved in one access
  int32_t nt, stages;          // tensor-core kernels: tokens per tile, stages of the ring
  uint64_t timeout_ns;
};

// 2^(byte - 127); the bytes the quantisers write are 1 .. 134.
__device__ __forceinline__ float scale_of(uint8_t b) { return __uint_as_float((uint32_t)b << 23); }

// exp by ex2.approx and the quotient by rcp.approx, a few units in 2^-22 off (the result is
// rounded to bf16, 2^-9): a full division took a third of the epilogue's instructions. The quotient
// is 0 once 1 + e^-v passes 2^126, for sums below about -87.3, where sigmoid is below 1.2e-38 and silu
// below 1.1e-36 in magnitude (in fp32 the formulas give 0 from -88.7 on, where e^-v overflows).
__device__ __forceinline__ float sigmoid(float v) { return __fdividef(1.f, 1.f + __expf(-v)); }
__device__ __forceinline__ float silu(float v) { return __fdividef(v, 1.f + __expf(-v)); }
// v Phi(v). The lower tail Q(x) = Phi(-x) = e^(-x^2 / 2) R(x) for x = |v|, where R falls smoothly
// from 1/2 to 0 (like 0.4 / x): a polynomial in t = 1 / (1 + 0.35 x) without a constant term,
// fitted here to R by weighted least squares on x <= 14 (relative error 3.2e-8; above 13.2 the
// exponential is 0 in fp32). The exponent's roundings (x^2, and its product with log2(e) / 2)
// are carried to first order, or they would be 1e-5 of the tail. All in all 1e-6 of the result;
// erfcf took twice the time of a 4685 x 2802 output's whole epilogue.
// Two elements at a time: all but the exponential, the quotient and the choice of the side
// are paired instructions.
__device__ __forceinline__ void gelu(float& v0, float& v1) {
  using ptx::F2;
  auto both = [](float c) { return ptx::f2(c, c); };
  const float x0 = fminf(fabsf(v0), 20.f), x1 = fminf(fabsf(v1), 20.f);      // above, Q is 0 as well; keeps x^2 finite
  const F2 x = ptx::f2(x0, x1), minus = both(-1.f);
  float d0, d1;
  ptx::split(ptx::fma2(both(0.35f), x, both(1.f)), d0, d1);
  const F2 t = ptx::f2(__fdividef(1.f, d0), __fdividef(1.f, d1));
  F2 r = both(-0.029146350920200348f);
  r = ptx::fma2(r, t, both(0.143973708152771f));
  r = ptx::fma2(r, t, both(-0.25571832060813904f));
  r = ptx::fma2(r, t, both(0.1591787040233612f));
  r = ptx::fma2(r, t, both(-0.02311287634074688f));
  r = ptx::fma2(r, t, both(0.10550924390554428f));
  r = ptx::fma2(r, t, both(0.11983256787061691f));
  r = ptx::fma2(r, t, both(0.13986191153526306f));
  r = ptx::fma2(r, t, both(0.13962140679359436f));
  // s = -x^2 and y = s log2(e) / 2, each with what its rounding left
  const F2 c = both(0.72134752f), c_lo = both(9.629815167500055e-09f);
  const F2 s = ptx::mul2(x, ptx::mul2(x, minus)), s_lo = ptx::fma2(x, x, s);
  const F2 y = ptx::mul2(s, c), y_lo = ptx::fma2(s, c_lo, ptx::fma2(s, c, ptx::mul2(y, minus)));
  float y0, y1, q0, q1, u0, u1;
  ptx::split(y, y0, y1);
  const F2 e = ptx::f2(ptx::ex2(y0), ptx::ex2(y1));
  const F2 q = ptx::mul2(ptx::mul2(e, ptx::mul2(r, t)),
                         ptx::fma2(both(-0.5f), s_lo, ptx::fma2(both(0.69314718f), y_lo, both(1.f))));
  ptx::split(q, q0, q1);
  ptx::split(ptx::fma2(q, minus, both(1.f)), u0, u1);
  v0 *= v0 > 0.f ? u0 : q0;
  v1 *= v1 > 0.f ? u1 : q1;
}
// All of a thread's elements: one branch, straight code behind it (a branch per element of an
// unrolled epilogue ran out of the instruction cache).
template <int CNT>
__device__ __forceinline__ void activate(float (&v)[CNT], int act) {
  if (act == kActSigmoid) {
#pragma unroll
    for (int j = 0; j < CNT; ++j) v[j] = sigmoid(v[j]);
  } else if (act == kActSilu) {
#pragma unroll
    for (int j = 0; j < CNT; ++j) v[j] = silu(v[j]);
  } else if (act == kActGelu) {
#pragma unroll
    for (int j = 0; j + 1 < CNT; j += 2) gelu(v[j], v[j + 1]);
    if (CNT % 2) {
      float other = 0.f;
      gelu(v[CNT - 1], other);
    }
  }
}

// One output element from its fp32 sum (8-bit operands: already times both scales).
__device__ __forceinline__ void finish(const Params& p, float v, int64_t t, int32_t n, float bias) {
  const int64_t at = t * p.N + n;
  float y[1] = {v + bias};
  activate(y, p.act);
  if (p.mul) y[0] *= __bfloat162float(p.mul[at]);
  if (p.res) y[0] += __bfloat162float(p.res[at]);
  p.out[at] = __float2bfloat16_rn(y[0]);
}

// ------------------------------------------------------------------ CUDA cores
// A block of 256 threads computes 64 tokens x 64 features, 16 K elements at a time through
// shared memory, 4 x 4 sums per thread. Any size and alignment. Blocks are numbered along
// the token tiles first, so that neighbours share a weight tile.
constexpr int kTile = 64, kStep = 16;

template <bool F8>
__global__ void __launch_bounds__(256) linear_simt_kernel(const void* __restrict__ x, const void* __restrict__ W,
                                                          const Params p) {
  __shared__ float sx[kStep][kTile + 4], sw[kStep][kTile + 4];
  const unsigned tiles_t = ((unsigned)p.T + kTile - 1) / kTile;      // T may be all of 31 bits
  const int t0 = (int)(blockIdx.x % tiles_t) * kTile, n0 = (int)(blockIdx.x / tiles_t) * kTile;
  const int tid = threadIdx.x;
  const int ty = tid / 16, tx = tid % 16;     // tokens 4 ty .., features tx, tx + 16, ..
  auto fetch = [&](const void* base, int64_t row, int64_t rows, int k) -> float {
    if (row >= rows || k >= p.K) return 0.f;
    const int64_t at = row * p.K + k;
    if constexpr (F8) return f8::from_e4m3x2(static_cast<const uint8_t*>(base)[at]).x;
    else return __bfloat162float(static_cast<const __nv_bfloat16*>(base)[at]);
  };
  float acc[4][4] = {};
  for (int k0 = 0; k0 < p.K; k0 += kStep) {
#pragma unroll
    for (int i = 0; i < kTile * kStep / 256; ++i) {
      const int e = tid + 256 * i, r = e / kStep, k = e % kStep;
      sx[k][r] = fetch(x, t0 + r, p.T, k0 + k);
      sw[k][r] = fetch(W, n0 + r, p.N, k0 + k);
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kStep; ++k) {
      float a[4], b[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) a[i] = sx[k][4 * ty + i];
#pragma unroll
      for (int j = 0; j < 4; ++j) b[j] = sw[k][tx + 16 * j];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] += a[i] * b[j];
    }
    __syncthreads();
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int n = n0 + tx + 16 * j;
    if (n >= p.N) continue;
    const float bias = p.bias ? __bfloat162float(p.bias[n]) : 0.f;
    const float ws = F8 ? scale_of(p.ws[n]) : 1.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = t0 + 4 * ty + i;
      if (t >= p.T) continue;
      float v = acc[i][j];
      if (F8) v = v * ws * scale_of(p.xs[t]);
      finish(p, v, t, n, bias);
    }
  }
}

}  // namespace lin
}  // namespace mla
