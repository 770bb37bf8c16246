// What a product ends in: y = residual + act(sum + bias), in fp32 on the fp32
// sum, rounded once.  It costs its reads of bias and residual and no pass of its
// own over y: one token on 4096 x 4096 with a residual 5.5 us where the product
// alone takes 5.0; 1024 tokens on 11008 x 4096 with bias and GELU 106 us, with a
// residual 102, the product alone 93 (short runs at 1965 MHz; seconds of calls at
// the power cap, 1.65 - 1.75 GHz: 120, 117 and 106).  What is left is the last tile's
// epilogue, which no products hide.
#pragma once

#include "common.cuh"
#include "internal.h"

namespace qk {

struct EpiArgs {
  const uint16_t* bias;       // [N] or null
  const uint16_t* residual;   // [M, N] or null; may be y (an element is read by the thread that writes it)
  int act;                    // QMM_ACT_*
};

inline EpiArgs epi_args(const Problem& p) {
  return EpiArgs{static_cast<const uint16_t*>(p.bias), static_cast<const uint16_t*>(p.residual), p.act};
}

template <bool BF16>
__device__ __forceinline__ float epi_load(const uint16_t* p) {
  // plain loads: the residual may be written by this grid
  if constexpr (BF16) return __uint_as_float((uint32_t)*p << 16);
  else return __half2float(__ushort_as_half(*p));
}

// GELU v Phi(v) = max(v, 0) - |v| Phi(-|v|): no cancellation in the lower tail, whose
// values bf16 can hold down to v = -13.  Phi(-x) = R(x) e^(-x^2 / 2), and R falls from
// 1/2 like 0.4 / x: a polynomial of degree 8 in t = 1 / (1 + 0.3 x) without a constant
// term, fitted to the smallest relative error on 0 .. 14 (iteratively reweighted least
// squares, 1.5e-7).  In all the value is off by less than 2^-19 + 2^-23 v^2 of itself,
// the second term the rounding of the exponent.  (The rational form 7.1.26 of
// Abramowitz and Stegun, three terms shorter, is good to 1.5e-7 absolutely but only to
// 4e-3 of the value at v = -6, half a step of bf16 by itself; these three terms cost
// 1 % of a call of 1024 tokens.)  17 instructions, where erfcf's branches made the
// epilogue of a tile slower than its products.
__device__ __forceinline__ float gelu(float v) {
  const float x = fminf(fabsf(v), 1e4f);                  // inf 0 is not needed below
  const float t = __fdividef(1.0f, fmaf(0.3f, x, 1.0f));
  float p = fmaf(3.567477688e-2f, t, -1.572031081e-1f);
  p = fmaf(p, t, 2.063535303e-1f);
  p = fmaf(p, t, -5.368367210e-2f);
  p = fmaf(p, t, 1.285616457e-1f);
  p = fmaf(p, t, 9.991348535e-2f);
  p = fmaf(p, t, 1.207539588e-1f);
  p = fmaf(p, t, 1.196293011e-1f);
  return (v > 0.0f ? v : (v == v ? 0.0f : v)) - x * (p * t * __expf(-0.5f * x * x));
}

template <int ACT>
__device__ __forceinline__ float epi_act(float v) {
  if constexpr (ACT == QMM_ACT_RELU) return v > 0.0f ? v : (v == v ? 0.0f : v);
  if constexpr (ACT == QMM_ACT_GELU) return gelu(v);
  if constexpr (ACT == QMM_ACT_GELU_TANH)
    // 0.5 v (1 + tanh u) = v / (1 + e^-2u), u = sqrt(2 / pi) (v + 0.044715 v^3)
    return __fdividef(v, 1.0f + __expf(-1.5957691216f * (v + 0.044715f * v * v * v)));
  if constexpr (ACT == QMM_ACT_SILU) return silu(v);
  return v;
}

// N values at once: v[i] + bias(i), activated, + the residual of element at(i) of
// y.  The choices are made once; at(i) is always an element of y (that of another
// value where value i is none), so that the residual's loads need no branches and
// are in flight together.
template <bool BF16, int N, class Bias, class At>
__device__ __forceinline__ void epi_apply(const EpiArgs& e, float (&v)[N], Bias&& bias, At&& at) {
  uint16_t res[N];
#pragma unroll
  for (int i = 0; i < N; ++i) res[i] = 0;
  if (e.residual) {
#pragma unroll
    for (int i = 0; i < N; ++i) res[i] = e.residual[at(i)];
  }
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] += bias(i);
  switch (e.act) {   // the same for every thread of the grid
    case QMM_ACT_RELU:
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = epi_act<QMM_ACT_RELU>(v[i]);
      break;
    case QMM_ACT_GELU:
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = epi_act<QMM_ACT_GELU>(v[i]);
      break;
    case QMM_ACT_GELU_TANH:
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = epi_act<QMM_ACT_GELU_TANH>(v[i]);
      break;
    case QMM_ACT_SILU:
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = epi_act<QMM_ACT_SILU>(v[i]);
      break;
    default: break;
  }
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] += epi_load<BF16>(&res[i]);
}

}  // namespace qk
