// What a product ends in: y = residual + act(sum + bias), in fp32 on the fp32
// sum, rounded once.
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

// Phi(v), the normal distribution function, as 1/2 erfc(-v / sqrt 2) by the rational
// approximation 7.1.26 of Abramowitz and Stegun (absolute error below 1.5e-7, no
// cancellation in the lower tail): about 15 instructions, where erfcf's branches
// made the epilogue of a tile slower than its products.
__device__ __forceinline__ float normal_cdf(float v) {
  const float x = fabsf(v) * 0.70710678118f;
  const float t = __fdividef(1.0f, fmaf(0.3275911f, x, 1.0f));
  float p = fmaf(1.061405429f, t, -1.453152027f);
  p = fmaf(p, t, 1.421413741f);
  p = fmaf(p, t, -0.284496736f);
  p = fmaf(p, t, 0.254829592f);
  const float half_erfc = 0.5f * p * t * __expf(-x * x);   // of |v| / sqrt 2
  return v < 0.0f ? half_erfc : 1.0f - half_erfc;
}

template <int ACT>
__device__ __forceinline__ float epi_act(float v) {
  if constexpr (ACT == QMM_ACT_RELU) return v > 0.0f ? v : (v == v ? 0.0f : v);
  if constexpr (ACT == QMM_ACT_GELU) return v * normal_cdf(v);
  if constexpr (ACT == QMM_ACT_GELU_TANH)
    // 0.5 v (1 + tanh u) = v / (1 + e^-2u), u = sqrt(2 / pi) (v + 0.044715 v^3)
    return __fdividef(v, 1.0f + __expf(-1.5957691216f * (v + 0.044715f * v * v * v)));
  if constexpr (ACT == QMM_ACT_SILU) return silu(v);
  return v;
}

// N values at once, v[i] of weight row row(i) and element at(i) of y where ok(i): the choices of activation, bias and residual
// are made once, and the residual's loads are in flight together.
template <bool BF16, int N, class Ok, class Row, class At>
__device__ __forceinline__ void epi_apply(const EpiArgs& e, float (&v)[N], Ok&& ok, Row&& row, At&& at) {
  float res[N];
#pragma unroll
  for (int i = 0; i < N; ++i) res[i] = 0.0f;
  if (e.residual) {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (ok(i)) res[i] = epi_load<BF16>(e.residual + at(i));
  }
  if (e.bias) {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (ok(i)) v[i] += epi_load<BF16>(e.bias + row(i));
  }
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
  for (int i = 0; i < N; ++i) v[i] += res[i];
}

}  // namespace qk
