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

__device__ __forceinline__ float epi_act(int act, float v) {
  switch (act) {   // the same for every thread of the grid
    case QMM_ACT_RELU: return v > 0.0f ? v : (v == v ? 0.0f : v);
    // erfc: no cancellation in the negative tail
    case QMM_ACT_GELU: return 0.5f * v * erfcf(v * -0.70710678118f);
    case QMM_ACT_GELU_TANH:
      // 0.5 v (1 + tanh u) = v / (1 + e^-2u), u = sqrt(2 / pi) (v + 0.044715 v^3)
      return v / (1.0f + __expf(-1.5957691216f * (v + 0.044715f * v * v * v)));
    case QMM_ACT_SILU: return silu(v);
    default: return v;
  }
}

// row: the weight row (bias); at: the element of y.
template <bool BF16>
__device__ __forceinline__ float epi_apply(const EpiArgs& e, float v, int row, size_t at) {
  if (e.bias) v += epi_load<BF16>(e.bias + row);
  v = epi_act(e.act, v);
  if (e.residual) v += epi_load<BF16>(e.residual + at);
  return v;
}

}  // namespace qk
