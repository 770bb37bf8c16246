// Tensor-core path: the plan of a call, and its plain kernels (tc.cuh).
#include "tc.cuh"

namespace qk {

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  if (!fn) {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    else
      cudaGetLastError();
  }
  return fn;
}

// Combinations the tensor path takes: 4-bit codes without the zero-point
// options.  fp16 activations: the operand is fp16((q - z) s) or fp16(T s), one
// rounding of 2^-11.  bf16 activations: per-row scales keep the exact integer
// q - z (the scale multiplies the fp32 result); group scales and tables split
// each weight into bf16 hi + lo parts (SPLIT above).
bool tc_supported(int bits, int mode, bool bf16, int group) {
  (void)bf16;
  (void)group;
  return bits == 4 && !zero_opts(mode);
}

TcPlan plan_tc(int M, int N, int K, int mode, bool bf16, int group, int sms) {
  TcPlan p{};
  p.bn = M <= 64 ? 64 : (M <= 128 ? 128 : 256);
  // two k blocks per unit where the kernel has them: 64 tokens unless a
  // table meets split operands; 128 tokens without a table or a split; 256
  // tokens SYM only, and only for more than one token tile (with a single one,
  // M = 256, the two A / B stages measured 1-2.5% slower than three of 64
  // columns).  A K that ends mid-unit is zero-filled.
  const bool split = bf16 && (group != -1 || mode == kLUT);
  const bool table = mode == kLUT;
  if (p.bn == 64)
    p.ku = (split && table) ? 1 : 2;
  else if (p.bn == 128)
    p.ku = (split || table) ? 1 : 2;
  else
    p.ku = (!split && mode == kSYM && M > 256) ? 2 : 1;
  p.tiles_n = (N + kRowsTile - 1) / kRowsTile;
  p.tiles_m = (M + p.bn - 1) / p.bn;
  p.nkb = (K / kKB + p.ku - 1) / p.ku;
  const long long units = (long long)p.tiles_n * p.tiles_m * p.nkb;
  long long ctas = sms;   // one CTA per SM (shared memory bound)
  if (ctas > units) ctas = units;
  p.ctas = (int)ctas;
  const int tiles = p.tiles_n * p.tiles_m;
  const bool partial = !(units % ctas == 0 && (units / ctas) % p.nkb == 0);
  p.ws_bytes = partial ? ((size_t)tiles * 4 + 255) / 256 * 256 +
                           (size_t)2 * p.ctas * p.bn * kRowsTile * sizeof(float)
                     : 0;
  return p;
}

cudaError_t launch_tc(const Problem& pr, const TcPlan& plan, void* workspace,
                      long long wait_limit, cudaStream_t stream) {
  return pr.epilogue ? launch_tc_epi(pr, plan, workspace, wait_limit, stream)
                     : launch_tc_any<false>(pr, plan, workspace, wait_limit, stream);
}

unsigned tc_read_and_clear_error() {
  const unsigned a = read_and_clear_tc_error(), b = tc_epi_read_and_clear_error();
  return a | b;
}

}  // namespace qk
