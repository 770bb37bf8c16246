// Tensor-core path: the kernels that end in bias, activation and residual.
#include "tc.cuh"

namespace qk {

cudaError_t launch_tc_epi(const Problem& pr, const TcPlan& plan, void* workspace,
                          long long wait_limit, cudaStream_t stream) {
  return launch_tc_any<true>(pr, plan, workspace, wait_limit, stream);
}

unsigned tc_epi_read_and_clear_error() { return read_and_clear_tc_error(); }

}  // namespace qk
