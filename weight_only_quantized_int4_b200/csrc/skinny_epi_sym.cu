// Decode path: the SYM kernels that end in bias, activation and residual.
#include "skinny.cuh"

namespace qk {

cudaError_t launch_skinny_epi_sym(const Problem& pr, const SkinnyPlan& plan, void* workspace,
                               cudaStream_t stream) {
  return launch_skinny_t<true, kSYM>(pr, plan, workspace, stream);
}

}  // namespace qk
