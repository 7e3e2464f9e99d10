// The gated recurrence's kernels for bfloat16 elements.
#include "sc_gated.cuh"

namespace scg {
cudaError_t launch_gated_bf16(const GatedParams& p, bool grad, cudaStream_t s) { return launch_gated_as<bf16>(p, grad, s); }
}  // namespace scg
