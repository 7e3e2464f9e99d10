// The gated recurrence's kernels for float16 elements.
#include "sc_gated.cuh"

namespace scg {
cudaError_t launch_gated_f16(const GatedParams& p, bool grad, cudaStream_t s) { return launch_gated_as<f16>(p, grad, s); }
}  // namespace scg
