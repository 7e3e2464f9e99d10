// The gated recurrence's kernels for float32 elements.
#include "sc_gated.cuh"

namespace scg {
cudaError_t launch_gated_f32(const GatedParams& p, bool grad, cudaStream_t s) { return launch_gated_as<float>(p, grad, s); }
}  // namespace scg
