// The norm's kernels for float32 rows.
#include "sc_norm.cuh"

namespace scg {
cudaError_t launch_norm_f32(NormParams& p, bool grad, cudaStream_t s) { return launch_norm_as<float>(p, grad, s); }
}  // namespace scg
