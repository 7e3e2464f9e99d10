// The norm's kernels for float16 rows.
#include "sc_norm.cuh"

namespace scg {
cudaError_t launch_norm_f16(NormParams& p, bool grad, cudaStream_t s) { return launch_norm_as<f16>(p, grad, s); }
}  // namespace scg
