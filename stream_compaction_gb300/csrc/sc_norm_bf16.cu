// The norm's kernels for bfloat16 rows.
#include "sc_norm.cuh"

namespace scg {
cudaError_t launch_norm_bf16(NormParams& p, bool grad, cudaStream_t s) { return launch_norm_as<bf16>(p, grad, s); }
}  // namespace scg
