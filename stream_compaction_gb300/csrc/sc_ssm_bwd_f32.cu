// Gradient of the selective scan, f32 activations.
#include "sc_ssm_bwd.cuh"

namespace scg {
cudaError_t launch_ssm_grad_f32(const SsmParams& p, const SsmPlan& plan, int* launches, cudaStream_t s) {
    return ssm_back_type<float>(p, plan, launches, s);
}
}  // namespace scg
