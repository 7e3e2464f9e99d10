// Gradient of the selective scan, bf16 activations.
#include "sc_ssm_bwd.cuh"

namespace scg {
cudaError_t launch_ssm_grad_bf16(const SsmParams& p, const SsmPlan& plan, int* launches, cudaStream_t s) {
    return ssm_back_type<bf16>(p, plan, launches, s);
}
}  // namespace scg
