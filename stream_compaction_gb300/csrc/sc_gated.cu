// The gated recurrence: dispatch by element type, and its form for one token
// (sc_gated.cuh has the kernels).
#include "sc_gated.cuh"

namespace scg {

namespace {
cudaError_t by_type(int dtype, const GatedParams& p, bool grad, cudaStream_t s) {
    return dtype == SC_F32 ? launch_gated_f32(p, grad, s) : dtype == SC_F16 ? launch_gated_f16(p, grad, s)
                                                                           : launch_gated_bf16(p, grad, s);
}
}  // namespace

cudaError_t launch_gated(int dtype, const GatedParams& p, cudaStream_t s) { return by_type(dtype, p, false, s); }
cudaError_t launch_gated_grad(int dtype, const GatedParams& p, cudaStream_t s) { return by_type(dtype, p, true, s); }
cudaError_t launch_gated_step(int dtype, const GatedParams& p, cudaStream_t s) {
    return dtype == SC_F32 ? launch_gated_step_as<float>(p, s) : dtype == SC_F16 ? launch_gated_step_as<f16>(p, s)
                                                                                : launch_gated_step_as<bf16>(p, s);
}

}  // namespace scg
