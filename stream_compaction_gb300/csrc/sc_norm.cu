// The norm: plans, dispatch by element type, and the sum of the gradient's partial
// rows (sc_norm.cuh has the kernels of the rows).
#include "sc_norm.cuh"

namespace scg {

namespace {

// Column c of dweight (blockIdx.y == 0) or dbias: kSumRows threads take every
// kSumRows-th row of partial sums, then their sums are added in order.  Launched while
// the kernel before it ends, it waits for that one's rows.
constexpr int kSumCols = 32, kSumRows = 32, kSumAhead = 8;
__global__ void __launch_bounds__(kSumCols* kSumRows) norm_parameters_kernel(NormParams p) {
    __shared__ float s_part[kSumRows][kSumCols];
    const int tx = threadIdx.x % kSumCols, ty = threadIdx.x / kSumCols;
    const long long c = (long long)blockIdx.x * kSumCols + tx;
    const int which = blockIdx.y;
    float* to = which ? p.dbias : p.dweight;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (!to) return;
    float sum = 0.0f;
    if (c < p.channels) {
        const float* from = p.partials + which * p.channels + c;
        for (long long i0 = ty; i0 < p.parts; i0 += kSumAhead * kSumRows) {
            float v[kSumAhead];
#pragma unroll
            for (int k = 0; k < kSumAhead; ++k) {
                const long long i = i0 + k * kSumRows;
                v[k] = i < p.parts ? from[i * 2 * p.channels] : 0.0f;
            }
#pragma unroll
            for (int k = 0; k < kSumAhead; ++k) sum += v[k];
        }
    }
    s_part[ty][tx] = sum;
    __syncthreads();
    if (ty == 0 && c < p.channels) {
        float all = 0.0f;
#pragma unroll
        for (int k = 0; k < kSumRows; ++k) all += s_part[k][tx];
        to[c] = all;
    }
}

cudaError_t by_type(int dtype, NormParams& p, bool grad, cudaStream_t s) {
    return dtype == SC_F32 ? launch_norm_f32(p, grad, s) : dtype == SC_F16 ? launch_norm_f16(p, grad, s)
                                                                          : launch_norm_bf16(p, grad, s);
}

}  // namespace

cudaError_t launch_norm(int dtype, NormParams p, cudaStream_t s) { return by_type(dtype, p, false, s); }

// One row of partial sums for each CTA of the gradient's kernel, at most three an SM and a
// row each; of wide rows, one for each part of the columns' sums.
size_t norm_grad_scratch(long long rows, long long channels) {
    const long long parts = channels > kRowMax ? kColumnParts : 3 * seq_sms();
    return (size_t)std::min(rows, parts) * 2 * channels * sizeof(float);
}

cudaError_t launch_norm_grad(int dtype, NormParams p, cudaStream_t s) {
    const cudaError_t e = by_type(dtype, p, true, s);
    if (e != cudaSuccess || !p.partials) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)((p.channels + kSumCols - 1) / kSumCols), 2);
    cfg.blockDim = dim3(kSumCols * kSumRows);
    cfg.stream = s;
    cudaLaunchAttribute a{};
    a.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    a.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &a;
    cfg.numAttrs = 1;
    count_launches(1);
    return cudaLaunchKernelEx(&cfg, norm_parameters_kernel, p);
}

}  // namespace scg
