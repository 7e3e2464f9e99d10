// The norm: plans, dispatch by element type, and the sum of the gradient's partial
// rows (sc_norm.cuh has the kernels of the rows).
#include "sc_norm.cuh"

namespace scg {

namespace {

// Column c of dweight (blockIdx.y == 0) or dbias: kSumRows threads take every
// kSumRows-th row of partial sums, then their sums are added in order.
constexpr int kSumCols = 32, kSumRows = 16;
__global__ void __launch_bounds__(kSumCols* kSumRows) norm_parameters_kernel(NormParams p) {
    __shared__ float s_part[kSumRows][kSumCols];
    const int tx = threadIdx.x % kSumCols, ty = threadIdx.x / kSumCols;
    const long long c = (long long)blockIdx.x * kSumCols + tx;
    const int which = blockIdx.y;
    float* to = which ? p.dbias : p.dweight;
    if (!to) return;
    float sum = 0.0f;
    if (c < p.channels) {
        const float* from = p.partials + which * p.channels + c;
        long long i = ty;
        for (; i + 3 * kSumRows < p.parts; i += 4 * kSumRows) {
            float v[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) v[k] = from[(i + k * kSumRows) * 2 * p.channels];
#pragma unroll
            for (int k = 0; k < 4; ++k) sum += v[k];
        }
        for (; i < p.parts; i += kSumRows) sum += from[i * 2 * p.channels];
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

// One row of partial sums for each CTA of the gradient's kernel: at most two an SM, and
// a row each.
size_t norm_grad_scratch(long long rows, long long channels) {
    return (size_t)std::min(rows, std::max<long long>(2 * seq_sms(), kColumnParts)) * 2 * channels * sizeof(float);
}

cudaError_t launch_norm_grad(int dtype, NormParams p, cudaStream_t s) {
    const cudaError_t e = by_type(dtype, p, true, s);
    if (e != cudaSuccess || !p.partials) return e;
    const dim3 grid((unsigned)((p.channels + kSumCols - 1) / kSumCols), 2);
    norm_parameters_kernel<<<grid, kSumCols * kSumRows, 0, s>>>(p);
    count_launches(1);
    return cudaGetLastError();
}

}  // namespace scg
