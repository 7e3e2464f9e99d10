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

}  // namespace

cudaError_t launch_norm(int dtype, const NormParams& p, cudaStream_t s) {
    return dtype == SC_F32 ? launch_norm_f32(p, false, s) : dtype == SC_F16 ? launch_norm_f16(p, false, s)
                                                                          : launch_norm_bf16(p, false, s);
}

// One row of partial sums for each CTA of the gradient's kernel: as many as the
// machine holds at once (kResident), fewer where there are fewer rows.  Rows beyond
// kRowMax are summed by columns, in 32 parts.
NormGradPlan norm_grad_plan(int dtype, long long rows, long long channels) {
    NormGradPlan g{};
    if (channels > kRowMax) {
        g.parts = std::min<long long>(rows, 32);
    } else {
        const long long n = (channels + (dtype == SC_F32 ? 4 : 8) - 1) / (dtype == SC_F32 ? 4 : 8);
        // the kernel's groups of threads and CTAs an SM, by width as in by_width
        const long long lanes = n <= 8 ? 8 : n <= 16 ? 16 : n <= 64 ? 32 : n <= 128 ? 64 : n <= 256 ? 128 : n <= 512 ? 256 : n <= 1024 ? 512 : 1024;
        const long long threads = std::max<long long>(lanes, 256), groups = threads / lanes;
        g.parts = std::min((rows + groups - 1) / groups, seq_sms() * (threads == 256 ? 2 : 1));
    }
    g.partials = 0;
    g.total = (size_t)g.parts * 2 * channels * sizeof(float);
    return g;
}

cudaError_t launch_norm_grad(int dtype, const NormParams& p, cudaStream_t s) {
    const cudaError_t e = dtype == SC_F32 ? launch_norm_f32(p, true, s) : dtype == SC_F16 ? launch_norm_f16(p, true, s)
                                                                                         : launch_norm_bf16(p, true, s);
    if (e != cudaSuccess || !p.partials) return e;
    const dim3 grid((unsigned)((p.channels + kSumCols - 1) / kSumCols), 2);
    norm_parameters_kernel<<<grid, kSumCols * kSumRows, 0, s>>>(p);
    count_launches(1);
    return cudaGetLastError();
}

}  // namespace scg
