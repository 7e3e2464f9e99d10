// Selective scan: the form for one token, the split of a problem over the
// machine, the sums over partial rows, and the dispatch by type.
#include <algorithm>

#include "sc_ssm.cuh"

namespace scg {

cudaError_t launch_ssm_bf16(const SsmParams&, const SsmPlan&, int*, cudaStream_t);
cudaError_t launch_ssm_f16(const SsmParams&, const SsmPlan&, int*, cudaStream_t);
cudaError_t launch_ssm_f32(const SsmParams&, const SsmPlan&, int*, cudaStream_t);
cudaError_t launch_ssm_grad_bf16(const SsmParams&, const SsmPlan&, int*, cudaStream_t);
cudaError_t launch_ssm_grad_f16(const SsmParams&, const SsmPlan&, int*, cudaStream_t);
cudaError_t launch_ssm_grad_f32(const SsmParams&, const SsmPlan&, int*, cudaStream_t);

namespace {

constexpr int kStepNT = 256;
constexpr long long kSms = 152;

long long ceil_div(long long a, long long b) { return (a + b - 1) / b; }

// dA, dD and dbias: the partial rows of the batch and the chunks, in order.
__global__ void __launch_bounds__(256) ssm_sum_kernel(SsmParams p, int np) {
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x, na = p.channels * p.states;
    const float* src;
    float* dst;
    long long step;
    if (i < na) {
        src = p.part_a + (i % p.states / 4 * p.channels + i / p.states) * 4 + i % p.states % 4;
        step = p.channels * np;
        dst = p.dA + i;
    } else if (i < na + 2 * p.channels) {
        const long long c = (i - na) % p.channels, which = (i - na) / p.channels;
        src = p.part_d + which * p.batch * p.chunks * p.channels + c;
        step = p.channels;
        dst = which ? p.ddt_bias : p.dD;
        if (!dst) return;
        dst += c;
    } else {
        return;
    }
    const long long rows = p.batch * p.chunks;
    float sum = 0.0f;
    long long r = 0;
    for (; r + 8 <= rows; r += 8) {
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = __ldg(src + (r + j) * step);
        sum += ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
    }
    for (; r < rows; ++r) sum += __ldg(src + r * step);
    *dst = sum;
}

// One token: S lanes per channel, four states each; the state is read and
// written once, the floor of the call.
template <class T, int S, bool kVec>
__global__ void __launch_bounds__(kStepNT) ssm_step_kernel(SsmParams p, unsigned cblocks) {
    const long long b = blockIdx.x / cblocks;
    const long long e = (long long)(blockIdx.x % cblocks) * (kStepNT / S) + threadIdx.x / S;
    const int n0 = 4 * (threadIdx.x % S);
    const bool live = e < p.channels;
    const long long slot = p.slots ? (long long)__ldg(p.slots + b) : b;
    T* yp = static_cast<T*>(p.y) + b * p.y_batch + e;
    if (slot < 0 || slot >= p.pool_rows) {  // the whole row
        if (live && n0 == 0) *yp = from_f32<T>(0.0f);
        return;
    }
    float sum = 0.0f, x = 0.0f;
    if (live) {
        const long long group = e / (p.channels / p.groups);
        float* hp = p.pool + (slot * p.channels + e) * p.states + n0;
        const float* Ap = p.A + e * p.states + n0;
        const T* Bp = static_cast<const T*>(p.B) + b * p.B_batch + group * p.B_group + n0;
        const T* Cp = static_cast<const T*>(p.C) + b * p.C_batch + group * p.C_group + n0;
        float h[4], A[4], B[4], C[4];
        const bool on = n0 < p.states;
        if constexpr (kVec) {  // states a multiple of 4
            float4 hv = make_float4(0.0f, 0.0f, 0.0f, 0.0f), av = hv;
            Vec<T, 4> bv, cv;
            bv.zero();
            cv.zero();
            if (on) {
                hv = *reinterpret_cast<const float4*>(hp);
                av = __ldg(reinterpret_cast<const float4*>(Ap));
                bv.load(Bp);
                cv.load(Cp);
            }
            h[0] = hv.x; h[1] = hv.y; h[2] = hv.z; h[3] = hv.w;
            A[0] = av.x; A[1] = av.y; A[2] = av.z; A[3] = av.w;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                B[k] = bv.get(k);
                C[k] = cv.get(k);
            }
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const bool in = n0 + k < p.states;
                h[k] = in ? hp[k] : 0.0f;
                A[k] = in ? __ldg(Ap + k) : 0.0f;
                B[k] = in ? to_f32(__ldg(Bp + k)) : 0.0f;
                C[k] = in ? to_f32(__ldg(Cp + k)) : 0.0f;
            }
        }
        x = to_f32(__ldg(static_cast<const T*>(p.x) + b * p.x_batch + e));
        float d = to_f32(__ldg(static_cast<const T*>(p.dt) + b * p.dt_batch + e)) + (p.dt_bias ? __ldg(p.dt_bias + e) : 0.0f);
        if (p.softplus) d = softplus(d);
        const float u = d * x, d2 = d * kLog2e;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            h[k] = fmaf(ex2(d2 * A[k]), h[k], u * B[k]);
            sum = fmaf(C[k], h[k], sum);
        }
        if constexpr (kVec) {
            if (on) *reinterpret_cast<float4*>(hp) = make_float4(h[0], h[1], h[2], h[3]);
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (n0 + k < p.states) hp[k] = h[k];
        }
    }
#pragma unroll
    for (int m = 1; m < S; m <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
    if (live && n0 == 0) {
        float y = fmaf(p.D ? __ldg(p.D + e) : 0.0f, x, sum);
        if (p.z) {
            const float z = to_f32(__ldg(static_cast<const T*>(p.z) + b * p.z_batch + e));
            y *= z * sigmoid(z);
        }
        *yp = from_f32<T>(y);
    }
}

template <class T, int S>
cudaError_t step_lanes(const SsmParams& p, cudaStream_t s) {
    const unsigned cblocks = (unsigned)ceil_div(p.channels, kStepNT / S), grid = cblocks * (unsigned)p.batch;
    if (p.vec) ssm_step_kernel<T, S, true><<<grid, kStepNT, 0, s>>>(p, cblocks);
    else ssm_step_kernel<T, S, false><<<grid, kStepNT, 0, s>>>(p, cblocks);
    return cudaGetLastError();
}

template <class T>
cudaError_t step_of(const SsmParams& p, cudaStream_t s) {
    switch (ssm_lanes(p.states)) {
    case 2: return step_lanes<T, 2>(p, s);
    case 4: return step_lanes<T, 4>(p, s);
    case 8: return step_lanes<T, 8>(p, s);
    default: return step_lanes<T, 16>(p, s);
    }
}

}  // namespace

int ssm_lanes(long long states) { return states <= 8 ? 2 : states <= 16 ? 4 : states <= 32 ? 8 : 16; }

SsmPlan ssm_plan(long long batch, long long length, long long channels, long long states, long long groups, bool grad) {
    SsmPlan g{};
    g.lanes = ssm_lanes(states);
    const long long per = channels / groups, ch = g.lanes <= 4 ? 32 : g.lanes == 8 ? 16 : 8;
    const long long block = ch * (g.lanes == 16 ? 2 : 4), np = 4 * g.lanes;
    g.blocks_per_group = ceil_div(per, block);
    const long long warps = batch * groups * ceil_div(per, ch), tiles = ceil_div(length, kTile);
    // Split where even one warp per SM sub-partition is not there.
    long long chunks = 1;
    if (warps < 4 * kSms) chunks = std::min(ceil_div(8 * kSms, warps), std::max(tiles / 4, 1ll));
    g.chunk_tiles = ceil_div(tiles, chunks);
    g.chunks = (int)ceil_div(tiles, g.chunk_tiles);
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t o = at;
        at += (bytes + 255) / 256 * 256;
        return o;
    };
    const size_t rows = (size_t)batch * g.chunks;
    if (g.chunks > 1) {
        g.carry = take(rows * channels * np * 4);
        g.sum_d = take(rows * channels * 4);
        g.cut = take(rows);
    }
    if (grad) {
        g.part_bc = take((size_t)(g.blocks_per_group * groups) * batch * length * 2 * np * 4);
        g.part_a = take(rows * channels * np * 4);
        g.part_d = take(2 * rows * channels * 4);
    }
    g.total = at;
    return g;
}

cudaError_t launch_ssm(int dtype, const SsmParams& p, const SsmPlan& plan, cudaStream_t s) {
    int launches = 0;
    cudaError_t e = cudaErrorInvalidValue;
    switch (dtype) {
    case SC_F32: e = launch_ssm_f32(p, plan, &launches, s); break;
    case SC_F16: e = launch_ssm_f16(p, plan, &launches, s); break;
    case SC_BF16: e = launch_ssm_bf16(p, plan, &launches, s); break;
    default: break;
    }
    count_launches(launches);
    return e;
}

cudaError_t launch_ssm_grad(int dtype, const SsmParams& p, const SsmPlan& plan, cudaStream_t s) {
    int launches = 0;
    cudaError_t e = cudaErrorInvalidValue;
    switch (dtype) {
    case SC_F32: e = launch_ssm_grad_f32(p, plan, &launches, s); break;
    case SC_F16: e = launch_ssm_grad_f16(p, plan, &launches, s); break;
    case SC_BF16: e = launch_ssm_grad_bf16(p, plan, &launches, s); break;
    default: break;
    }
    count_launches(launches);
    if (e != cudaSuccess) return e;
    const long long n = p.channels * (p.states + 2);
    ssm_sum_kernel<<<(unsigned)ceil_div(n, 256), 256, 0, s>>>(p, 4 * plan.lanes);
    return cudaGetLastError();
}

cudaError_t launch_ssm_step(int dtype, const SsmParams& p, cudaStream_t s) {
    count_launches(1);
    switch (dtype) {
    case SC_F32: return step_of<float>(p, s);
    case SC_F16: return step_of<f16>(p, s);
    case SC_BF16: return step_of<bf16>(p, s);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace scg
