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

constexpr int kStepNT = 128;

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
// written once, the floor of the call.  A thread serves R rows of the batch, so
// that R states are under way in it, A is read once for them, and the work per
// row and channel (softplus, gate) is done once: by lane r of the channel's
// lanes for row r, the others get d and d x from it.  The loads' latency bounds it
// (half of a warp's time).  256 x 4096 x 16 states, a tenth of the rows idle: 42 us
// with one row a thread, whose S lanes all did that work; 25 to 30 so (129 MB, 4.3
// to 5.2 TB/s); one sequence of 2048 channels: 5 us, a chain of loads.
template <class T, int S, bool kVec>
__global__ void __launch_bounds__(kStepNT) ssm_step_kernel(SsmParams p, unsigned cblocks) {
    constexpr int R = S < 4 ? S : 4;
    const long long b0 = (long long)(blockIdx.x / cblocks) * R;
    const long long e = (long long)(blockIdx.x % cblocks) * (kStepNT / S) + threadIdx.x / S;
    const int s = threadIdx.x % S, n0 = 4 * s, first = (int)(threadIdx.x & 31) - s;  // first: the channel's first lane
    const bool live = e < p.channels, on = live && n0 < p.states;
    // the row that this lane does the elements of
    const long long b = b0 + s % R;
    int slot = -1;
    if (live && b < p.batch) {
        const long long q = p.slots ? (long long)__ldg(p.slots + b) : b;
        slot = q >= 0 && q < p.pool_rows ? (int)q : -1;
    }
    const bool run = slot >= 0;
    const long long group = live ? e / (p.channels / p.groups) : 0;
    const float x = run ? to_f32(__ldg(static_cast<const T*>(p.x) + b * p.x_batch + e)) : 0.0f;
    float d = run ? to_f32(__ldg(static_cast<const T*>(p.dt) + b * p.dt_batch + e)) : 0.0f;
    const float z = run && p.z ? to_f32(__ldg(static_cast<const T*>(p.z) + b * p.z_batch + e)) : 0.0f;
    const float bias = run && p.dt_bias ? __ldg(p.dt_bias + e) : 0.0f, D = run && p.D ? __ldg(p.D + e) : 0.0f;
    float A[4] = {0.0f, 0.0f, 0.0f, 0.0f}, h[R][4], B[R][4], C[R][4];
    float* hp[R];
    const float* Ap = p.A + e * p.states + n0;
    if constexpr (kVec) {  // states a multiple of 4
        if (on) {
            const float4 av = __ldg(reinterpret_cast<const float4*>(Ap));
            A[0] = rate(av.x); A[1] = rate(av.y); A[2] = rate(av.z); A[3] = rate(av.w);
        }
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (live && n0 + k < p.states) A[k] = rate(__ldg(Ap + k));
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int row = __shfl_sync(0xffffffffu, slot, first + r);
        hp[r] = row >= 0 && on ? p.pool + ((long long)row * p.channels + e) * p.states + n0 : nullptr;
        const T* Bp = static_cast<const T*>(p.B) + (b0 + r) * p.B_batch + group * p.B_group + n0;
        const T* Cp = static_cast<const T*>(p.C) + (b0 + r) * p.C_batch + group * p.C_group + n0;
        if constexpr (kVec) {
            float4 hv = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            Vec<T, 4> bv, cv;
            bv.zero();
            cv.zero();
            if (hp[r]) {
                hv = *reinterpret_cast<const float4*>(hp[r]);
                bv.load(Bp);
                cv.load(Cp);
            }
            h[r][0] = hv.x; h[r][1] = hv.y; h[r][2] = hv.z; h[r][3] = hv.w;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                B[r][k] = bv.get(k);
                C[r][k] = cv.get(k);
            }
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const bool in = hp[r] && n0 + k < p.states;
                h[r][k] = in ? hp[r][k] : 0.0f;
                B[r][k] = in ? to_f32(__ldg(Bp + k)) : 0.0f;
                C[r][k] = in ? to_f32(__ldg(Cp + k)) : 0.0f;
            }
        }
    }
    d += bias;
    if (p.softplus) d = softplus<T>(d);
    const float u = d * x;
    float sum[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const float dr = __shfl_sync(0xffffffffu, d, first + r), ur = __shfl_sync(0xffffffffu, u, first + r);
        sum[r] = 0.0f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            h[r][k] = fmaf(decay(dr, A[k]), h[r][k], ur * B[r][k]);
            // (a state past the last would be infinity times 0 where d or d x is infinite)
            sum[r] = kVec || n0 + k < p.states ? fmaf(C[r][k], h[r][k], sum[r]) : sum[r];
        }
        if constexpr (kVec) {
            if (!on) sum[r] = 0.0f;
            if (hp[r]) *reinterpret_cast<float4*>(hp[r]) = make_float4(h[r][0], h[r][1], h[r][2], h[r][3]);
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (hp[r] && n0 + k < p.states) hp[r][k] = h[r][k];
        }
    }
    // over the channel's lanes; lane r keeps row r's
    float y;
    const bool b0s = s & 1, b1s = s & 2;
    const float t0 = (b0s ? sum[1] : sum[0]) + __shfl_xor_sync(0xffffffffu, b0s ? sum[0] : sum[1], 1);
    if constexpr (R == 4) {
        const float t1 = (b0s ? sum[3] : sum[2]) + __shfl_xor_sync(0xffffffffu, b0s ? sum[2] : sum[3], 1);
        y = (b1s ? t1 : t0) + __shfl_xor_sync(0xffffffffu, b1s ? t0 : t1, 2);
#pragma unroll
        for (int m = 4; m < S; m <<= 1) y += __shfl_xor_sync(0xffffffffu, y, m);
    } else {
        y = t0;
    }
    if (live && s < R && b < p.batch) {
        y = fmaf(D, x, y);
        if (p.z) y *= z * sigmoid<T>(z);
        static_cast<T*>(p.y)[b * p.y_batch + e] = from_f32<T>(run ? y : 0.0f);  // a row that sits out: 0
    }
}

template <class T, int S>
cudaError_t step_lanes(const SsmParams& p, cudaStream_t s) {
    const unsigned cblocks = (unsigned)ceil_div(p.channels, kStepNT / S);
    const unsigned grid = cblocks * (unsigned)ceil_div(p.batch, S < 4 ? S : 4);
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

// Chunks of the backward pass, of `ctas` CTAs each where the machine holds
// `slots`, by the least of what a token costs: the places that stay empty in the
// last wave, a chunk's start (about a tile's time, and a twentieth for each chunk's
// part that it folds), and the first kernel, which takes a quarter of the second's
// time for all tokens but the first chunk's.  4 x 4096 x 4096, 128 CTAs, with the
// forward pass: 2.87 ms whole, 1.98 in 2 chunks (256 of 304 places), 1.87 in 7
// (896 in three waves of 304), 1.88 in 14.
long long back_chunks(long long ctas, long long slots, long long tiles) {
    long long best = 1;
    double least = 0;
    const long long most = ctas > 0 ? std::min(std::max(slots / ctas, 24ll), tiles / 2) : 1;
    for (long long c = 1; c <= most; ++c) {
        const long long per = ceil_div(tiles, c), n = ceil_div(tiles, per);
        const double waves = (double)(ceil_div(ctas * n, slots) * slots) / (double)(ctas * n);
        const double cost = waves * (1 + (1 + 0.05 * n) / per) + 0.25 * (n - 1) / n;
        if (c == 1 || cost < least) {
            least = cost;
            best = n;
        }
    }
    return best;
}

}  // namespace

int ssm_lanes(long long states) { return states <= 8 ? 2 : states <= 16 ? 4 : states <= 32 ? 8 : 16; }

SsmPlan ssm_plan(long long batch, long long length, long long channels, long long states, long long groups, bool grad) {
    SsmPlan g{};
    g.lanes = ssm_lanes(states);
    const long long sms = seq_sms(), per = channels / groups, ch = g.lanes <= 4 ? 32 : g.lanes == 8 ? 16 : 8;
    const long long block = ch * (g.lanes == 16 ? 2 : 4), np = 4 * g.lanes;
    g.blocks_per_group = ceil_div(per, block);
    const long long warps = batch * groups * ceil_div(per, ch), tiles = ceil_div(length, kTile);
    // Forward: a pair of warps alone takes about 90 ns a token, and an SM's pairs
    // together 27 ns each, so three or four keep it busy; a split costs the
    // recurrence nearly twice.  Below 1.7 pairs an SM it pays, and then into about
    // 7 pairs an SM (1 x 4096 x 4096, 128 pairs: 192 us in 4 chunks, 167 in 8 to 10;
    // 4 x 4096 x 4096, 512 pairs, with gradient: 2.17 ms whole, 2.29 in 2).
    // Backward: see back_chunks; a first kernel walks the chunks in runs, about 4
    // warps' an SM (4 x 4096 x 4096 in 2 chunks, with the forward pass: 2.03 ms with
    // a run a chunk, 1.98 so, and the same with 8 or 16; 2 x 1000 x 1002 with 24
    // states: 209 us, 206, 213 and 234).
    long long chunks = 1;
    if (grad) {
        chunks = back_chunks(g.blocks_per_group * groups * batch, (g.lanes == 16 ? 3 : 2) * sms, tiles);
    } else if (10 * warps < 17 * sms) {
        chunks = std::min(ceil_div(7 * sms, warps), std::max(tiles / 4, 1ll));
    }
    g.chunk_tiles = ceil_div(tiles, chunks);
    const long long split = grad && chunks > 1 ? std::min(ceil_div(4 * sms, warps * (chunks - 1)), g.chunk_tiles) : 1;
    g.run_tiles = ceil_div(g.chunk_tiles, split);
    g.chunk_tiles = g.run_tiles * split;
    g.chunks = (int)ceil_div(tiles, g.chunk_tiles);
    g.runs = (int)ceil_div(tiles, g.run_tiles);
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t o = at;
        at += (bytes + 255) / 256 * 256;
        return o;
    };
    const size_t rows = (size_t)batch * g.chunks, runs = (size_t)batch * g.runs;
    if (g.chunks > 1) {
        g.carry = take(runs * channels * np * 4);
        g.sum_d = take(runs * channels * 4);
        g.cut = take(runs);
    }
    if (grad) {
        g.part_bc = take((size_t)(g.blocks_per_group * groups) * batch * length * 2 * np * 4);
        g.part_a = take(rows * channels * np * 4);
        g.part_d = take(2 * rows * channels * 4);
        if (states != np) g.odd = take(rows * (size_t)(g.blocks_per_group * groups));
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
