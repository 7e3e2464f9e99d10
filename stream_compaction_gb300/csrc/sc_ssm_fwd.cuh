// Forward selective scan.
//
// Per token, channel and state: one exponential, two products and two
// multiply-adds; per token and channel 4 elements of memory.  With 16 states the
// exponentials bound it (32 a clock and SM), close to the memory's time.  The
// tile of a warp is staged through shared memory by the warp itself (no CTA
// barrier): the next tile's elements travel to registers while this one is
// computed.
//
// Where rows x channels give the machine too few warps the length is split
// into chunks: a first kernel scans each chunk from a zero state (kSummary: no
// C, no y), and the second folds the chunks before its own, h = exp(A * sum of
// d) * h + (their result), and scans its chunk from there.  The exponentials
// are computed twice then, which is why the split waits for idle SMs.
#pragma once
#include "sc_ssm.cuh"

namespace scg {

template <class T, class G, bool kVec, bool kSummary>
__global__ void __launch_bounds__(G::kThreads) ssm_kernel(SsmParams p, long long blocks_per_group, int grid_chunks) {
    using Rows = TileRows<T, G, kVec>;
    using States = TileStates<T, G, kVec>;
    __shared__ alignas(16) float s_d[G::kWarps][kTile * G::CH], s_u[G::kWarps][kTile * G::CH];
    __shared__ alignas(16) float s_y[kSummary ? 1 : G::kWarps][kSummary ? 4 : kTile * G::CH];
    __shared__ alignas(16) float2 s_B[G::kWarps][kTile * G::NP];
    __shared__ alignas(16) float2 s_C[kSummary ? 1 : G::kWarps][kSummary ? 2 : kTile * G::NP];
    const SsmPlace<G> at(p, blocks_per_group, grid_chunks);
    if (at.left <= 0) return;  // warps of a CTA do not meet
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, left = (int)at.left;
    const int s = lane % G::S, c = lane / G::S;
    const long long b = at.b;

    float raw[G::CPL][4];
    f2 A2[G::PC][4], h[G::PC][4];
    load_lane_of<G>(p.A + at.ch0 * p.states, p.states, left, lane, raw);
    to_pairs<G>(raw, kLog2e, A2);
    if constexpr (kSummary) {
#pragma unroll
        for (int q = 0; q < G::PC; ++q)
#pragma unroll
            for (int k = 0; k < 4; ++k) h[q][k] = 0ull;
    } else {
        load_lane_of<G>(p.state ? p.state + (b * p.channels + at.ch0) * p.states : nullptr, p.states, left, lane, raw);
        to_pairs<G>(raw, 1.0f, h);
        for (long long j = 0; j < at.chunk; ++j) fold_chunk<G>(p, A2, b, j, at.ch0, left, lane, h);
    }
    float bias[Rows::kChannels], D[Rows::kChannels];
#pragma unroll
    for (int i = 0; i < Rows::kChannels; ++i) {
        const int ch = Rows::ch(i, lane);
        bias[i] = p.dt_bias && ch < left ? p.dt_bias[at.ch0 + ch] : 0.0f;
        D[i] = p.D && ch < left ? p.D[at.ch0 + ch] : 0.0f;
    }

    const long long tiles = (p.length + kTile - 1) / kTile;
    const long long tile0 = at.chunk * p.chunk_tiles;
    const long long tile1 = tile0 + p.chunk_tiles < tiles ? tile0 + p.chunk_tiles : tiles;
    const T* xp = static_cast<const T*>(p.x) + b * p.x_batch + at.ch0;
    const T* dtp = static_cast<const T*>(p.dt) + b * p.dt_batch + at.ch0;
    const T* zp = p.z && !kSummary ? static_cast<const T*>(p.z) + b * p.z_batch + at.ch0 : nullptr;
    const T* Bp = static_cast<const T*>(p.B) + b * p.B_batch + at.group * p.B_group;
    const T* Cp = static_cast<const T*>(p.C) + b * p.C_batch + at.group * p.C_group;
    T* yp = kSummary ? nullptr : static_cast<T*>(p.y) + b * p.y_batch + at.ch0;
    const uint8_t* heads = p.heads ? p.heads + b * p.length : nullptr;

    Rows x, dt, z;
    States B, C;
    auto fetch = [&](long long tile) {
        const long long t0 = tile * kTile;
        const int nt = (int)(p.length - t0 < kTile ? p.length - t0 : kTile);
        x.load(xp + t0 * p.x_token, p.x_token, nt, left, lane);
        dt.load(dtp + t0 * p.dt_token, p.dt_token, nt, left, lane);
        B.load(Bp + t0 * p.B_token, p.B_token, nt, (int)p.states, lane);
        if constexpr (!kSummary) {
            if (zp) z.load(zp + t0 * p.z_token, p.z_token, nt, left, lane);
            C.load(Cp + t0 * p.C_token, p.C_token, nt, (int)p.states, lane);
        }
    };
    f2 dsum[G::PC];
#pragma unroll
    for (int q = 0; q < G::PC; ++q) dsum[q] = 0ull;
    unsigned cut = 0;
    if (tile0 < tile1) fetch(tile0);
    for (long long tile = tile0; tile < tile1; ++tile) {
        const long long t0 = tile * kTile;
        const int nt = (int)(p.length - t0 < kTile ? p.length - t0 : kTile);
        const unsigned hm = tile_heads(heads, t0, nt, lane);
        cut |= hm;
        {
            float fd[Rows::kCount], fu[Rows::kCount];
#pragma unroll
            for (int i = 0; i < Rows::kCount; ++i) {
                const float v = dt.get(i) + bias[Rows::channel_of(i)];
                // d of a token past the end is 0, whatever the bias
                fd[i] = Rows::valid(i, lane, nt, left) ? (p.softplus ? softplus(v) : v) : 0.0f;
                fu[i] = fd[i] * x.get(i);
            }
            Rows::to_shared(s_d[warp], fd, lane);
            Rows::to_shared(s_u[warp], fu, lane);
            B.to_shared(s_B[warp], lane);
            if constexpr (!kSummary) C.to_shared(s_C[warp], lane);
        }
        const Rows xc = x, zc = z;
        if (!kSummary && p.saved)
            store_lane<G>(p.saved + ((b * tiles + tile) * p.channels + at.ch0) * G::NP, left, lane, h);
        __syncwarp();
        if (tile + 1 < tile1) fetch(tile + 1);
#pragma unroll 4
        for (int t = 0; t < kTile; ++t) {
            f2 d[G::PC], u[G::PC], Bv[4], acc[G::PC];
            read_channels<G>(s_d[warp] + t * G::CH + G::CPL * c, d);
            read_channels<G>(s_u[warp] + t * G::CH + G::CPL * c, u);
            read_states(s_B[warp] + t * G::NP + 4 * s, Bv);
            if (hm >> t & 1u) {
#pragma unroll
                for (int q = 0; q < G::PC; ++q)
#pragma unroll
                    for (int k = 0; k < 4; ++k) h[q][k] = 0ull;
            }
#pragma unroll
            for (int q = 0; q < G::PC; ++q)
#pragma unroll
                for (int k = 0; k < 4; ++k) h[q][k] = fma2(ex2_2(mul2(d[q], A2[q][k])), h[q][k], mul2(u[q], Bv[k]));
            if constexpr (kSummary) {
#pragma unroll
                for (int q = 0; q < G::PC; ++q) dsum[q] = add2(dsum[q], d[q]);
            } else {
                f2 Cv[4];
                read_states(s_C[warp] + t * G::NP + 4 * s, Cv);
#pragma unroll
                for (int q = 0; q < G::PC; ++q) {
                    acc[q] = mul2(Cv[0], h[q][0]);
#pragma unroll
                    for (int k = 1; k < 4; ++k) acc[q] = fma2(Cv[k], h[q][k], acc[q]);
                }
                const float y = sum_states<G>(acc, lane);
                if (s < G::CPL) s_y[warp][t * G::CH + G::CPL * c + s] = y;
            }
        }
        __syncwarp();
        if constexpr (!kSummary) {
            float y[Rows::kCount];
            Rows::from_shared(s_y[warp], y, lane);
#pragma unroll
            for (int i = 0; i < Rows::kCount; ++i) {
                y[i] = fmaf(D[Rows::channel_of(i)], xc.get(i), y[i]);
                if (zp) y[i] *= zc.get(i) * sigmoid(zc.get(i));
            }
            Rows::store(yp + t0 * p.y_token, p.y_token, y, nt, left, lane);
        }
    }
    if constexpr (kSummary) {
        const long long row = b * p.chunks + at.chunk;
        store_lane<G>(p.carry + (row * p.channels + at.ch0) * G::NP, left, lane, h);
        if (s == 0)
#pragma unroll
            for (int j = 0; j < G::CPL; ++j)
                if (G::CPL * c + j < left)
                    p.sum_d[row * p.channels + at.ch0 + G::CPL * c + j] = j & 1 ? hi2(dsum[j / 2]) : lo2(dsum[j / 2]);
        if (at.cblock == 0 && warp == 0 && lane == 0) p.cut[row] = cut != 0;
    } else if (p.final_state && tile1 == tiles) {
        store_lane_of<G>(p.final_state + (b * p.channels + at.ch0) * p.states, p.states, left, lane, h);
    }
}

template <class T, class G, bool kVec>
cudaError_t ssm_of(const SsmParams& p, const SsmPlan& plan, int* launches, cudaStream_t s) {
    const long long ncb = plan.blocks_per_group * p.groups;
    *launches = 1;
    if (p.chunks > 1) {  // nobody waits for the last chunk's summary
        ssm_kernel<T, G, kVec, true><<<(unsigned)(ncb * (p.chunks - 1) * p.batch), G::kThreads, 0, s>>>(
            p, plan.blocks_per_group, p.chunks - 1);
        *launches = 2;
    }
    ssm_kernel<T, G, kVec, false><<<(unsigned)(ncb * p.chunks * p.batch), G::kThreads, 0, s>>>(
        p, plan.blocks_per_group, p.chunks);
    return cudaGetLastError();
}

template <class T>
cudaError_t ssm_type(const SsmParams& p, const SsmPlan& plan, int* launches, cudaStream_t s) {
    switch (plan.lanes) {
    case 2: return p.vec ? ssm_of<T, Geo<2>, true>(p, plan, launches, s) : ssm_of<T, Geo<2>, false>(p, plan, launches, s);
    case 4: return p.vec ? ssm_of<T, Geo<4>, true>(p, plan, launches, s) : ssm_of<T, Geo<4>, false>(p, plan, launches, s);
    case 8: return p.vec ? ssm_of<T, Geo<8>, true>(p, plan, launches, s) : ssm_of<T, Geo<8>, false>(p, plan, launches, s);
    case 16:
        return p.vec ? ssm_of<T, Geo<16>, true>(p, plan, launches, s) : ssm_of<T, Geo<16>, false>(p, plan, launches, s);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace scg
