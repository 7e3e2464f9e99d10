// Gradient of the selective scan.
//
// With q = exp(d A), y0 = sum_n C h + D x, y = y0 z sig(z), and g the gradient
// by y0 (dy z sig(z); dy without a gate):
//
//   dh[t]   = q[t+1] dh[t+1] + C[t] g[t]          (the first term dropped where
//                                                  a segment starts at t + 1)
//   dC[t]   = sum_e g h[t]          dB[t] = sum_e dh[t] d x     (e: the group's channels)
//   r       = dh[t] q[t] h[t-1]     the derivative by the exponent d A
//   dA      = sum_t r d             dd = sum_n r A + x sum_n dh B
//   dx      = d sum_n dh B + D g    dD = sum g x
//   ddt     = dd sig(dt + bias)     (softplus), dbias its sum
//   dz      = dy y0 sig(z) (1 + z (1 - sig(z)))
//
// A warp walks its channels' tokens backwards in tiles of kTile, from the state
// that the forward pass saved at each tile's start.  Nothing of the states is
// kept per token: a tile's states are recomputed, first in one run that leaves
// the states at its quarters in shared memory, then quarter by quarter, where q
// and q h[t-1] of four tokens stay in registers for the way back (in shared
// memory they would cost more accesses than the second exponential).  The sums
// over states go across the S lanes of a channel, those over channels across
// the other lanes, then over the CTA's warps in shared memory, and the rest in
// a second kernel over the CTAs' partial rows; each in a fixed order.
// Instruction issue bounds it, then the exponentials.
//
// Rows too few for the machine: the length is split as in the forward pass,
// with a first kernel that runs each chunk backwards from zero (kSummary).
#pragma once
#include "sc_ssm.cuh"

namespace scg {

constexpr int kQuarter = 4;

// A warp's part of the shared memory, in floats.
template <class G>
struct BwdShared {
    static constexpr int kRow = kTile * G::CH, kStates = kTile * G::NP * 2, kHold = G::CPL * 4 * 32;
    static constexpr int d = 0, u = kRow, g = 2 * kRow, y = 3 * kRow, gu = 4 * kRow, ga = 5 * kRow;
    static constexpr int B = 6 * kRow, C = B + kStates, h = C + kStates, bc = h + kTile / kQuarter * kHold;
    static constexpr int kFloats = bc + kTile * 2 * G::NP;
    static constexpr size_t kBytes = (size_t)kFloats * 4 * G::kWarps;
};

// dh of a chunk's first token, taken one token further back, with nothing
// coming in from behind; and the chunk's sum of d.
template <class T, class G, bool kVec>
__global__ void __launch_bounds__(G::kThreads) ssm_back_summary_kernel(SsmParams p, long long blocks_per_group,
                                                                       int grid_chunks) {
    using Rows = TileRows<T, G, kVec>;
    using States = TileStates<T, G, kVec>;
    __shared__ alignas(16) float s_d[G::kWarps][kTile * G::CH], s_g[G::kWarps][kTile * G::CH];
    __shared__ alignas(16) float2 s_C[G::kWarps][kTile * G::NP];
    SsmPlace<G> at(p, blocks_per_group, grid_chunks);
    if (at.left <= 0) return;
    at.chunk += 1;  // nobody waits for the first chunk's
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, left = (int)at.left;
    const int s = lane % G::S, c = lane / G::S;
    const long long b = at.b;
    float raw[G::CPL][4];
    f2 A2[G::PC][4], dh[G::PC][4], dsum[G::PC];
    load_lane_of<G>(p.A + at.ch0 * p.states, p.states, left, lane, raw);
    to_pairs<G>(raw, kLog2e, A2);
#pragma unroll
    for (int q = 0; q < G::PC; ++q) {
        dsum[q] = 0ull;
#pragma unroll
        for (int k = 0; k < 4; ++k) dh[q][k] = 0ull;
    }
    float bias[Rows::kChannels];
#pragma unroll
    for (int i = 0; i < Rows::kChannels; ++i) {
        const int ch = Rows::ch(i, lane);
        bias[i] = p.dt_bias && ch < left ? p.dt_bias[at.ch0 + ch] : 0.0f;
    }
    const long long tiles = (p.length + kTile - 1) / kTile;
    const long long tile0 = at.chunk * p.chunk_tiles;
    const long long tile1 = tile0 + p.chunk_tiles < tiles ? tile0 + p.chunk_tiles : tiles;
    const T* dtp = static_cast<const T*>(p.dt) + b * p.dt_batch + at.ch0;
    const T* zp = p.z ? static_cast<const T*>(p.z) + b * p.z_batch + at.ch0 : nullptr;
    const T* dyp = static_cast<const T*>(p.dy) + b * p.dy_batch + at.ch0;
    const T* Cp = static_cast<const T*>(p.C) + b * p.C_batch + at.group * p.C_group;
    const uint8_t* heads = p.heads ? p.heads + b * p.length : nullptr;
    Rows dt, z, dy;
    States C;
    auto fetch = [&](long long tile) {
        const long long t0 = tile * kTile;
        const int nt = (int)(p.length - t0 < kTile ? p.length - t0 : kTile);
        dt.load(dtp + t0 * p.dt_token, p.dt_token, nt, left, lane);
        dy.load(dyp + t0 * p.dy_token, p.dy_token, nt, left, lane);
        if (zp) z.load(zp + t0 * p.z_token, p.z_token, nt, left, lane);
        C.load(Cp + t0 * p.C_token, p.C_token, nt, (int)p.states, lane);
    };
    unsigned cut = 0;
    if (tile0 < tile1) fetch(tile1 - 1);
    for (long long tile = tile1 - 1; tile >= tile0; --tile) {
        const long long t0 = tile * kTile;
        const int nt = (int)(p.length - t0 < kTile ? p.length - t0 : kTile);
        const unsigned hm = tile_heads(heads, t0, nt, lane);
        cut |= hm;
        float fd[Rows::kCount], fg[Rows::kCount];
#pragma unroll
        for (int i = 0; i < Rows::kCount; ++i) {
            const float v = dt.get(i) + bias[Rows::channel_of(i)];
            fd[i] = Rows::valid(i, lane, nt, left) ? (p.softplus ? softplus(v) : v) : 0.0f;
            fg[i] = dy.get(i);
            if (zp) fg[i] *= z.get(i) * sigmoid(z.get(i));
        }
        Rows::to_shared(s_d[warp], fd, lane);
        Rows::to_shared(s_g[warp], fg, lane);
        C.to_shared(s_C[warp], lane);
        __syncwarp();
        if (tile > tile0) fetch(tile - 1);
#pragma unroll 4
        for (int t = kTile - 1; t >= 0; --t) {
            f2 d[G::PC], g[G::PC], Cv[4];
            read_channels<G>(s_d[warp] + t * G::CH + G::CPL * c, d);
            read_channels<G>(s_g[warp] + t * G::CH + G::CPL * c, g);
            read_states(s_C[warp] + t * G::NP + 4 * s, Cv);
#pragma unroll
            for (int q = 0; q < G::PC; ++q) {
                dsum[q] = add2(dsum[q], d[q]);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    dh[q][k] = mul2(ex2_2(mul2(d[q], A2[q][k])), fma2(Cv[k], g[q], dh[q][k]));
            }
            if (hm >> t & 1u) {
#pragma unroll
                for (int q = 0; q < G::PC; ++q)
#pragma unroll
                    for (int k = 0; k < 4; ++k) dh[q][k] = 0ull;
            }
        }
        __syncwarp();
    }
    const long long row = b * p.chunks + at.chunk;
    store_lane<G>(p.carry + (row * p.channels + at.ch0) * G::NP, left, lane, dh);
    if (s == 0)
#pragma unroll
        for (int j = 0; j < G::CPL; ++j)
            if (G::CPL * c + j < left)
                p.sum_d[row * p.channels + at.ch0 + G::CPL * c + j] = j & 1 ? hi2(dsum[j / 2]) : lo2(dsum[j / 2]);
    if (at.cblock == 0 && warp == 0 && lane == 0) p.cut[row] = cut != 0;
}

// Sums of eight values (four of dB, four of dC) over the lanes along the
// channels; `base` becomes the index of v[0], and v[0 .. 8 / CL) hold them
// (8 / CL at least 1).
template <class G>
__device__ __forceinline__ int sum_channels(float (&v)[8], int lane) {
    int base = 0;
    int n = 8;
#pragma unroll
    for (int m = G::S; m < 32; m <<= 1) {
        const bool up = lane & m;
        if (n > 1) {
            n /= 2;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (i < n) {
                    const float keep = up ? v[i + n] : v[i], send = up ? v[i] : v[i + n];
                    v[i] = keep + __shfl_xor_sync(0xffffffffu, send, m);
                }
            base += up ? n : 0;
        } else {
            v[0] += __shfl_xor_sync(0xffffffffu, v[0], m);
        }
    }
    return base;
}

template <class T, class G, bool kVec>
__global__ void __launch_bounds__(G::kThreads) ssm_back_kernel(SsmParams p, long long blocks_per_group) {
    using Rows = TileRows<T, G, kVec>;
    using States = TileStates<T, G, kVec>;
    using Sh = BwdShared<G>;
    extern __shared__ __align__(16) float s_all[];
    const SsmPlace<G> at(p, blocks_per_group, p.chunks);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int left = at.left > 0 ? (int)at.left : 0;  // a warp without channels still meets the CTA's barriers
    const int s = lane % G::S, c = lane / G::S;
    const long long b = at.b;
    float* sm = s_all + warp * Sh::kFloats;
    float4* hold = reinterpret_cast<float4*>(sm + Sh::h) + lane;
    const long long tiles = (p.length + kTile - 1) / kTile;
    const long long tile0 = at.chunk * p.chunk_tiles;
    const long long tile1 = tile0 + p.chunk_tiles < tiles ? tile0 + p.chunk_tiles : tiles;

    float raw[G::CPL][4];
    f2 A2[G::PC][4], dh[G::PC][4], dA[G::PC][4];
    load_lane_of<G>(p.A + at.ch0 * p.states, p.states, left, lane, raw);
    to_pairs<G>(raw, kLog2e, A2);
    load_lane_of<G>(p.dfinal ? p.dfinal + (b * p.channels + at.ch0) * p.states : nullptr, p.states, left, lane, raw);
    to_pairs<G>(raw, 1.0f, dh);
    for (long long j = p.chunks - 1; j > at.chunk; --j) fold_chunk<G>(p, A2, b, j, at.ch0, left, lane, dh);
#pragma unroll
    for (int q = 0; q < G::PC; ++q)
#pragma unroll
        for (int k = 0; k < 4; ++k) dA[q][k] = 0ull;
    float bias[Rows::kChannels], D[Rows::kChannels], dD[Rows::kChannels], dbias[Rows::kChannels];
#pragma unroll
    for (int i = 0; i < Rows::kChannels; ++i) {
        const int ch = Rows::ch(i, lane);
        bias[i] = p.dt_bias && ch < left ? p.dt_bias[at.ch0 + ch] : 0.0f;
        D[i] = p.D && ch < left ? p.D[at.ch0 + ch] : 0.0f;
        dD[i] = dbias[i] = 0.0f;
    }
    const T* xp = static_cast<const T*>(p.x) + b * p.x_batch + at.ch0;
    const T* dtp = static_cast<const T*>(p.dt) + b * p.dt_batch + at.ch0;
    const T* zp = p.z ? static_cast<const T*>(p.z) + b * p.z_batch + at.ch0 : nullptr;
    const T* dyp = static_cast<const T*>(p.dy) + b * p.dy_batch + at.ch0;
    const T* Bp = static_cast<const T*>(p.B) + b * p.B_batch + at.group * p.B_group;
    const T* Cp = static_cast<const T*>(p.C) + b * p.C_batch + at.group * p.C_group;
    const long long orow = b * p.length * p.channels + at.ch0;  // dx, ddt, dz are contiguous
    const uint8_t* heads = p.heads ? p.heads + b * p.length : nullptr;

    for (long long tile = tile1 - 1; tile >= tile0; --tile) {
        const long long t0 = tile * kTile;
        const int nt = (int)(p.length - t0 < kTile ? p.length - t0 : kTile);
        const unsigned hm = tile_heads(heads, t0, nt, lane);
        Rows x, dt, z, dy;
        {
            States B, C;
            x.load(xp + t0 * p.x_token, p.x_token, nt, left, lane);
            dt.load(dtp + t0 * p.dt_token, p.dt_token, nt, left, lane);
            dy.load(dyp + t0 * p.dy_token, p.dy_token, nt, left, lane);
            if (zp) z.load(zp + t0 * p.z_token, p.z_token, nt, left, lane);
            B.load(Bp + t0 * p.B_token, p.B_token, nt, (int)p.states, lane);
            C.load(Cp + t0 * p.C_token, p.C_token, nt, (int)p.states, lane);
            float fd[Rows::kCount], fu[Rows::kCount], fg[Rows::kCount];
#pragma unroll
            for (int i = 0; i < Rows::kCount; ++i) {
                const float v = dt.get(i) + bias[Rows::channel_of(i)];
                fd[i] = Rows::valid(i, lane, nt, left) ? (p.softplus ? softplus(v) : v) : 0.0f;
                fu[i] = fd[i] * x.get(i);
                fg[i] = dy.get(i);
                if (zp) fg[i] *= z.get(i) * sigmoid(z.get(i));
            }
            Rows::to_shared(sm + Sh::d, fd, lane);
            Rows::to_shared(sm + Sh::u, fu, lane);
            Rows::to_shared(sm + Sh::g, fg, lane);
            B.to_shared(reinterpret_cast<float2*>(sm + Sh::B), lane);
            C.to_shared(reinterpret_cast<float2*>(sm + Sh::C), lane);
        }
        const float2* sB = reinterpret_cast<const float2*>(sm + Sh::B);
        const float2* sC = reinterpret_cast<const float2*>(sm + Sh::C);
        f2 h[G::PC][4];
        load_lane<G>(p.saved + ((b * tiles + tile) * p.channels + at.ch0) * G::NP, left, lane, raw);
        to_pairs<G>(raw, 1.0f, h);
        __syncwarp();
        // the states before each quarter
#pragma unroll 1
        for (int q4 = 0; q4 < kTile / kQuarter; ++q4) {
#pragma unroll
            for (int q = 0; q < G::PC; ++q) {
                hold[(q4 * G::CPL + 2 * q) * 32] = make_float4(lo2(h[q][0]), hi2(h[q][0]), lo2(h[q][1]), hi2(h[q][1]));
                hold[(q4 * G::CPL + 2 * q + 1) * 32] =
                    make_float4(lo2(h[q][2]), hi2(h[q][2]), lo2(h[q][3]), hi2(h[q][3]));
            }
            if (q4 == kTile / kQuarter - 1) break;
#pragma unroll
            for (int j = 0; j < kQuarter; ++j) {
                const int t = q4 * kQuarter + j;
                f2 d[G::PC], u[G::PC], Bv[4];
                read_channels<G>(sm + Sh::d + t * G::CH + G::CPL * c, d);
                read_channels<G>(sm + Sh::u + t * G::CH + G::CPL * c, u);
                read_states(sB + t * G::NP + 4 * s, Bv);
                const bool head = hm >> t & 1u;
#pragma unroll
                for (int q = 0; q < G::PC; ++q)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        h[q][k] = fma2(ex2_2(mul2(d[q], A2[q][k])), head ? 0ull : h[q][k], mul2(u[q], Bv[k]));
            }
        }
#pragma unroll 1
        for (int q4 = kTile / kQuarter - 1; q4 >= 0; --q4) {
            f2 a[kQuarter][G::PC][4], ah[kQuarter][G::PC][4];  // q and q h[t-1]
#pragma unroll
            for (int q = 0; q < G::PC; ++q) {
                const float4 v = hold[(q4 * G::CPL + 2 * q) * 32], w = hold[(q4 * G::CPL + 2 * q + 1) * 32];
                h[q][0] = pack2(v.x, v.y);
                h[q][1] = pack2(v.z, v.w);
                h[q][2] = pack2(w.x, w.y);
                h[q][3] = pack2(w.z, w.w);
            }
#pragma unroll
            for (int j = 0; j < kQuarter; ++j) {
                const int t = q4 * kQuarter + j;
                f2 d[G::PC], u[G::PC], Bv[4];
                read_channels<G>(sm + Sh::d + t * G::CH + G::CPL * c, d);
                read_channels<G>(sm + Sh::u + t * G::CH + G::CPL * c, u);
                read_states(sB + t * G::NP + 4 * s, Bv);
                const bool head = hm >> t & 1u;
#pragma unroll
                for (int q = 0; q < G::PC; ++q)
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        a[j][q][k] = ex2_2(mul2(d[q], A2[q][k]));
                        ah[j][q][k] = head ? 0ull : mul2(a[j][q][k], h[q][k]);
                        h[q][k] = fma2(u[q], Bv[k], ah[j][q][k]);
                    }
            }
#pragma unroll
            for (int j = kQuarter - 1; j >= 0; --j) {
                const int t = q4 * kQuarter + j;
                f2 d[G::PC], u[G::PC], g[G::PC], Bv[4], Cv[4];
                read_channels<G>(sm + Sh::d + t * G::CH + G::CPL * c, d);
                read_channels<G>(sm + Sh::u + t * G::CH + G::CPL * c, u);
                read_channels<G>(sm + Sh::g + t * G::CH + G::CPL * c, g);
                read_states(sB + t * G::NP + 4 * s, Bv);
                read_states(sC + t * G::NP + 4 * s, Cv);
                f2 y[G::PC], gu[G::PC], ga[G::PC], dB[4], dC[4];
#pragma unroll
                for (int q = 0; q < G::PC; ++q) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        dh[q][k] = fma2(Cv[k], g[q], dh[q][k]);
                        const f2 ht = fma2(u[q], Bv[k], ah[j][q][k]);
                        const f2 r = mul2(dh[q][k], ah[j][q][k]);
                        y[q] = k ? fma2(Cv[k], ht, y[q]) : mul2(Cv[k], ht);
                        gu[q] = k ? fma2(dh[q][k], Bv[k], gu[q]) : mul2(dh[q][k], Bv[k]);
                        ga[q] = k ? fma2(r, A2[q][k], ga[q]) : mul2(r, A2[q][k]);
                        dA[q][k] = fma2(r, d[q], dA[q][k]);
                        dC[k] = q ? fma2(g[q], ht, dC[k]) : mul2(g[q], ht);
                        dB[k] = q ? fma2(dh[q][k], u[q], dB[k]) : mul2(dh[q][k], u[q]);
                        dh[q][k] = mul2(dh[q][k], a[j][q][k]);
                    }
                }
                if (hm >> t & 1u) {
#pragma unroll
                    for (int q = 0; q < G::PC; ++q)
#pragma unroll
                        for (int k = 0; k < 4; ++k) dh[q][k] = 0ull;
                }
                const float sy = sum_states<G>(y, lane), su = sum_states<G>(gu, lane), sa = sum_states<G>(ga, lane);
                if (s < G::CPL) {
                    const int o = t * G::CH + G::CPL * c + s;
                    sm[Sh::y + o] = sy;
                    sm[Sh::gu + o] = su;
                    sm[Sh::ga + o] = sa;
                }
                float bc[8];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    bc[k] = lo2(dB[k]) + hi2(dB[k]);
                    bc[4 + k] = lo2(dC[k]) + hi2(dC[k]);
                }
                const int base = sum_channels<G>(bc, lane);
                constexpr int kHeld = G::CL >= 8 ? 1 : 8 / G::CL;
                if (G::CL <= 8 || lane < 16) {
#pragma unroll
                    for (int i = 0; i < kHeld; ++i) {
                        const int v = base + i;  // dB of state v, or dC of state v - 4
                        sm[Sh::bc + (t * 2 + (v >> 2)) * G::NP + 4 * s + (v & 3)] = bc[i];
                    }
                }
            }
        }
        __syncwarp();
        {
            float fy[Rows::kCount], fu[Rows::kCount], fa[Rows::kCount], fd[Rows::kCount], fg[Rows::kCount];
            Rows::from_shared(sm + Sh::y, fy, lane);
            Rows::from_shared(sm + Sh::gu, fu, lane);
            Rows::from_shared(sm + Sh::ga, fa, lane);
            Rows::from_shared(sm + Sh::d, fd, lane);
            Rows::from_shared(sm + Sh::g, fg, lane);
#pragma unroll
            for (int i = 0; i < Rows::kCount; ++i) {
                const int ch = Rows::channel_of(i);
                const bool ok = Rows::valid(i, lane, nt, left);
                const float xi = x.get(i);
                if (zp) {
                    const float zi = z.get(i), sg = sigmoid(zi);
                    fy[i] = dy.get(i) * fmaf(D[ch], xi, fy[i]) * sg * fmaf(zi, 1.0f - sg, 1.0f);  // dz
                }
                float dd = fmaf(fu[i], xi, fa[i] * kLn2);
                if (p.softplus) dd *= sigmoid(dt.get(i) + bias[ch]);
                fu[i] = fmaf(fu[i], fd[i], fg[i] * D[ch]);  // dx
                fa[i] = dd;
                if (ok) {
                    dbias[ch] += dd;
                    dD[ch] = fmaf(fg[i], xi, dD[ch]);
                }
            }
            const long long o = orow + t0 * p.channels;
            Rows::store(static_cast<T*>(p.dx) + o, p.channels, fu, nt, left, lane);
            Rows::store(static_cast<T*>(p.ddt) + o, p.channels, fa, nt, left, lane);
            if (zp) Rows::store(static_cast<T*>(p.dz) + o, p.channels, fy, nt, left, lane);
        }
        __syncthreads();
        float* part = p.part_bc + ((at.cblock * p.batch + b) * p.length + t0) * 2 * G::NP;
        for (int i = threadIdx.x; i < nt * 2 * G::NP; i += G::kThreads) {
            float sum = s_all[Sh::bc + i];
#pragma unroll
            for (int w = 1; w < G::kWarps; ++w) sum += s_all[w * Sh::kFloats + Sh::bc + i];
            part[i] = sum;
        }
        __syncthreads();
    }
    if (left <= 0) return;
    const long long row = b * p.chunks + at.chunk;
    store_lane<G>(p.part_a + (row * p.channels + at.ch0) * G::NP, left, lane, dA);
    {
        const long long rows = p.batch * p.chunks;
        Rows::sum_tokens(dD, lane);
        const bool mine = Rows::sum_tokens(dbias, lane);
#pragma unroll
        for (int i = 0; i < Rows::kChannels; ++i) {
            const int ch = Rows::ch(i, lane);
            if (mine && ch < left) {
                p.part_d[row * p.channels + at.ch0 + ch] = dD[i];
                p.part_d[(rows + row) * p.channels + at.ch0 + ch] = dbias[i];
            }
        }
    }
    if (p.dstate && at.chunk == 0)
        store_lane_of<G>(p.dstate + (b * p.channels + at.ch0) * p.states, p.states, left, lane, dh);
}

// dB and dC: the channel blocks' partial sums of a group, in order.
template <class T>
__global__ void __launch_bounds__(256) ssm_back_bc_kernel(SsmParams p, long long blocks_per_group, int np) {
    const long long n = p.batch * p.length * p.groups * p.states;
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
    if (i >= n) return;
    const long long state = i % p.states, bg = i / p.states, group = bg % p.groups, bt = bg / p.groups;
    const long long step = p.batch * p.length * 2 * np;
    const float* src = p.part_bc + group * blocks_per_group * step + bt * 2 * np + state;
    float sb = 0.0f, sc = 0.0f;
    for (long long j = 0; j < blocks_per_group; ++j) {
        sb += __ldg(src + j * step);
        sc += __ldg(src + j * step + np);
    }
    static_cast<T*>(p.dB)[i] = from_f32<T>(sb);
    static_cast<T*>(p.dC)[i] = from_f32<T>(sc);
}

template <class T, class G, bool kVec>
cudaError_t ssm_back_of(const SsmParams& p, const SsmPlan& plan, int* launches, cudaStream_t s) {
    const long long ncb = plan.blocks_per_group * p.groups;
    *launches = p.chunks > 1 ? 4 : 3;
    if (p.chunks > 1)
        ssm_back_summary_kernel<T, G, kVec><<<(unsigned)(ncb * (p.chunks - 1) * p.batch), G::kThreads, 0, s>>>(
            p, plan.blocks_per_group, p.chunks - 1);
    auto kernel = ssm_back_kernel<T, G, kVec>;
    constexpr size_t bytes = BwdShared<G>::kBytes;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e != cudaSuccess) return e;
    kernel<<<(unsigned)(ncb * p.chunks * p.batch), G::kThreads, bytes, s>>>(p, plan.blocks_per_group);
    const long long n = p.batch * p.length * p.groups * p.states;
    ssm_back_bc_kernel<T><<<(unsigned)((n + 255) / 256), 256, 0, s>>>(p, plan.blocks_per_group, G::NP);
    return cudaGetLastError();
}

template <class T>
cudaError_t ssm_back_type(const SsmParams& p, const SsmPlan& plan, int* launches, cudaStream_t s) {
    switch (plan.lanes) {
    case 2:
        return p.vec ? ssm_back_of<T, Geo<2>, true>(p, plan, launches, s)
                     : ssm_back_of<T, Geo<2>, false>(p, plan, launches, s);
    case 4:
        return p.vec ? ssm_back_of<T, Geo<4>, true>(p, plan, launches, s)
                     : ssm_back_of<T, Geo<4>, false>(p, plan, launches, s);
    case 8:
        return p.vec ? ssm_back_of<T, Geo<8>, true>(p, plan, launches, s)
                     : ssm_back_of<T, Geo<8>, false>(p, plan, launches, s);
    case 16:
        return p.vec ? ssm_back_of<T, Geo<16>, true>(p, plan, launches, s)
                     : ssm_back_of<T, Geo<16>, false>(p, plan, launches, s);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace scg
