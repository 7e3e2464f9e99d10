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
// kept per token: a tile's states are recomputed, first in one walk that leaves
// the states at its quarters in shared memory, then quarter by quarter, where q
// and h of four tokens stay in registers for the way back (in shared memory
// they would cost more accesses than the second exponential).  Sums over states
// and over channels go through shared memory, four tokens at a time; the sum
// over a CTA's warps per tile; and those over CTAs, rows and chunks in kernels
// of their own over the CTAs' partial rows.  Each in a fixed order.
//
// Per token and state 14 products and multiply-adds against 1.75 exponentials:
// the multipliers' time, 0.43 ms at 4 x 4096 tokens, 4096 channels and 16 states
// in bfloat16, is the nearest bound; the pass takes 1.20 ms, and the first kernel
// (below) 0.22 more; the whole step, forward pass included, 1.87.  What keeps it
// from the bound is that an SM holds 8 warps, 2 a quarter, which issue in 40 % of
// the clocks: 255 registers (A, dh and dA of 16 states a lane, q and h of a
// quarter) and 28 KB of shared memory a warp.  The quarters' work takes 44 % of a
// warp's time, the walk before it 8 %, the elements at both ends 22 %.  What
// shared memory leaves of the L1 is too little for spilled registers to stay in
// it, so what is used seldom (bias, D, their sums, a quarter's first state) lies
// in shared memory.
//
// States past `states`, where their number is none of 8, 16, 32 and 64, have A = B =
// C = 0 and take no part, as long as d, d x and g are finite; an infinity times their
// zeros would be NaN in every sum over states.  A CTA that meets one leaves, and a
// second launch of the kernel, whose CTAs return at once where that did not happen,
// sets those states to 0 token by token.  (Both in one kernel: 4 % more time in every
// call, by other registers in the loops that never meet one.)
//
// Rows too few for the machine: the length is split as in the forward pass,
// with a first kernel that walks the chunks backwards from zero, in shorter
// runs, of which there are enough for all SMs.
#pragma once
#include "sc_ssm.cuh"

namespace scg {

constexpr int kQuarter = 4;  // tokens kept in registers
constexpr int kQuarters = kTile / kQuarter;
constexpr int kBackWarps = 2;  // of a CTA of the first kernel

// The shared memory, in floats: the CTA's B and C, then each warp's part.
template <class G>
struct BwdShared {
    static constexpr int kRow = kTile * G::CH, kSums = G::TP * G::kSumRow, kStates = kTile * G::NP * 2;
    static constexpr int kHold = G::CPL * 4 * 32;                      // a warp's states
    static constexpr int d = 0, u = kRow, g = 2 * kRow;                // [kTile][CH]
    static constexpr int y = 3 * kRow, gu = y + kSums, ga = gu + kSums;  // [TP][kSumRow]
    static constexpr int h = ga + kSums;                               // states before each quarter
    static constexpr int bc = h + kQuarters * kHold;                   // [kQuarter][2][CL][S] fours of dB, dC
    static constexpr int sums = bc + kQuarter * 2 * 32 * 4;            // [kTile][2][NP]
    static constexpr int ends = sums + kTile * 2 * G::NP;               // [dD, dbias][32] fours, the lanes' own
    static constexpr int per = ends + 2 * 32 * 4;                      // [bias, D][CH]
    static constexpr int kFloats = per + 2 * G::CH;
    static constexpr int kWarp0 = 2 * kStates;                         // [B, C][kTile][NP] pairs before it
    static constexpr size_t kBytes = (size_t)(kWarp0 + kFloats * G::kBwdWarps) * 4;
};

// A tile's B and C, fours of states (or one) a thread of the CTA's, to (v, v) pairs.
template <class T, class G, bool kVec>
struct CtaStates {
    static constexpr int kNT = 32 * G::kBwdWarps, kPer = kVec ? 4 : 1;
    static constexpr int kLine = G::NP / kPer, kAll = kTile * kLine, NA = (2 * kAll + kNT - 1) / kNT;
    struct One {
        T e;
    };
    typename std::conditional<kVec, Vec<T, kVec ? 4 : 2>, One>::type v[NA];
    __device__ __forceinline__ void load(const T* B, const T* C, const SsmParams& p, long long t0, int nt) {
#pragma unroll
        for (int a = 0; a < NA; ++a) {
            const int q = threadIdx.x + kNT * a, kind = q / kAll, t = q % kAll / kLine, n = q % kLine * kPer;
            const T* from = kind ? C + (t0 + t) * p.C_token + n : B + (t0 + t) * p.B_token + n;
            const bool in = (2 * kAll % kNT == 0 || q < 2 * kAll) && t < nt && n < p.states;
            if constexpr (kVec) {
                v[a].zero();
                if (in) v[a].load(from);
            } else {
                v[a].e = in ? __ldg(from) : from_f32<T>(0.0f);
            }
        }
    }
    __device__ __forceinline__ void to_shared(float* s) const {
#pragma unroll
        for (int a = 0; a < NA; ++a) {
            const int q = threadIdx.x + kNT * a;
            if (2 * kAll % kNT != 0 && q >= 2 * kAll) break;
            if constexpr (kVec) {
                float4* o = reinterpret_cast<float4*>(s) + q * 2;
                o[0] = make_float4(v[a].get(0), v[a].get(0), v[a].get(1), v[a].get(1));
                o[1] = make_float4(v[a].get(2), v[a].get(2), v[a].get(3), v[a].get(3));
            } else {
                reinterpret_cast<float2*>(s)[q] = make_float2(to_f32(v[a].e), to_f32(v[a].e));
            }
        }
    }
};

// Whether any of kN floats of this warp's in shared memory is an infinity or NaN;
// after a barrier of the warp.  (Read again: in registers they would have to be kept
// for it, where the kernels have none to spare.)
template <int kN>
__device__ __forceinline__ bool not_finite(const float* s, int lane) {
    static_assert(kN % 128 == 0, "whole passes");
    f2 zero = 0ull;  // times 0: 0, or NaN
#pragma unroll
    for (int i = 0; i < kN / 128; ++i) {
        const ulonglong2 v = reinterpret_cast<const ulonglong2*>(s)[lane + 32 * i];
        zero = fma2(v.x, 0ull, fma2(v.y, 0ull, zero));
    }
    return __any_sync(0xffffffffu, lo2(zero) + hi2(zero) != 0.0f);
}

// Padding: no states past `states`; some, and CTAs that meet an infinity or NaN leave;
// some, for those CTAs.
enum Pad { kNoPad, kLeaveOdd, kOnlyOdd };

// dh of a run's first token, taken one token further back, with nothing
// coming in from behind; and the run's sum of d.
template <class T, class G, bool kVec, bool kPadded>
__global__ void __launch_bounds__(32 * kBackWarps) ssm_back_summary_kernel(SsmParams p, int blocks_per_group,
                                                                             int grid_runs) {
    using Rows = TileRows<T, G, kVec, kTile>;
    using States = TileStates<T, G, kVec, kTile>;
    constexpr int kWarps = kBackWarps;
    __shared__ alignas(16) float s_d[kWarps][kTile * G::CH], s_g[kWarps][kTile * G::CH];
    __shared__ alignas(16) float2 s_C[kWarps][kTile * G::NP];
    const SsmPlace<G, kWarps> at(p, blocks_per_group, grid_runs, threadIdx.x >> 5);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, left = at.left;
    if (left == 0) return;
    const long long run = at.chunk + p.chunk_tiles / p.run_tiles;  // nobody waits for the first chunk's
    const int s = lane % G::S, c = lane / G::S;
    const long long b = at.b;
    float raw[G::CPL][4];
    f2 A2[G::PC][4], dh[G::PC][4], dsum[G::PC], bias[2];
    load_lane_of<G>(p.A + at.ch0 * p.states, p.states, left, lane, raw);
    to_rates<G>(raw, A2);
    clear<G>(dh);
#pragma unroll
    for (int q = 0; q < G::PC; ++q) dsum[q] = 0ull;
    Rows::per_channel(p.dt_bias ? p.dt_bias + at.ch0 : nullptr, left, lane, bias);
    const long long tiles = (p.length + kTile - 1) / kTile;
    const long long tile0 = run * p.run_tiles;
    const long long tile1 = tile0 + p.run_tiles < tiles ? tile0 + p.run_tiles : tiles;
    const T* dtp = static_cast<const T*>(p.dt) + b * p.dt_batch + at.ch0;
    const T* zp = p.z ? static_cast<const T*>(p.z) + b * p.z_batch + at.ch0 : nullptr;
    const T* dyp = static_cast<const T*>(p.dy) + b * p.dy_batch + at.ch0;
    const T* Cp = static_cast<const T*>(p.C) + b * p.C_batch + at.group * p.C_group;
    const uint8_t* heads = p.heads ? p.heads + b * p.length : nullptr;
    Rows dt, z, dy;
    States C;
    auto fetch = [&](long long tile, auto as_whole) {
        constexpr bool F = decltype(as_whole)::value;
        const long long t0 = tile * kTile;
        const int nt = F ? kTile : tile_tokens<kTile>(p, tile * kTile);
        dt.template load<F>(dtp + t0 * p.dt_token, p.dt_token, nt, left, lane);
        dy.template load<F>(dyp + t0 * p.dy_token, p.dy_token, nt, left, lane);
        if (F || zp) z.template load<F>(zp + t0 * p.z_token, p.z_token, nt, left, lane);
        C.load(Cp + t0 * p.C_token, p.C_token, nt, (int)p.states, lane);
    };
    unsigned cut = 0;
    const float *ld = s_d[warp] + G::CPL * c, *lg = s_g[warp] + G::CPL * c;
    const float2* lC = s_C[warp] + 4 * s;
    if (tile0 < tile1) fetch(tile1 - 1, std::false_type{});
    for (long long tile = tile1 - 1; tile >= tile0; --tile) {
        const int nt = tile_tokens<kTile>(p, tile * kTile);
        const unsigned hm = tile_heads(heads, tile * kTile, nt, lane);
        cut |= hm;
        auto stage = [&](auto as_plain) {
            constexpr bool F = decltype(as_plain)::value;
            f2 d[Rows::NA][2], g[Rows::NA][2];
#pragma unroll
            for (int a = 0; a < Rows::NA; ++a) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    d[a][i] = add2(dt.pair(a, i), bias[i]);
                    if (F || p.softplus) d[a][i] = softplus_2<T>(d[a][i]);
                    g[a][i] = dy.pair(a, i);
                    if (F || zp) g[a][i] = mul2(g[a][i], mul2(z.pair(a, i), sigmoid_2<T>(z.pair(a, i))));
                }
                Rows::template mask<F>(d[a], a, nt, left, lane);
            }
#pragma unroll
            for (int a = 0; a < Rows::NA; ++a) {
                Rows::put(s_d[warp] + a * G::TP * G::CH, d[a], lane);
                Rows::put(s_g[warp] + a * G::TP * G::CH, g[a], lane);
            }
        };
        if (left == G::CH && nt == kTile && zp && p.softplus) stage(std::true_type{});
        else stage(std::false_type{});
        C.to_shared(s_C[warp], lane);
        __syncwarp();
        // states past `states` that would not stay 0 (infinity times 0)
        const bool odd = kPadded && (not_finite<kTile * G::CH>(s_d[warp], lane) || not_finite<kTile * G::CH>(s_g[warp], lane));
        if (tile > tile0) {  // only the last tile of a row may be short of tokens
            if (left == G::CH && zp) fetch(tile - 1, std::true_type{});
            else fetch(tile - 1, std::false_type{});
        }
        auto tokens = [&](auto with_care) {  // segment starts, or states to be kept at 0
#pragma unroll
            for (int t = kTile - 1; t >= 0; --t) {
                f2 d[G::PC], g[G::PC], Cv[4];
                read_channels<G>(ld + t * G::CH, d);
                read_channels<G>(lg + t * G::CH, g);
                read_states(lC + t * G::NP, Cv);
#pragma unroll
                for (int q = 0; q < G::PC; ++q) {
                    dsum[q] = add2(dsum[q], d[q]);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        dh[q][k] = mul2(decay_2(d[q], A2[q][k]), fma2(Cv[k], g[q], dh[q][k]));
                }
                if constexpr (decltype(with_care)::value && kPadded) drop_padding<G>(p.states, dh);
                if (decltype(with_care)::value && (hm >> t & 1u)) clear<G>(dh);
            }
        };
        if (odd || hm) tokens(std::true_type{});
        else tokens(std::false_type{});
        __syncwarp();
    }
    leave_run<G>(p, b, run, at.ch0, left, lane, dh, dsum);
    if (at.cblock == 0 && threadIdx.x == 0) p.cut[b * p.runs + run] = cut != 0;
}

__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// h = q h[t-1] + d x B over the tokens of a quarter.
template <class G, bool kHeads, bool kMask>
__device__ __forceinline__ void run_quarter(const float* ld, const float* lu, const float2* lB, int t0, unsigned hm,
                                            long long states, const f2 (&A2)[G::PC][4], f2 (&h)[G::PC][4]) {
#pragma unroll
    for (int j = 0; j < kQuarter; ++j) {
        f2 d[G::PC], u[G::PC], Bv[4];
        read_channels<G>(ld + (t0 + j) * G::CH, d);
        read_channels<G>(lu + (t0 + j) * G::CH, u);
        read_states(lB + (t0 + j) * G::NP, Bv);
        if (kHeads && (hm >> (t0 + j) & 1u)) clear<G>(h);
#pragma unroll
        for (int q = 0; q < G::PC; ++q)
#pragma unroll
            for (int k = 0; k < 4; ++k) h[q][k] = fma2(decay_2(d[q], A2[q][k]), h[q][k], mul2(u[q], Bv[k]));
        if constexpr (kMask) drop_padding<G>(states, h);
    }
}

template <class T, class G, bool kVec, Pad kPad>
__global__ void __launch_bounds__(32 * G::kBwdWarps) ssm_back_kernel(SsmParams p, int blocks_per_group) {
    if (kPad == kOnlyOdd && p.odd[blockIdx.x] == 0) return;
    if (kPad == kLeaveOdd && threadIdx.x == 0) p.odd[blockIdx.x] = 0;
    using Rows = TileRows<T, G, kVec, kTile>;
    using Sh = BwdShared<G>;
    constexpr int kWarps = G::kBwdWarps;
    extern __shared__ __align__(16) float s_all[];
    const SsmPlace<G, kWarps> at(p, blocks_per_group, p.chunks, threadIdx.x >> 5);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int left = at.left;  // a warp without channels still meets the CTA's barriers
    const int s = lane % G::S, c = lane / G::S;
    const long long b = at.b;
    float* sm = s_all + Sh::kWarp0 + warp * Sh::kFloats;
    const float *ld = sm + Sh::d + G::CPL * c, *lu = sm + Sh::u + G::CPL * c, *lg = sm + Sh::g + G::CPL * c;
    const float2 *lB = reinterpret_cast<const float2*>(s_all) + 4 * s, *lC = lB + kTile * G::NP;
    ulonglong2* hold = reinterpret_cast<ulonglong2*>(sm + Sh::h) + lane;
    const long long tiles = (p.length + kTile - 1) / kTile;
    const long long tile0 = at.chunk * p.chunk_tiles;
    const long long tile1 = tile0 + p.chunk_tiles < tiles ? tile0 + p.chunk_tiles : tiles;

    f2 A2[G::PC][4], dh[G::PC][4], dA[G::PC][4];
    {
        float raw[G::CPL][4];
        load_lane_of<G>(p.A + at.ch0 * p.states, p.states, left, lane, raw);
        to_rates<G>(raw, A2);
        load_lane_of<G>(p.dfinal ? p.dfinal + (b * p.channels + at.ch0) * p.states : nullptr, p.states, left, lane, raw);
        to_pairs<G>(raw, dh);
    }
    for (long long j = p.runs - 1; j >= (at.chunk + 1) * (p.chunk_tiles / p.run_tiles); --j)
        fold_run<G, kPad != kNoPad>(p, A2, b, j, at.ch0, left, lane, dh);
    clear<G>(dA);
    // Registers are what this kernel has least of: the bias, D and their gradients'
    // sums, used once a pass, stay in shared memory.
    ulonglong2* ends = reinterpret_cast<ulonglong2*>(sm + Sh::ends) + lane;
    ends[0] = ends[32] = make_ulonglong2(0ull, 0ull);
    for (int i = lane; i < 2 * G::CH; i += 32) {
        const float* from = i < G::CH ? p.dt_bias : p.D;
        sm[Sh::per + i] = from && i % G::CH < left ? __ldg(from + at.ch0 + i % G::CH) : 0.0f;
    }
    __syncwarp();
    const T* xp = static_cast<const T*>(p.x) + b * p.x_batch + at.ch0;
    const T* dtp = static_cast<const T*>(p.dt) + b * p.dt_batch + at.ch0;
    const T* zp = p.z ? static_cast<const T*>(p.z) + b * p.z_batch + at.ch0 : nullptr;
    const T* dyp = static_cast<const T*>(p.dy) + b * p.dy_batch + at.ch0;
    const T* Bp = static_cast<const T*>(p.B) + b * p.B_batch + at.group * p.B_group;
    const T* Cp = static_cast<const T*>(p.C) + b * p.C_batch + at.group * p.C_group;
    const long long orow = b * p.length * p.channels + at.ch0;  // dx, ddt, dz are contiguous
    const bool whole = left == G::CH;
    const uint8_t* heads = p.heads ? p.heads + b * p.length : nullptr;

    auto held_states = [&](int q4, f2(&h)[G::PC][4]) {
#pragma unroll
        for (int q = 0; q < G::PC; ++q) {
            const ulonglong2 v = hold[(q4 * G::CPL + 2 * q) * 32], w = hold[(q4 * G::CPL + 2 * q + 1) * 32];
            h[q][0] = v.x;
            h[q][1] = v.y;
            h[q][2] = w.x;
            h[q][3] = w.y;
        }
    };
    auto hold_states = [&](int q4, const f2(&h)[G::PC][4]) {
#pragma unroll
        for (int q = 0; q < G::PC; ++q) {
            hold[(q4 * G::CPL + 2 * q) * 32] = make_ulonglong2(h[q][0], h[q][1]);
            hold[(q4 * G::CPL + 2 * q + 1) * 32] = make_ulonglong2(h[q][2], h[q][3]);
        }
    };
    // a tile's B and C and the states at its start, asked for before the sums of
    // the tile walked before it (its other elements too: 2.08 ms a training step
    // against 2.01, 4 x 4096 x 4096; they do not fit in the registers)
    CtaStates<T, G, kVec> BC;
    float start[G::CPL][4];
    auto fetch = [&](long long tile) {
        BC.load(Bp, Cp, p, tile * kTile, tile_tokens<kTile>(p, tile * kTile));
        load_lane<G>(p.saved + (b * tiles + tile) * p.channels * G::NP + at.ch0 * 4, p.channels, left, lane, start);
    };
    if (tile0 < tile1) fetch(tile1 - 1);
    for (long long tile = tile1 - 1; tile >= tile0; --tile) {
        const long long t0 = tile * kTile;
        const int nt = tile_tokens<kTile>(p, tile * kTile);
        const unsigned hm = tile_heads(heads, t0, nt, lane);
        // Whole tiles of whole channel groups with a gate and a softplus, the
        // common ones, take loops without a branch among the elements, which would
        // keep their latencies from overlapping; so below.
        const bool plain = whole && nt == kTile && zp && p.softplus;
        auto stage = [&](auto as_plain) {
            constexpr bool F = decltype(as_plain)::value;
            Rows x, dt, z, dy;
            dt.template load<F>(dtp + t0 * p.dt_token, p.dt_token, nt, left, lane);
            x.template load<F>(xp + t0 * p.x_token, p.x_token, nt, left, lane);
            dy.template load<F>(dyp + t0 * p.dy_token, p.dy_token, nt, left, lane);
            if (F || zp) z.template load<F>(zp + t0 * p.z_token, p.z_token, nt, left, lane);
            f2 bias[2];
            Rows::channel_values(sm + Sh::per, bias, lane);
            f2 d[Rows::NA][2], u[Rows::NA][2], g[Rows::NA][2];
#pragma unroll
            for (int a = 0; a < Rows::NA; ++a) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    d[a][i] = add2(dt.pair(a, i), bias[i]);
                    if (F || p.softplus) d[a][i] = softplus_2<T>(d[a][i]);
                    g[a][i] = dy.pair(a, i);
                    if (F || zp) g[a][i] = mul2(g[a][i], mul2(z.pair(a, i), sigmoid_2<T>(z.pair(a, i))));
                }
                Rows::template mask<F>(d[a], a, nt, left, lane);
#pragma unroll
                for (int i = 0; i < 2; ++i) u[a][i] = mul2(d[a][i], x.pair(a, i));
            }
#pragma unroll
            for (int a = 0; a < Rows::NA; ++a) {
                Rows::put(sm + Sh::d + a * G::TP * G::CH, d[a], lane);
                Rows::put(sm + Sh::u + a * G::TP * G::CH, u[a], lane);
                Rows::put(sm + Sh::g + a * G::TP * G::CH, g[a], lane);
            }
        };
        if (plain) stage(std::true_type{});
        else stage(std::false_type{});
        BC.to_shared(s_all);
        f2 h0[G::PC][4];
        to_pairs<G>(start, h0);
        hold_states(0, h0);
        if (tile > tile0 && left > 0) {  // the next tile and its states on their way into the L2
            const long long t = t0 - kTile + lane % kTile;  // lanes 0 .. 15: x and dy, 16 ..: dt and z
            prefetch_l2(lane < kTile ? xp + t * p.x_token : dtp + t * p.dt_token);
            prefetch_l2(lane < kTile ? dyp + t * p.dy_token : zp ? zp + t * p.z_token : dtp + t * p.dt_token);
            const float* sv = p.saved + (b * tiles + tile - 1) * p.channels * G::NP + at.ch0 * 4;
            constexpr int kLines = G::CH * 16 / 128 > 0 ? G::CH * 16 / 128 : 1;  // of 128 bytes a four of states
            if (lane < G::S * kLines && lane % kLines * 8 < left) prefetch_l2(sv + (lane / kLines * p.channels + lane % kLines * 8) * 4);
        }
        // The elements of pass pa once more, asked for before the pass's states are
        // worked on and used after.
        using Raw = decltype(Rows::template fetch<true>(xp, 0, 0, 0, 0, 0));
        struct Pass {
            Raw x, dt, dy, z;
        };
        auto again = [&](int pa, auto as_plain) {
            constexpr bool F = decltype(as_plain)::value;
            Pass r;
            r.x = Rows::template fetch<F>(xp + t0 * p.x_token, p.x_token, pa, nt, left, lane);
            r.dt = Rows::template fetch<F>(dtp + t0 * p.dt_token, p.dt_token, pa, nt, left, lane);
            r.dy = Rows::template fetch<F>(dyp + t0 * p.dy_token, p.dy_token, pa, nt, left, lane);
            r.z = r.dy;
            if (F || zp) r.z = Rows::template fetch<F>(zp + t0 * p.z_token, p.z_token, pa, nt, left, lane);
            return r;
        };
        // the gradients by the elements of pass pa, whose first token is tq
        auto finish = [&](int pa, int tq, const Pass& e, auto as_plain) {
            constexpr bool F = decltype(as_plain)::value;
            const auto &rx = e.x, &rt = e.dt, &ry = e.dy, &rz = e.z;
            f2 y[2], gu[2], ga[2], d[2], g[2], dd[2], bias[2], D[2];
            Rows::channel_values(sm + Sh::per, bias, lane);
            Rows::channel_values(sm + Sh::per + G::CH, D, lane);
            ulonglong2 dD = ends[0], db = ends[32];
            Rows::get_sums(sm + Sh::gu, gu, lane);
            Rows::get_sums(sm + Sh::ga, ga, lane);
            Rows::get_sums(sm + Sh::y, y, lane);
            Rows::get(sm + Sh::d + tq * G::CH, d, lane);
            Rows::get(sm + Sh::g + tq * G::CH, g, lane);
            const long long o = orow + t0 * p.channels;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const f2 x = Rows::pair_of(rx, i);
                dd[i] = fma2(gu[i], x, mul2(ga[i], both(kLn2)));
                if (F || p.softplus) dd[i] = mul2(dd[i], sigmoid_2<T>(add2(Rows::pair_of(rt, i), bias[i])));
                gu[i] = fma2(gu[i], d[i], mul2(g[i], D[i]));  // dx
                (i ? dD.y : dD.x) = fma2(g[i], x, i ? dD.y : dD.x);
                if (F || zp) {
                    const f2 z = Rows::pair_of(rz, i), sg = sigmoid_2<T>(z);
                    const f2 slope = mul2(sg, fma2(z, fma2(sg, both(-1.0f), both(1.0f)), both(1.0f)));
                    y[i] = mul2(mul2(Rows::pair_of(ry, i), fma2(D[i], x, y[i])), slope);
                }
            }
            Rows::template store<F>(static_cast<T*>(p.dx) + o, p.channels, gu, pa, nt, left, lane);
            Rows::template store<F>(static_cast<T*>(p.ddt) + o, p.channels, dd, pa, nt, left, lane);
            if (F || zp) Rows::template store<F>(static_cast<T*>(p.dz) + o, p.channels, y, pa, nt, left, lane);
            Rows::template mask<F>(dd, pa, nt, left, lane);
            ends[0] = dD;
            ends[32] = make_ulonglong2(add2(db.x, dd[0]), add2(db.y, dd[1]));
        };
        if constexpr (kPad == kLeaveOdd) {  // d, u and g lie together
            __syncwarp();
            if (__syncthreads_or(not_finite<3 * Sh::kRow>(sm + Sh::d, lane))) {
                if (threadIdx.x == 0) p.odd[blockIdx.x] = 1;
                return;
            }
        } else {
            __syncthreads();
        }
        auto work = [&](auto with_heads) {
            constexpr bool kHeads = decltype(with_heads)::value;
#pragma unroll 1
            for (int q4 = 1; q4 < kQuarters; ++q4) {  // the states before quarters 1, 2, ...
                run_quarter<G, kHeads, kPad == kOnlyOdd>(ld, lu, lB, (q4 - 1) * kQuarter, hm, p.states, A2, h0);
                hold_states(q4, h0);
            }
#pragma unroll 1
            for (int q4 = kQuarters - 1; q4 >= 0; --q4) {
                const int tq = q4 * kQuarter;
                Pass raws;
                if (tq % G::TP == 0) raws = plain ? again(tq / G::TP, std::true_type{}) : again(tq / G::TP, std::false_type{});
                f2 a[kQuarter][G::PC][4], h[kQuarter + 1][G::PC][4];  // q, and h before each token
                held_states(q4, h[0]);
#pragma unroll
                for (int j = 0; j < kQuarter; ++j) {
                    f2 d[G::PC], u[G::PC], Bv[4];
                    read_channels<G>(ld + (tq + j) * G::CH, d);
                    read_channels<G>(lu + (tq + j) * G::CH, u);
                    read_states(lB + (tq + j) * G::NP, Bv);
                    const bool head = kHeads && (hm >> (tq + j) & 1u);
#pragma unroll
                    for (int q = 0; q < G::PC; ++q)
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            a[j][q][k] = decay_2(d[q], A2[q][k]);
                            h[j + 1][q][k] = fma2(a[j][q][k], head ? 0ull : h[j][q][k], mul2(u[q], Bv[k]));
                        }
                    if constexpr (kPad == kOnlyOdd) drop_padding<G>(p.states, h[j + 1]);
                }
#pragma unroll
                for (int j = kQuarter - 1; j >= 0; --j) {
                    const int t = tq + j;
                    const bool head = kHeads && (hm >> t & 1u);
                    const int real = kPad == kOnlyOdd ? (int)p.states - lane_anew() % G::S * 4 : 4;
                    f2 d[G::PC], u[G::PC], g[G::PC], Bv[4], Cv[4];
                    read_channels<G>(ld + t * G::CH, d);
                    read_channels<G>(lu + t * G::CH, u);
                    read_channels<G>(lg + t * G::CH, g);
                    read_states(lB + t * G::NP, Bv);
                    read_states(lC + t * G::NP, Cv);
                    if (j == 0) held_states(q4, h[0]);  // read again: not kept in registers meanwhile
                    f2 y[G::PC], gu[G::PC], ga[G::PC], dB[4], dC[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
#pragma unroll
                        for (int q = 0; q < G::PC; ++q) {
                            const f2 ht = h[j + 1][q][k];
                            dh[q][k] = fma2(Cv[k], g[q], dh[q][k]);
                            if (kPad == kOnlyOdd && k >= real) dh[q][k] = 0ull;
                            y[q] = k ? fma2(Cv[k], ht, y[q]) : mul2(Cv[k], ht);
                            dC[k] = q ? fma2(g[q], ht, dC[k]) : mul2(g[q], ht);
                            gu[q] = k ? fma2(dh[q][k], Bv[k], gu[q]) : mul2(dh[q][k], Bv[k]);
                            dB[k] = q ? fma2(dh[q][k], u[q], dB[k]) : mul2(dh[q][k], u[q]);
                            dh[q][k] = head ? 0ull : mul2(dh[q][k], a[j][q][k]);
                            if (kPad == kOnlyOdd && k >= real) dh[q][k] = 0ull;
                            const f2 r = mul2(dh[q][k], head ? 0ull : h[j][q][k]);
                            ga[q] = k ? fma2(r, A2[q][k], ga[q]) : mul2(r, A2[q][k]);
                            dA[q][k] = fma2(r, d[q], dA[q][k]);
                        }
                    }
                    const int row = (t % G::TP) * G::kSumRow;
                    put_sums<G>(sm + Sh::y + row, y, lane);
                    put_sums<G>(sm + Sh::gu + row, gu, lane);
                    put_sums<G>(sm + Sh::ga + row, ga, lane);
                    float4* o = reinterpret_cast<float4*>(sm + Sh::bc) + j * 64 + lane;  // lane = c * S + s
                    o[0] = make_float4(lo2(dB[0]) + hi2(dB[0]), lo2(dB[1]) + hi2(dB[1]), lo2(dB[2]) + hi2(dB[2]),
                                       lo2(dB[3]) + hi2(dB[3]));
                    o[32] = make_float4(lo2(dC[0]) + hi2(dC[0]), lo2(dC[1]) + hi2(dC[1]), lo2(dC[2]) + hi2(dC[2]),
                                        lo2(dC[3]) + hi2(dC[3]));
                }
                __syncwarp();
                // the quarter's dB and dC over the warp's channels: four states (o) of one token and kind at a time
#pragma unroll
                for (int o = lane; o < kQuarter * 2 * G::S; o += 32) {
                    const int kind = o / G::S;  // token * 2 + (0: dB, 1: dC)
                    const ulonglong2* in = reinterpret_cast<const ulonglong2*>(sm + Sh::bc) + kind * 32 + o % G::S;
                    ulonglong2 v = in[kind % G::CL * G::S];
#pragma unroll
                    for (int i = 1; i < G::CL; ++i) {  // starting points apart: the kinds meet in no bank
                        const ulonglong2 w = in[(kind + i) % G::CL * G::S];
                        v.x = add2(v.x, w.x);
                        v.y = add2(v.y, w.y);
                    }
                    reinterpret_cast<ulonglong2*>(sm + Sh::sums)[tq * 2 * G::S + o] = v;
                }
                if (tq % G::TP == 0) {
                    if (plain) finish(tq / G::TP, tq, raws, std::true_type{});
                    else finish(tq / G::TP, tq, raws, std::false_type{});
                }
                __syncwarp();
            }
        };
        if (hm) work(std::true_type{});
        else work(std::false_type{});
        if (tile > tile0) fetch(tile - 1);
        // dA goes to its partial row every 128 tokens: one running sum over
        // thousands of tokens of either sign would lose a digit to rounding
        if ((tile - tile0) % 8 == 0 && left > 0) {
            float* pa = p.part_a + (b * p.chunks + at.chunk) * p.channels * G::NP + at.ch0 * 4;
            if (tile + 8 < tile1) {
                float raw[G::CPL][4];
                f2 old[G::PC][4];
                load_lane<G>(pa, p.channels, left, lane, raw);
                to_pairs<G>(raw, old);
#pragma unroll
                for (int q = 0; q < G::PC; ++q)
#pragma unroll
                    for (int k = 0; k < 4; ++k) dA[q][k] = add2(dA[q][k], old[q][k]);
            }
            store_lane<G>(pa, p.channels, left, lane, dA);
            clear<G>(dA);
        }
        __syncthreads();
        float4* part = reinterpret_cast<float4*>(p.part_bc + ((at.cblock * p.batch + b) * p.length + t0) * 2 * G::NP);
        for (int i = threadIdx.x; i < nt * 2 * G::S; i += 32 * kWarps) {
            float4 sum = reinterpret_cast<const float4*>(s_all + Sh::kWarp0 + Sh::sums)[i];
#pragma unroll
            for (int w = 1; w < kWarps; ++w) {
                const float4 v = reinterpret_cast<const float4*>(s_all + Sh::kWarp0 + w * Sh::kFloats + Sh::sums)[i];
                sum.x += v.x;
                sum.y += v.y;
                sum.z += v.z;
                sum.w += v.w;
            }
            part[i] = sum;
        }
    }
    if (left == 0) return;
    const long long row = b * p.chunks + at.chunk, rows = p.batch * p.chunks;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const f2 sum[2] = {ends[32 * i].x, ends[32 * i].y};
        Rows::put_channel_sums(p.part_d + (i * rows + row) * p.channels + at.ch0, sum, left, lane);
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

template <class T, class G, bool kVec, bool kPadded>
cudaError_t ssm_back_of(const SsmParams& p, const SsmPlan& plan, int* launches, cudaStream_t s) {
    const long long per = p.channels / p.groups;
    *launches = (p.chunks > 1 ? 4 : 3) + (kPadded ? 1 : 0);  // with the last sums, which the caller launches
    if (p.chunks > 1) {
        const long long block = kBackWarps * G::CH;
        const int bpg = (int)((per + block - 1) / block), runs = p.runs - (int)(p.chunk_tiles / p.run_tiles);
        auto first = ssm_back_summary_kernel<T, G, kVec, kPadded>;
        first<<<(unsigned)(bpg * p.groups * runs * p.batch), 32 * kBackWarps, 0, s>>>(p, bpg, runs);
    }
    const int bpg = (int)plan.blocks_per_group;
    auto go = [&](auto kernel) {
        constexpr size_t bytes = BwdShared<G>::kBytes;
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
        if (e == cudaSuccess)
            kernel<<<(unsigned)(bpg * p.groups * p.chunks * p.batch), 32 * G::kBwdWarps, bytes, s>>>(p, bpg);
        return e;
    };
    cudaError_t e = go(ssm_back_kernel<T, G, kVec, kPadded ? kLeaveOdd : kNoPad>);
    if constexpr (kPadded)
        if (e == cudaSuccess) e = go(ssm_back_kernel<T, G, false, kOnlyOdd>);
    if (e != cudaSuccess) return e;
    const long long n = p.batch * p.length * p.groups * p.states;
    ssm_back_bc_kernel<T><<<(unsigned)((n + 255) / 256), 256, 0, s>>>(p, plan.blocks_per_group, G::NP);
    return cudaGetLastError();
}

template <class T>
cudaError_t ssm_back_type(const SsmParams& p, const SsmPlan& plan, int* launches, cudaStream_t s) {
    auto go = [&](auto g) {
        using G = decltype(g);
        if (p.states == G::NP)
            return p.vec ? ssm_back_of<T, G, true, false>(p, plan, launches, s)
                         : ssm_back_of<T, G, false, false>(p, plan, launches, s);
        return p.vec ? ssm_back_of<T, G, true, true>(p, plan, launches, s)
                     : ssm_back_of<T, G, false, true>(p, plan, launches, s);
    };
    switch (plan.lanes) {
    case 2: return go(Geo<2>{});
    case 4: return go(Geo<4>{});
    case 8: return go(Geo<8>{});
    case 16: return go(Geo<16>{});
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace scg
