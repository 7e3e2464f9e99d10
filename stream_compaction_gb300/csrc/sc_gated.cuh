// The gated recurrence h[t] = f[t] h[t-1] + b[t], f = sigmoid(gate), b = (1 - f) x
// (or f = gate, b = x), its gradient and its form for one token: kernels, by element
// type in sc_gated_*.cu.
//
//   dh[t] = dy[t] + f[t+1] dh[t+1];  dx = dh (1 - f);  dgate = dh (h[t-1] - x) f (1 - f)
//
// Three elements moved forward and five backward for some ten operations each: bytes
// bound it, if the length is split.  A tile of kTokens tokens by 32 or 64 channels
// lies in a warp's registers, a lane's channels side by side with all their tokens, so
// the recurrence needs no exchange inside a tile.  The warps of a CTA take consecutive
// tiles of the same channels, and the CTAs of a cluster consecutive runs of them; a
// round of kWarps x cluster tiles goes like a scan:
//
//   each warp   its tile's map h -> A h + B (A the product of f, B the recurrence from 0);
//   the CTA     the maps meet in shared memory; the CTA's own map goes to every CTA of
//               the cluster (distributed shared memory, one cluster barrier a round);
//   each warp   the state before its tile: the carry, through the maps before it in order;
//               then the recurrence again, on registers, and the results.
//
// So every element is read once and written once, no scratch memory is needed, and the
// order of all roundings is fixed.  The next round's elements are loaded into registers
// before the exchange and arrive during it.
//
// The gradient runs the same rounds backwards on q[t] = f[t] dh[t], with the states
// recomputed from those that the forward pass saved (one in kTokens: 1/16 of an
// element's place in float32, where keeping h itself would cost an element read and
// rounding errors of 16 bits in dgate).
#pragma once
#include <algorithm>

#include <cooperative_groups.h>

#include "sc_seq.cuh"
#include "sc_seq_launch.h"

namespace scg {

namespace {

namespace cg = cooperative_groups;

constexpr int kTokens = SC_GATED_SAVE;
constexpr int kMaxCluster = 8;

// A lane's K channels of a token.
template <class T, int K> struct Raw;
template <> struct Raw<float, 1> { using type = float; };
template <> struct Raw<f16, 1> { using type = unsigned short; };
template <> struct Raw<bf16, 1> { using type = unsigned short; };
template <> struct Raw<f16, 2> { using type = uint32_t; };
template <> struct Raw<bf16, 2> { using type = uint32_t; };

template <class T, int K>
struct Cell {
    typename Raw<T, K>::type r;
    __device__ __forceinline__ void load(const T* p) { r = __ldg(reinterpret_cast<const typename Raw<T, K>::type*>(p)); }
    __device__ __forceinline__ void zero() { memset(&r, 0, sizeof(r)); }
    __device__ __forceinline__ float get(int k) const {
        T e[K];
        memcpy(e, &r, sizeof(r));
        return to_f32(e[k]);
    }
    __device__ __forceinline__ static void store(T* p, const float (&v)[K]) {
        T e[K];
#pragma unroll
        for (int k = 0; k < K; ++k) e[k] = from_f32<T>(v[k]);
        typename Raw<T, K>::type w;
        memcpy(&w, e, sizeof(w));
        *reinterpret_cast<typename Raw<T, K>::type*>(p) = w;
    }
};

// f = sigmoid(g) and 1 - f, each without cancellation: the smaller of the two is
// e / (1 + e), e = exp(-|g|), and the other 1 minus it.  So a decay close to 1 is off
// by its own rounding alone, however many of them are multiplied.
template <class T>
__device__ __forceinline__ void gate_of(float g, float& f, float& rest) {
    const float e = exp_minus<kFine<T>>(fabsf(g));
    const float small = e * rcp(1.0f + e), large = 1.0f - small;
    f = g < 0.0f ? small : large;  // NaN: both are NaN
    rest = g < 0.0f ? large : small;
}

// Tokens of a tile where a segment starts, one bit each.
__device__ __forceinline__ uint32_t cuts_of(const uint8_t* heads, long long row, long long t0, long long length, int lane) {
    if (!heads) return 0u;
    const long long t = t0 + lane;
    return __ballot_sync(0xffffffffu, lane < kTokens && t < length && heads[row * length + t] != 0);
}

// The map of a run of tokens on the state before it: h -> A h + B, or B alone where a
// segment starts inside (whatever h is, infinities too).
__device__ __forceinline__ float through(float A, float B, bool cut, float h) { return cut ? B : fmaf(A, h, B); }

// What the warps and CTAs of a round exchange.
template <int K, int kWarps>
struct Exchange {
    float A[2][kWarps][K][32], B[2][kWarps][K][32];
    float rank_A[2][kMaxCluster][K][32], rank_B[2][kMaxCluster][K][32];
    int cut[2][kWarps], rank_cut[2][kMaxCluster];
};

// One round: takes this warp's map, returns the value before its tile in `in` and
// moves `carry`, the value before the round, to behind it (the same in all warps).
// Warps and CTAs count in the direction of the recurrence.  Buffers alternate: a warp
// writes for the next round while others still read this one's, and two rounds on a
// barrier lies between.
template <int K, int kWarps>
__device__ __forceinline__ void exchange(Exchange<K, kWarps>& x, int turn, int warp, int lane, int rank, int ranks,
                                         const float (&A)[K], const float (&B)[K], bool cut, float (&carry)[K],
                                         float (&in)[K]) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
        x.A[turn][warp][k][lane] = A[k];
        x.B[turn][warp][k][lane] = B[k];
    }
    if (lane == 0) x.cut[turn][warp] = cut;
    __syncthreads();
    if (ranks > 1) {
        if (warp == 0) {
            float a[K], b[K];
            bool any = false;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                a[k] = 1.0f;
                b[k] = 0.0f;
            }
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const bool c = x.cut[turn][w] != 0;
                any |= c;
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    b[k] = through(x.A[turn][w][k][lane], x.B[turn][w][k][lane], c, b[k]);
                    a[k] *= x.A[turn][w][k][lane];
                }
            }
            const cg::cluster_group cluster = cg::this_cluster();
            for (int r = 0; r < ranks; ++r) {
                Exchange<K, kWarps>* other = cluster.map_shared_rank(&x, r);
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    other->rank_A[turn][rank][k][lane] = a[k];
                    other->rank_B[turn][rank][k][lane] = b[k];
                }
                if (lane == 0) other->rank_cut[turn][rank] = any;
            }
        }
        cg::this_cluster().sync();
    }
#pragma unroll
    for (int k = 0; k < K; ++k) in[k] = carry[k];
    if (ranks > 1) {
        for (int r = 0; r < ranks; ++r) {
            if (r == rank) {
#pragma unroll
                for (int k = 0; k < K; ++k) in[k] = carry[k];
            }
            const bool c = x.rank_cut[turn][r] != 0;
#pragma unroll
            for (int k = 0; k < K; ++k) carry[k] = through(x.rank_A[turn][r][k][lane], x.rank_B[turn][r][k][lane], c, carry[k]);
        }
    }
    float h[K];
#pragma unroll
    for (int k = 0; k < K; ++k) h[k] = in[k];
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        const bool c = x.cut[turn][w] != 0;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if (w == warp) in[k] = h[k];
            h[k] = through(x.A[turn][w][k][lane], x.B[turn][w][k][lane], c, h[k]);
        }
    }
    if (ranks == 1) {
#pragma unroll
        for (int k = 0; k < K; ++k) carry[k] = h[k];
    }
}

// Where a CTA works: row b, the lane's first channel, the rounds.
struct Place {
    long long b, ch, rounds, tiles;
    int rank, ranks, warp, lane;
    bool live;
};
template <int K, int kWarps>
__device__ __forceinline__ Place place_of(const GatedParams& p) {
    Place c;
    c.rank = (int)cg::this_cluster().block_rank();
    c.ranks = (int)cg::this_cluster().num_blocks();
    const long long blocks = (p.channels + 32 * K - 1) / (32 * K), group = blockIdx.x / c.ranks;
    c.b = group / blocks;
    c.warp = threadIdx.x / 32;
    c.lane = threadIdx.x % 32;
    c.ch = ((group - c.b * blocks) * 32 + c.lane) * K;
    c.live = c.ch < p.channels;
    c.tiles = (p.length + kTokens - 1) / kTokens;
    c.rounds = (c.tiles + c.ranks * kWarps - 1) / (c.ranks * kWarps);
    return c;
}

template <class T, int K>
__device__ __forceinline__ void load_tile(const T* p, long long stride, int valid, Cell<T, K> (&v)[kTokens]) {
    if (valid == kTokens) {
#pragma unroll
        for (int j = 0; j < kTokens; ++j) v[j].load(p + j * stride);
    } else {
#pragma unroll
        for (int j = 0; j < kTokens; ++j) {
            if (j < valid) v[j].load(p + j * stride);
            else v[j].zero();
        }
    }
}

// ---------------------------------------------------------------- forward
template <class T, int K, bool kSigmoid, int kWarps>
__global__ void __launch_bounds__(32 * kWarps, 16 / kWarps) gated_kernel(GatedParams p) {
    __shared__ Exchange<K, kWarps> s_ex;
    const Place c = place_of<K, kWarps>(p);
    const T* x = static_cast<const T*>(p.x) + c.b * p.x_batch + c.ch;
    const T* g = static_cast<const T*>(p.gate) + c.b * p.gate_batch + c.ch;
    T* y = static_cast<T*>(p.y) + c.b * p.y_batch + c.ch;
    Cell<T, K> xr[kTokens], gr[kTokens];
    uint32_t cuts;
    auto tokens = [&](long long tile) { return (int)max(0ll, min((long long)kTokens, p.length - tile * kTokens)); };
    auto fetch = [&](long long tile) {
        const long long t0 = tile * kTokens;
        const int valid = c.live ? tokens(tile) : 0;
        load_tile<T, K>(x + t0 * p.x_token, p.x_token, valid, xr);
        load_tile<T, K>(g + t0 * p.gate_token, p.gate_token, valid, gr);
        cuts = cuts_of(p.heads, c.b, t0, p.length, c.lane);
    };
    float carry[K], h[K];
#pragma unroll
    for (int k = 0; k < K; ++k) carry[k] = p.state && c.live ? __ldg(p.state + c.b * p.channels + c.ch + k) : 0.0f;
    long long tile = (long long)c.rank * kWarps + c.warp;
    const long long step = (long long)c.ranks * kWarps;
    fetch(tile);
    if (c.ranks > 1) cg::this_cluster().sync();  // every CTA has begun before one writes to its shared memory
    for (long long round = 0; round < c.rounds; ++round, tile += step) {
        float f[kTokens][K], b[kTokens][K];
        const uint32_t cut = cuts;
        const int valid = tokens(tile);
#pragma unroll
        for (int j = 0; j < kTokens; ++j)
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const float xv = xr[j].get(k), gv = gr[j].get(k);
                if constexpr (kSigmoid) {
                    gate_of<T>(gv, f[j][k], b[j][k]);
                    b[j][k] *= xv;
                } else {
                    f[j][k] = gv;
                    b[j][k] = xv;
                }
            }
        if (valid < kTokens) {  // behind the row's end: the state stays
#pragma unroll
            for (int j = 0; j < kTokens; ++j)
#pragma unroll
                for (int k = 0; k < K; ++k)
                    if (j >= valid) {
                        f[j][k] = 1.0f;
                        b[j][k] = 0.0f;
                    }
        }
        if (cut) {
#pragma unroll
            for (int j = 0; j < kTokens; ++j)
                if (cut >> j & 1u)
#pragma unroll
                    for (int k = 0; k < K; ++k) f[j][k] = 0.0f;
        }
        if (round + 1 < c.rounds) fetch(tile + step);
        float A[K], B[K];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            A[k] = f[0][k];
            B[k] = b[0][k];
        }
        if (!cut) {
#pragma unroll
            for (int j = 1; j < kTokens; ++j)
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    A[k] *= f[j][k];
                    B[k] = fmaf(f[j][k], B[k], b[j][k]);
                }
        } else {
#pragma unroll
            for (int j = 1; j < kTokens; ++j)
#pragma unroll
                for (int k = 0; k < K; ++k) B[k] = cut >> j & 1u ? b[j][k] : fmaf(f[j][k], B[k], b[j][k]);
#pragma unroll
            for (int k = 0; k < K; ++k) A[k] = 0.0f;
        }
        exchange<K, kWarps>(s_ex, (int)(round & 1), c.warp, c.lane, c.rank, c.ranks, A, B, cut != 0, carry, h);
        if (c.live && valid > 0) {
            if (p.saved) {
                float* to = p.saved + (c.b * c.tiles + tile) * p.channels + c.ch;
#pragma unroll
                for (int k = 0; k < K; ++k) to[k] = h[k];
            }
            T* to = y + tile * kTokens * p.y_token;
#pragma unroll
            for (int j = 0; j < kTokens; ++j) {
#pragma unroll
                for (int k = 0; k < K; ++k) h[k] = through(f[j][k], b[j][k], cut >> j & 1u, h[k]);
                if (j < valid) Cell<T, K>::store(to + j * p.y_token, h);
            }
        }
    }
    if (p.final_state && c.live && c.rank == 0 && c.warp == 0) {
#pragma unroll
        for (int k = 0; k < K; ++k) p.final_state[c.b * p.channels + c.ch + k] = carry[k];
    }
    if (c.ranks > 1) cg::this_cluster().sync();  // no CTA leaves while another writes to its shared memory
}

// --------------------------------------------------------------- gradient
// Warps, CTAs and rounds count from the end of the row.
template <class T, int K, bool kSigmoid, int kWarps>
__global__ void __launch_bounds__(32 * kWarps, (K == 2 ? 12 : 16) / kWarps) gated_grad_kernel(GatedParams p) {
    __shared__ Exchange<K, kWarps> s_ex;
    const Place c = place_of<K, kWarps>(p);
    const T* x = static_cast<const T*>(p.x) + c.b * p.x_batch + c.ch;
    const T* g = static_cast<const T*>(p.gate) + c.b * p.gate_batch + c.ch;
    const T* dy = static_cast<const T*>(p.dy) + c.b * p.dy_batch + c.ch;
    Cell<T, K> xr[kTokens], gr[kTokens], dr[kTokens];
    float start[K];
    uint32_t cuts;
    auto tokens = [&](long long tile) {
        return tile < 0 ? 0 : (int)max(0ll, min((long long)kTokens, p.length - tile * kTokens));
    };
    auto fetch = [&](long long tile) {
        const long long t0 = tile * kTokens;
        const int valid = c.live ? tokens(tile) : 0;
        load_tile<T, K>(x + t0 * p.x_token, p.x_token, valid, xr);
        load_tile<T, K>(g + t0 * p.gate_token, p.gate_token, valid, gr);
        load_tile<T, K>(dy + t0 * p.dy_token, p.dy_token, valid, dr);
        const float* from = p.saved + (c.b * c.tiles + tile) * p.channels + c.ch;
#pragma unroll
        for (int k = 0; k < K; ++k) start[k] = valid ? __ldg(from + k) : 0.0f;
        cuts = tile < 0 ? 0u : cuts_of(p.heads, c.b, t0, p.length, c.lane);
    };
    float carry[K], q[K];
#pragma unroll
    for (int k = 0; k < K; ++k) carry[k] = p.dfinal && c.live ? __ldg(p.dfinal + c.b * p.channels + c.ch + k) : 0.0f;
    const long long step = (long long)c.ranks * kWarps;
    long long tile = c.tiles - 1 - ((long long)c.rank * kWarps + c.warp);
    fetch(tile);
    if (c.ranks > 1) cg::this_cluster().sync();  // every CTA has begun before one writes to its shared memory
    for (long long round = 0; round < c.rounds; ++round, tile -= step) {
        // u: what dh is multiplied with for dgate; w: for dx (sigmoid), or f itself
        float u[kTokens][K], w[kTokens][K], h[K];
        Cell<T, K> d[kTokens];
        const uint32_t cut = cuts;
        const int valid = tokens(tile);
#pragma unroll
        for (int k = 0; k < K; ++k) h[k] = start[k];
#pragma unroll
        for (int j = 0; j < kTokens; ++j) {
            d[j] = dr[j];
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const float xv = xr[j].get(k), gv = gr[j].get(k);
                if (cut >> j & 1u) h[k] = 0.0f;
                if constexpr (kSigmoid) {
                    float f;
                    gate_of<T>(gv, f, w[j][k]);
                    u[j][k] = (h[k] - xv) * (f * w[j][k]);
                    h[k] = fmaf(f, h[k], w[j][k] * xv);
                } else {
                    w[j][k] = gv;
                    u[j][k] = h[k];
                    h[k] = cut >> j & 1u ? xv : fmaf(gv, h[k], xv);
                }
            }
        }
        if (round + 1 < c.rounds) fetch(tile - step);
        if (valid < kTokens) {  // behind the row's end: q stays
#pragma unroll
            for (int j = 0; j < kTokens; ++j)
#pragma unroll
                for (int k = 0; k < K; ++k)
                    if (j >= valid) w[j][k] = kSigmoid ? 0.0f : 1.0f;
        }
        // f from 1 - f: it adds to q with its absolute error, 2^-25
        auto decay_at = [&](int j, int k) { return kSigmoid ? 1.0f - w[j][k] : w[j][k]; };
        float A[K], B[K];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            A[k] = 1.0f;
            B[k] = 0.0f;
        }
#pragma unroll
        for (int j = kTokens - 1; j >= 0; --j)
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const float f = decay_at(j, k);
                A[k] *= f;
                B[k] = cut >> j & 1u ? 0.0f : f * (d[j].get(k) + B[k]);
            }
        exchange<K, kWarps>(s_ex, (int)(round & 1), c.warp, c.lane, c.rank, c.ranks, A, B, cut != 0, carry, q);
        if (c.live && valid > 0) {
            const long long to = (c.b * p.length + tile * kTokens) * p.channels + c.ch;
            T* dx = static_cast<T*>(p.dx) + to;
            T* dg = static_cast<T*>(p.dgate) + to;
#pragma unroll
            for (int j = kTokens - 1; j >= 0; --j) {
                float ox[K], og[K];
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    const float dh = d[j].get(k) + q[k];
                    ox[k] = kSigmoid ? dh * w[j][k] : dh;
                    og[k] = !kSigmoid && (cut >> j & 1u) ? 0.0f : dh * u[j][k];
                    q[k] = cut >> j & 1u ? 0.0f : decay_at(j, k) * dh;
                }
                if (j < valid) {
                    Cell<T, K>::store(dx + j * p.channels, ox);
                    Cell<T, K>::store(dg + j * p.channels, og);
                }
            }
        }
    }
    if (p.dstate && c.live && c.rank == 0 && c.warp == 0) {
#pragma unroll
        for (int k = 0; k < K; ++k) p.dstate[c.b * p.channels + c.ch + k] = carry[k];
    }
    if (c.ranks > 1) cg::this_cluster().sync();
}

// -------------------------------------------------------------- one token
constexpr int kStepNT = 128;
template <class T, int K, bool kSigmoid>
__global__ void __launch_bounds__(kStepNT) gated_step_kernel(GatedParams p) {
    const unsigned blocks = (unsigned)((p.channels + kStepNT * K - 1) / (kStepNT * K));
    const long long row = blockIdx.x / blocks, ch = ((long long)(blockIdx.x % blocks) * kStepNT + threadIdx.x) * K;
    if (ch >= p.channels) return;
    const long long slot = p.slots ? __ldg(p.slots + row) : row;
    T* y = static_cast<T*>(p.y) + row * p.y_batch + ch;
    const T* xp = static_cast<const T*>(p.x) + row * p.x_batch + ch;
    const T* gp = static_cast<const T*>(p.gate) + row * p.gate_batch + ch;
    float x[K], g[K], h[K];
    const bool live = slot >= 0 && slot < p.pool_rows;
    float* state = p.pool + (live ? slot : 0) * p.channels + ch;
    if constexpr (K == 4) {
        Vec<T, 4> xv, gv;
        Vec<float, 4> hv;
        xv.load(xp);
        gv.load(gp);
        if (live) hv.load_rw(state);
        else hv.zero();
#pragma unroll
        for (int k = 0; k < K; ++k) {
            x[k] = xv.get(k);
            g[k] = gv.get(k);
            h[k] = hv.get(k);
        }
    } else {
        x[0] = to_f32(*xp);
        g[0] = to_f32(*gp);
        h[0] = live ? *state : 0.0f;
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
        if constexpr (kSigmoid) {
            float f, rest;
            gate_of<T>(g[k], f, rest);
            h[k] = fmaf(f, h[k], rest * x[k]);
        } else {
            h[k] = fmaf(g[k], h[k], x[k]);
        }
        if (!live) h[k] = 0.0f;
    }
    if constexpr (K == 4) {
        Vec<T, 4> o;
        o.set(h);
        o.store(y);
        if (live) {
            Vec<float, 4> hv;
            hv.set(h);
            hv.store(state);
        }
    } else {
        *y = from_f32<T>(h[0]);
        if (live) *state = h[0];
    }
}

// ---------------------------------------------------------------- launch
// CTAs in a cluster: enough that the machine has about two CTAs an SM, but no more
// than the length has rounds for.
inline int cluster_of(long long groups, long long tiles, int warps) {
    int n = 1;
    while (n < kMaxCluster && groups * n < 2 * seq_sms() && (long long)n * warps < tiles) n *= 2;
    return n;
}

template <class T, int K, bool kSigmoid, int kWarps>
cudaError_t go(const GatedParams& p, bool grad, cudaStream_t s) {
    const long long tiles = (p.length + kTokens - 1) / kTokens, groups = p.batch * ((p.channels + 32 * K - 1) / (32 * K));
    const int n = cluster_of(groups, tiles, kWarps);
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(groups * n));
    cfg.blockDim = dim3(32 * kWarps);
    cfg.stream = s;
    cudaLaunchAttribute a{};
    a.id = cudaLaunchAttributeClusterDimension;
    a.val.clusterDim.x = (unsigned)n;
    a.val.clusterDim.y = a.val.clusterDim.z = 1;
    cfg.attrs = &a;
    cfg.numAttrs = 1;
    const cudaError_t e = grad ? cudaLaunchKernelEx(&cfg, gated_grad_kernel<T, K, kSigmoid, kWarps>, p)
                               : cudaLaunchKernelEx(&cfg, gated_kernel<T, K, kSigmoid, kWarps>, p);
    count_launches(1);
    return e;
}

template <class T, int K, bool kSigmoid>
cudaError_t by_length(const GatedParams& p, bool grad, cudaStream_t s) {
    const long long tiles = (p.length + kTokens - 1) / kTokens;
    if (tiles <= 1) return go<T, K, kSigmoid, 1>(p, grad, s);
    if (tiles <= 4) return go<T, K, kSigmoid, 4>(p, grad, s);
    return go<T, K, kSigmoid, 8>(p, grad, s);
}

template <class T, int K>
cudaError_t by_gate(const GatedParams& p, bool grad, cudaStream_t s) {
    return p.sigmoid ? by_length<T, K, true>(p, grad, s) : by_length<T, K, false>(p, grad, s);
}

template <class T>
cudaError_t launch_gated_as(const GatedParams& p, bool grad, cudaStream_t s) {
    if constexpr (sizeof(T) == 2) {
        if (p.pairs) return by_gate<T, 2>(p, grad, s);
    }
    return by_gate<T, 1>(p, grad, s);
}

template <class T, int K>
cudaError_t step_by_gate(const GatedParams& p, cudaStream_t s) {
    const unsigned grid = (unsigned)(p.batch * ((p.channels + kStepNT * K - 1) / (kStepNT * K)));
    if (p.sigmoid) gated_step_kernel<T, K, true><<<grid, kStepNT, 0, s>>>(p);
    else gated_step_kernel<T, K, false><<<grid, kStepNT, 0, s>>>(p);
    count_launches(1);
    return cudaGetLastError();
}
template <class T>
cudaError_t launch_gated_step_as(const GatedParams& p, cudaStream_t s) {
    return p.vec ? step_by_gate<T, 4>(p, s) : step_by_gate<T, 1>(p, s);
}

}  // namespace

// By element type, one translation unit each.
cudaError_t launch_gated_f32(const GatedParams& p, bool grad, cudaStream_t s);
cudaError_t launch_gated_f16(const GatedParams& p, bool grad, cudaStream_t s);
cudaError_t launch_gated_bf16(const GatedParams& p, bool grad, cudaStream_t s);

}  // namespace scg
