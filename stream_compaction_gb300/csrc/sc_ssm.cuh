// Shared pieces of the selective scan's kernels: how a warp's lanes divide
// channels and states, how a tile of tokens is read, and the sums across lanes.
//
// A warp owns CH neighbouring channels and walks the tokens in tiles of kTile.
// S lanes share a channel group, four states each (n = 4 s + k), and a lane
// serves CPL channels, so that every B or C value that a lane reads from shared
// memory serves CPL channels and every d or d*x value four states:
//
//     states   S   channels per lane   channels per warp
//     <= 8     2          2                  32
//     <= 16    4          4                  32
//     <= 32    8          4                  16
//     <= 64   16          4                   8
//
// Channels go in pairs through the two-lane float32 instructions; B and C lie
// in shared memory as (v, v) pairs for them.  States beyond `states` have
// A = B = C = 0 and stay 0.  Tokens beyond the length have d = d*x = 0: the
// state passes them unchanged.
#pragma once
#include "sc_seq.cuh"
#include "sc_seq_launch.h"

namespace scg {

constexpr int kTile = SC_SSM_SAVE;

template <int S_>
struct Geo {
    static constexpr int S = S_;
    static constexpr int CPL = S == 2 ? 2 : 4;
    static constexpr int PC = CPL / 2;       // channel pairs per lane
    static constexpr int CL = 32 / S;        // lanes along the channels
    static constexpr int CH = CL * CPL;
    static constexpr int NP = 4 * S;         // padded states
    static constexpr int kWarps = S == 16 ? 2 : 4;
    static constexpr int kThreads = 32 * kWarps;
    static constexpr int kBlockCh = kWarps * CH;
};

// Which channels, chunk of the length and row a CTA works on.
template <class G>
struct SsmPlace {
    long long b, chunk, cblock, group, ch0, left;  // ch0: the warp's first channel; left: its channels (may be <= 0)
    __device__ __forceinline__ SsmPlace(const SsmParams& p, long long blocks_per_group, int chunks) {
        const long long ncb = blocks_per_group * p.groups;
        cblock = blockIdx.x % ncb;
        const long long q = blockIdx.x / ncb;
        chunk = q % chunks;
        b = q / chunks;
        group = cblock / blocks_per_group;
        const long long per = p.channels / p.groups;
        const long long in = (cblock % blocks_per_group) * G::kBlockCh + (threadIdx.x >> 5) * G::CH;
        ch0 = group * per + in;
        left = per - in < G::CH ? per - in : G::CH;
    }
};

// One tile of a batch x length x channels tensor: kTile tokens of the warp's
// channels, each lane a fixed set of (token, channel).
// kVec: eight neighbouring channels at a time in 16-byte accesses (channels a
// multiple of 8); else one element at a time, lanes along the channels.
template <class T, class G, bool kVec>
struct TileRows;

template <class T, class G>
struct TileRows<T, G, true> {
    static constexpr int LPT = G::CH / 8;              // lanes per token
    static constexpr int TP = 32 / LPT;                // tokens per access
    static constexpr int NA = TP >= kTile ? 1 : kTile / TP;
    static constexpr int kCount = 8 * NA;
    static constexpr int kChannels = 8;                // distinct channels of a lane: those of elements 0 .. 7
    Vec<T, 8> v[NA];
    __device__ __forceinline__ static int tok(int i, int lane) { return lane / LPT + (i / 8) * TP; }
    __device__ __forceinline__ static int ch(int i, int lane) { return (lane % LPT) * 8 + i % 8; }
    __device__ __forceinline__ static bool valid(int i, int lane, int nt, int left) {
        return tok(i, lane) < nt && (lane % LPT) * 8 < left;
    }
    __device__ __forceinline__ void load(const T* p, long long stride, int nt, int left, int lane) {
#pragma unroll
        for (int a = 0; a < NA; ++a) {
            v[a].zero();
            if (valid(8 * a, lane, nt, left)) v[a].load(p + tok(8 * a, lane) * stride + (lane % LPT) * 8);
        }
    }
    __device__ __forceinline__ float get(int i) const { return v[i / 8].get(i % 8); }
    // a lane's values into a [kTile][CH] array of shared memory
    __device__ __forceinline__ static void to_shared(float* s, const float (&f)[kCount], int lane) {
#pragma unroll
        for (int a = 0; a < NA; ++a) {
            if (tok(8 * a, lane) < kTile) {
                float4* q = reinterpret_cast<float4*>(s + tok(8 * a, lane) * G::CH + (lane % LPT) * 8);
                q[0] = make_float4(f[8 * a], f[8 * a + 1], f[8 * a + 2], f[8 * a + 3]);
                q[1] = make_float4(f[8 * a + 4], f[8 * a + 5], f[8 * a + 6], f[8 * a + 7]);
            }
        }
    }
    __device__ __forceinline__ static void from_shared(const float* s, float (&f)[kCount], int lane) {
#pragma unroll
        for (int a = 0; a < NA; ++a) {
            if (tok(8 * a, lane) < kTile) {
                const float4* q = reinterpret_cast<const float4*>(s + tok(8 * a, lane) * G::CH + (lane % LPT) * 8);
                const float4 x = q[0], y = q[1];
                f[8 * a] = x.x; f[8 * a + 1] = x.y; f[8 * a + 2] = x.z; f[8 * a + 3] = x.w;
                f[8 * a + 4] = y.x; f[8 * a + 5] = y.y; f[8 * a + 6] = y.z; f[8 * a + 7] = y.w;
            }
        }
    }
    __device__ __forceinline__ static void store(T* p, long long stride, const float (&f)[kCount], int nt, int left,
                                                 int lane) {
#pragma unroll
        for (int a = 0; a < NA; ++a)
            if (valid(8 * a, lane, nt, left)) {
                Vec<T, 8> q;
                q.set(f + 8 * a);
                q.store(p + tok(8 * a, lane) * stride + (lane % LPT) * 8);
            }
    }
    // sums over a lane's tokens -> over all tokens; true on the lanes that hold them
    __device__ __forceinline__ static bool sum_tokens(float (&c)[kChannels], int lane) {
#pragma unroll
        for (int m = LPT; m < 32; m <<= 1)
#pragma unroll
            for (int i = 0; i < kChannels; ++i) c[i] += __shfl_xor_sync(0xffffffffu, c[i], m);
        return lane < LPT;
    }
    __device__ __forceinline__ static int channel_of(int i) { return i % 8; }
};

template <class T, class G>
struct TileRows<T, G, false> {
    static constexpr int TP = 32 / G::CH;
    static constexpr int kCount = kTile / TP;
    static constexpr int kChannels = 1;
    T v[kCount];
    __device__ __forceinline__ static int tok(int i, int lane) { return lane / G::CH + i * TP; }
    __device__ __forceinline__ static int ch(int, int lane) { return lane % G::CH; }
    __device__ __forceinline__ static bool valid(int i, int lane, int nt, int left) {
        return tok(i, lane) < nt && lane % G::CH < left;
    }
    __device__ __forceinline__ void load(const T* p, long long stride, int nt, int left, int lane) {
#pragma unroll
        for (int i = 0; i < kCount; ++i) {
            v[i] = from_f32<T>(0.0f);
            if (valid(i, lane, nt, left)) v[i] = __ldg(p + tok(i, lane) * stride + lane % G::CH);
        }
    }
    __device__ __forceinline__ float get(int i) const { return to_f32(v[i]); }
    __device__ __forceinline__ static void to_shared(float* s, const float (&f)[kCount], int lane) {
#pragma unroll
        for (int i = 0; i < kCount; ++i) s[tok(i, lane) * G::CH + lane % G::CH] = f[i];
    }
    __device__ __forceinline__ static void from_shared(const float* s, float (&f)[kCount], int lane) {
#pragma unroll
        for (int i = 0; i < kCount; ++i) f[i] = s[tok(i, lane) * G::CH + lane % G::CH];
    }
    __device__ __forceinline__ static void store(T* p, long long stride, const float (&f)[kCount], int nt, int left,
                                                 int lane) {
#pragma unroll
        for (int i = 0; i < kCount; ++i)
            if (valid(i, lane, nt, left)) p[tok(i, lane) * stride + lane % G::CH] = from_f32<T>(f[i]);
    }
    __device__ __forceinline__ static bool sum_tokens(float (&c)[kChannels], int lane) {
#pragma unroll
        for (int m = G::CH; m < 32; m <<= 1) c[0] += __shfl_xor_sync(0xffffffffu, c[0], m);
        return lane < G::CH;
    }
    __device__ __forceinline__ static int channel_of(int) { return 0; }
};

// One tile of B or C (a group's states of kTile tokens), to (v, v) pairs.
template <class T, class G, bool kVec>
struct TileStates;

template <class T, class G>
struct TileStates<T, G, true> {  // states a multiple of 8
    static constexpr int PT = G::NP / 8;                              // eights per token
    static constexpr int NA = (kTile * PT + 31) / 32;
    Vec<T, 8> v[NA];
    __device__ __forceinline__ void load(const T* p, long long stride, int nt, int states, int lane) {
#pragma unroll
        for (int a = 0; a < NA; ++a) {
            const int q = lane + 32 * a, t = q / PT, n = (q % PT) * 8;
            v[a].zero();
            if (t < nt && n < states) v[a].load(p + t * stride + n);
        }
    }
    __device__ __forceinline__ void to_shared(float2* s, int lane) const {
#pragma unroll
        for (int a = 0; a < NA; ++a) {
            const int q = lane + 32 * a;
            if (q < kTile * PT) {
                float4* o = reinterpret_cast<float4*>(s + q * 8);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    o[i] = make_float4(v[a].get(2 * i), v[a].get(2 * i), v[a].get(2 * i + 1), v[a].get(2 * i + 1));
            }
        }
    }
};

template <class T, class G>
struct TileStates<T, G, false> {
    static constexpr int NA = kTile * G::NP / 32;
    T v[NA];
    __device__ __forceinline__ void load(const T* p, long long stride, int nt, int states, int lane) {
#pragma unroll
        for (int a = 0; a < NA; ++a) {
            const int q = lane + 32 * a, t = q / G::NP, n = q % G::NP;
            v[a] = from_f32<T>(0.0f);
            if (t < nt && n < states) v[a] = __ldg(p + t * stride + n);
        }
    }
    __device__ __forceinline__ void to_shared(float2* s, int lane) const {
#pragma unroll
        for (int a = 0; a < NA; ++a) s[lane + 32 * a] = make_float2(to_f32(v[a]), to_f32(v[a]));
    }
};

// CPL neighbouring floats of shared memory as channel pairs, and four (v, v) pairs.
template <class G>
__device__ __forceinline__ void read_channels(const float* s, f2 (&v)[G::PC]) {
    if constexpr (G::PC == 2) {
        const ulonglong2 q = *reinterpret_cast<const ulonglong2*>(s);
        v[0] = q.x;
        v[1] = q.y;
    } else {
        v[0] = *reinterpret_cast<const f2*>(s);
    }
}
__device__ __forceinline__ void read_states(const float2* s, f2 (&v)[4]) {
    const ulonglong2 a = reinterpret_cast<const ulonglong2*>(s)[0], b = reinterpret_cast<const ulonglong2*>(s)[1];
    v[0] = a.x;
    v[1] = a.y;
    v[2] = b.x;
    v[3] = b.y;
}

// Sum over the S lanes of a channel group; lane s < CPL of it gets channel s of
// the lane's CPL (the other lanes copies).
template <class G>
__device__ __forceinline__ float sum_states(const f2 (&v)[G::PC], int lane) {
    float r;
    if constexpr (G::PC == 2) {
        const bool b0 = lane & 1, b1 = lane & 2;
        const float a = lo2(v[0]), b = hi2(v[0]), c = lo2(v[1]), d = hi2(v[1]);
        const float x = (b0 ? b : a) + __shfl_xor_sync(0xffffffffu, b0 ? a : b, 1);
        const float y = (b0 ? d : c) + __shfl_xor_sync(0xffffffffu, b0 ? c : d, 1);
        r = (b1 ? y : x) + __shfl_xor_sync(0xffffffffu, b1 ? x : y, 2);
#pragma unroll
        for (int m = 4; m < G::S; m <<= 1) r += __shfl_xor_sync(0xffffffffu, r, m);
    } else {
        const bool b0 = lane & 1;
        const float a = lo2(v[0]), b = hi2(v[0]);
        r = (b0 ? b : a) + __shfl_xor_sync(0xffffffffu, b0 ? a : b, 1);
    }
    return r;
}

// A lane's four states of each of its channels, in rows of NP floats per channel.
template <class G>
__device__ __forceinline__ void load_lane(const float* p, int left, int lane, float (&v)[G::CPL][4]) {
    const int s = lane % G::S, c = lane / G::S;
#pragma unroll
    for (int j = 0; j < G::CPL; ++j) {
        float4 q = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (G::CPL * c + j < left) q = *reinterpret_cast<const float4*>(p + (long long)(G::CPL * c + j) * G::NP + 4 * s);
        v[j][0] = q.x;
        v[j][1] = q.y;
        v[j][2] = q.z;
        v[j][3] = q.w;
    }
}
template <class G>
__device__ __forceinline__ void store_lane(float* p, int left, int lane, const f2 (&v)[G::PC][4]) {
    const int s = lane % G::S, c = lane / G::S;
#pragma unroll
    for (int j = 0; j < G::CPL; ++j)
        if (G::CPL * c + j < left) {
            const f2(&r)[4] = v[j / 2];
            *reinterpret_cast<float4*>(p + (long long)(G::CPL * c + j) * G::NP + 4 * s) =
                j & 1 ? make_float4(hi2(r[0]), hi2(r[1]), hi2(r[2]), hi2(r[3]))
                      : make_float4(lo2(r[0]), lo2(r[1]), lo2(r[2]), lo2(r[3]));
        }
}
// The same in rows of `states` floats (the caller's layout), element by element.
template <class G>
__device__ __forceinline__ void load_lane_of(const float* p, long long states, int left, int lane,
                                             float (&v)[G::CPL][4]) {
    const int s = lane % G::S, c = lane / G::S;
#pragma unroll
    for (int j = 0; j < G::CPL; ++j)
#pragma unroll
        for (int k = 0; k < 4; ++k)
            v[j][k] = p && G::CPL * c + j < left && 4 * s + k < states ? p[(G::CPL * c + j) * states + 4 * s + k] : 0.0f;
}
template <class G>
__device__ __forceinline__ void store_lane_of(float* p, long long states, int left, int lane, const f2 (&v)[G::PC][4]) {
    const int s = lane % G::S, c = lane / G::S;
#pragma unroll
    for (int j = 0; j < G::CPL; ++j)
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (G::CPL * c + j < left && 4 * s + k < states)
                p[(G::CPL * c + j) * states + 4 * s + k] = j & 1 ? hi2(v[j / 2][k]) : lo2(v[j / 2][k]);
}
template <class G>
__device__ __forceinline__ void to_pairs(const float (&v)[G::CPL][4], float scale, f2 (&o)[G::PC][4]) {
#pragma unroll
    for (int q = 0; q < G::PC; ++q)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[q][k] = pack2(v[2 * q][k] * scale, v[2 * q + 1][k] * scale);
}

// Bit t: a segment starts at token t of the tile.
__device__ __forceinline__ unsigned tile_heads(const uint8_t* row, long long t0, int nt, int lane) {
    if (!row) return 0u;
    return __ballot_sync(0xffffffffu, lane < nt && row[t0 + (lane < nt ? lane : 0)] != 0);
}

// carry = decay of chunk j over its whole length * carry + what the chunk adds.
template <class G>
__device__ __forceinline__ void fold_chunk(const SsmParams& p, const f2 (&A2)[G::PC][4], long long b, long long j,
                                           long long ch0, int left, int lane, f2 (&carry)[G::PC][4]) {
    const long long row = b * p.chunks + j;
    float v[G::CPL][4], d[G::CPL];
    load_lane<G>(p.carry + (row * p.channels + ch0) * G::NP, left, lane, v);
    const int c = lane / G::S;
#pragma unroll
    for (int i = 0; i < G::CPL; ++i)
        d[i] = G::CPL * c + i < left ? p.sum_d[row * p.channels + ch0 + G::CPL * c + i] : 0.0f;
    const bool cut = p.cut[row] != 0;
#pragma unroll
    for (int q = 0; q < G::PC; ++q)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const f2 add = pack2(v[2 * q][k], v[2 * q + 1][k]);
            const f2 a = ex2_2(mul2(pack2(d[2 * q], d[2 * q + 1]), A2[q][k]));
            carry[q][k] = cut ? add : fma2(a, carry[q][k], add);
        }
}

}  // namespace scg
