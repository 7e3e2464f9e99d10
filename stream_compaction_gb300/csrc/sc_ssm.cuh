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
// Channels go in pairs through the two-lane float32 instructions (one issue
// slot for two multiply-adds; measured: two clocks each, so they relieve the
// issue, not the multipliers); B and C lie in shared memory as (v, v) pairs for
// them.  States beyond `states` have A = B = C = 0 and stay 0; tiles with an infinity
// or NaN, whose products with those zeros would be NaN, set them to 0 instead.  Tokens
// beyond the length have d = d*x = 0: the state passes them unchanged.
//
// The elements of a tile (token, channel) are worked on in passes of 128, four
// a lane: four channels of one token (kVec: 8 or 16-byte accesses, channels
// and strides multiples of 4), or one channel of four tokens.
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
    static constexpr int TP = 128 / CH;      // tokens of a pass
    // Sums over a channel's states: up to 4 lanes leave their parts in shared
    // memory for the pass that uses the sum (one store and S loads for every four
    // channels); 8 or 16 lanes' parts would crowd it, so those add across lanes first.
    static constexpr bool kParts = S <= 4;
    static constexpr int kSumRows = kParts ? S : 1;
    static constexpr int kSumRow = kSumRows * CH;  // floats per token
    // Row j of the parts has its channels at exchanged places, fours apart, so
    // that the S lanes of a channel group meet in no bank.
    __device__ __forceinline__ static int place(int j, int ch) { return j * CH + (ch ^ (j * (S == 4 ? 8 : 16))); }
    static constexpr int kBwdWarps = S == 16 ? 2 : 4;
};

// Which channels, chunk of the length and row a CTA works on.
template <class G, int kWarps>
struct SsmPlace {
    long long b, chunk, cblock, group, ch0;  // ch0: the warp's first channel
    int left;                                // its channels (0: none)
    // warp: the one of kWarps whose channels these are
    __device__ __forceinline__ SsmPlace(const SsmParams& p, int blocks_per_group, int chunks, int warp) {
        const int ncb = blocks_per_group * (int)p.groups;
        const unsigned q = blockIdx.x / (unsigned)ncb;
        cblock = blockIdx.x % (unsigned)ncb;
        chunk = q % (unsigned)chunks;
        b = q / (unsigned)chunks;
        group = cblock / blocks_per_group;
        const long long per = p.channels / p.groups;
        const long long in = (cblock % blocks_per_group) * (kWarps * G::CH) + warp * G::CH;
        ch0 = group * per + in;
        left = per - in < G::CH ? (per > in ? (int)(per - in) : 0) : G::CH;
    }
};

// Tokens of the tile of kT that starts at t0.
template <int kT>
__device__ __forceinline__ int tile_tokens(const SsmParams& p, long long t0) {
    const long long n = p.length - t0;
    return n < kT ? (int)n : kT;
}

// One tile (kT tokens) of a batch x length x channels tensor.
template <class T, class G, bool kVec, int kT>
struct TileRows;

template <class T, class G, int kT>
struct TileRows<T, G, true, kT> {
    static constexpr int LPT = G::CH / 4;  // lanes per token
    static constexpr int NA = kT / G::TP;  // passes
    Vec<T, 4> v[NA];
    __device__ __forceinline__ static int tok(int a, int lane) { return a * G::TP + lane / LPT; }
    __device__ __forceinline__ static int ch(int lane) { return (lane % LPT) * 4; }
    template <bool kFull>
    __device__ __forceinline__ static Vec<T, 4> fetch(const T* p, long long stride, int a, int nt, int left, int lane) {
        Vec<T, 4> q;
        if constexpr (!kFull) q.zero();
        if (kFull || (tok(a, lane) < nt && ch(lane) < left)) q.load(p + tok(a, lane) * stride + ch(lane));
        return q;
    }
    template <bool kFull>
    __device__ __forceinline__ void load(const T* p, long long stride, int nt, int left, int lane) {
#pragma unroll
        for (int a = 0; a < NA; ++a) v[a] = fetch<kFull>(p, stride, a, nt, left, lane);
    }
    __device__ __forceinline__ f2 pair(int a, int i) const { return v[a].pair(i); }
    __device__ __forceinline__ static f2 pair_of(const Vec<T, 4>& q, int i) { return q.pair(i); }
    // zeros for elements past the tokens or channels
    template <bool kFull>
    __device__ __forceinline__ static void mask(f2 (&f)[2], int a, int nt, int left, int lane) {
        if (!kFull && (tok(a, lane) >= nt || ch(lane) >= left)) f[0] = f[1] = 0ull;
    }
    // the pass's elements of a [tokens][CH] array whose row 0 is the pass's first token
    __device__ __forceinline__ static void put(float* s, const f2 (&f)[2], int lane) {
        *reinterpret_cast<ulonglong2*>(s + lane / LPT * G::CH + ch(lane)) = make_ulonglong2(f[0], f[1]);
    }
    __device__ __forceinline__ static void get(const float* s, f2 (&f)[2], int lane) {
        const ulonglong2 q = *reinterpret_cast<const ulonglong2*>(s + lane / LPT * G::CH + ch(lane));
        f[0] = q.x;
        f[1] = q.y;
    }
    // the same of a [tokens][kSumRow] array, the lanes' parts added
    __device__ __forceinline__ static void get_sums(const float* s, f2 (&f)[2], int lane) {
        const float* r = s + lane / LPT * G::kSumRow;
        const ulonglong2 q = *reinterpret_cast<const ulonglong2*>(r + ch(lane));
        f[0] = q.x;
        f[1] = q.y;
#pragma unroll
        for (int j = 1; j < G::kSumRows; ++j) {
            const ulonglong2 o = *reinterpret_cast<const ulonglong2*>(r + G::place(j, ch(lane)));
            f[0] = add2(f[0], o.x);
            f[1] = add2(f[1], o.y);
        }
    }
    template <bool kFull>
    __device__ __forceinline__ static void store(T* p, long long stride, const f2 (&f)[2], int a, int nt, int left,
                                                 int lane) {
        if (kFull || (tok(a, lane) < nt && ch(lane) < left)) {
            Vec<T, 4> q;
            q.set_pairs(f);
            q.store(p + tok(a, lane) * stride + ch(lane));
        }
    }
    // a value per channel, as a lane's elements meet it
    __device__ __forceinline__ static void per_channel(const float* p, int left, int lane, f2 (&f)[2]) {
        const int c = ch(lane);
        float v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = p && c + i < left ? __ldg(p + c + i) : 0.0f;
        f[0] = pack2(v[0], v[1]);
        f[1] = pack2(v[2], v[3]);
    }
    // the same from a [CH] array in shared memory
    __device__ __forceinline__ static void channel_values(const float* s, f2 (&f)[2], int lane) {
        const ulonglong2 q = *reinterpret_cast<const ulonglong2*>(s + ch(lane));
        f[0] = q.x;
        f[1] = q.y;
    }
    // sums per channel over all passes, written
    __device__ __forceinline__ static void put_channel_sums(float* p, const f2 (&f)[2], int left, int lane) {
        float v[4] = {lo2(f[0]), hi2(f[0]), lo2(f[1]), hi2(f[1])};
#pragma unroll
        for (int m = LPT; m < 32; m <<= 1)
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], m);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (lane < LPT && ch(lane) + i < left) p[ch(lane) + i] = v[i];
    }
};

template <class T, class G, int kT>
struct TileRows<T, G, false, kT> {
    static constexpr int TL = 32 / G::CH;  // tokens side by side
    static constexpr int NA = kT / G::TP;
    struct Four { T e[4]; };
    Four v[NA];
    __device__ __forceinline__ static int tok(int a, int i, int lane) { return a * G::TP + i * TL + lane / G::CH; }
    __device__ __forceinline__ static bool valid(int a, int i, int nt, int left, int lane) {
        return tok(a, i, lane) < nt && lane % G::CH < left;
    }
    template <bool kFull>
    __device__ __forceinline__ static Four fetch(const T* p, long long stride, int a, int nt, int left, int lane) {
        Four q;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (!kFull) q.e[i] = from_f32<T>(0.0f);
            if (kFull || valid(a, i, nt, left, lane)) q.e[i] = __ldg(p + tok(a, i, lane) * stride + lane % G::CH);
        }
        return q;
    }
    template <bool kFull>
    __device__ __forceinline__ void load(const T* p, long long stride, int nt, int left, int lane) {
#pragma unroll
        for (int a = 0; a < NA; ++a) v[a] = fetch<kFull>(p, stride, a, nt, left, lane);
    }
    __device__ __forceinline__ f2 pair(int a, int i) const { return pair_of(v[a], i); }
    __device__ __forceinline__ static f2 pair_of(const Four& q, int i) {
        return pack2(to_f32(q.e[2 * i]), to_f32(q.e[2 * i + 1]));
    }
    template <bool kFull>
    __device__ __forceinline__ static void mask(f2 (&f)[2], int a, int nt, int left, int lane) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (!kFull)
                f[i] = pack2(valid(a, 2 * i, nt, left, lane) ? lo2(f[i]) : 0.0f,
                             valid(a, 2 * i + 1, nt, left, lane) ? hi2(f[i]) : 0.0f);
    }
    __device__ __forceinline__ static int at(int i, int lane) {
        return (i * TL + lane / G::CH) * G::CH + lane % G::CH;
    }
    __device__ __forceinline__ static void put(float* s, const f2 (&f)[2], int lane) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            s[at(2 * i, lane)] = lo2(f[i]);
            s[at(2 * i + 1, lane)] = hi2(f[i]);
        }
    }
    __device__ __forceinline__ static void get(const float* s, f2 (&f)[2], int lane) {
#pragma unroll
        for (int i = 0; i < 2; ++i) f[i] = pack2(s[at(2 * i, lane)], s[at(2 * i + 1, lane)]);
    }
    __device__ __forceinline__ static void get_sums(const float* s, f2 (&f)[2], int lane) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float *x = s + (2 * i * TL + lane / G::CH) * G::kSumRow, *y = x + TL * G::kSumRow;
            f[i] = pack2(x[lane % G::CH], y[lane % G::CH]);
#pragma unroll
            for (int j = 1; j < G::kSumRows; ++j)
                f[i] = add2(f[i], pack2(x[G::place(j, lane % G::CH)], y[G::place(j, lane % G::CH)]));
        }
    }
    template <bool kFull>
    __device__ __forceinline__ static void store(T* p, long long stride, const f2 (&f)[2], int a, int nt, int left,
                                                 int lane) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (kFull || valid(a, i, nt, left, lane))
                p[tok(a, i, lane) * stride + lane % G::CH] = from_f32<T>(i & 1 ? hi2(f[i / 2]) : lo2(f[i / 2]));
    }
    __device__ __forceinline__ static void per_channel(const float* p, int left, int lane, f2 (&f)[2]) {
        f[0] = f[1] = both(p && lane % G::CH < left ? __ldg(p + lane % G::CH) : 0.0f);
    }
    __device__ __forceinline__ static void channel_values(const float* s, f2 (&f)[2], int lane) {
        f[0] = f[1] = both(s[lane % G::CH]);
    }
    __device__ __forceinline__ static void put_channel_sums(float* p, const f2 (&f)[2], int left, int lane) {
        float v = (lo2(f[0]) + hi2(f[0])) + (lo2(f[1]) + hi2(f[1]));
#pragma unroll
        for (int m = G::CH; m < 32; m <<= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
        if (lane < G::CH && lane < left) p[lane] = v;
    }
};

// One tile of B or C (a group's states of kT tokens), to (v, v) pairs.
template <class T, class G, bool kVec, int kT>
struct TileStates;

template <class T, class G, int kT>
struct TileStates<T, G, true, kT> {  // states a multiple of 4
    static constexpr int NA = (kT * G::S + 31) / 32;  // fours per lane
    Vec<T, 4> v[NA];
    __device__ __forceinline__ void load(const T* p, long long stride, int nt, int states, int lane) {
#pragma unroll
        for (int a = 0; a < NA; ++a) {
            const int q = lane + 32 * a, t = q / G::S, n = (q % G::S) * 4;
            v[a].zero();
            if (t < nt && n < states) v[a].load(p + t * stride + n);
        }
    }
    __device__ __forceinline__ void to_shared(float2* s, int lane) const {
#pragma unroll
        for (int a = 0; a < NA; ++a) {
            if (lane + 32 * a >= kT * G::S) break;
            float4* o = reinterpret_cast<float4*>(s + (lane + 32 * a) * 4);
            o[0] = make_float4(v[a].get(0), v[a].get(0), v[a].get(1), v[a].get(1));
            o[1] = make_float4(v[a].get(2), v[a].get(2), v[a].get(3), v[a].get(3));
        }
    }
};

template <class T, class G, int kT>
struct TileStates<T, G, false, kT> {
    static constexpr int NA = kT * G::NP / 32;
    T v[NA];
    __device__ __forceinline__ void load(const T* p, long long stride, int nt, int states, int lane) {
#pragma unroll
        for (int a = 0; a < NA; ++a) {
            const int q = lane + 32 * a, t = q / G::NP, n = q % G::NP;
            v[a] = t < nt && n < states ? __ldg(p + t * stride + n) : from_f32<T>(0.0f);
        }
    }
    __device__ __forceinline__ void to_shared(float2* s, int lane) const {
#pragma unroll
        for (int a = 0; a < NA; ++a) s[lane + 32 * a] = make_float2(to_f32(v[a]), to_f32(v[a]));
    }
};

// The elements of a tile in shared memory ([kT][CH], raw or float32), in passes
// of 128: each lane four channels of one token.
template <class T, int CH, int kT>
struct TileElems {
    static constexpr int LPT = CH / 4;       // lanes per token
    static constexpr int TP = 128 / CH;      // tokens of a pass
    static constexpr int NA = kT / TP;       // passes
    __device__ __forceinline__ static int tok(int a, int lane) { return a * TP + lane / LPT; }
    __device__ __forceinline__ static int ch(int lane) { return (lane % LPT) * 4; }
    // s: the pass's first element
    template <class E>
    __device__ __forceinline__ static void get(const E* s, f2 (&f)[2], int lane) {
        Vec<E, 4> q;
        q.load_rw(s + 4 * lane);
        f[0] = q.pair(0);
        f[1] = q.pair(1);
    }
    template <bool kVec, bool kFull>
    __device__ __forceinline__ static void store(T* p, long long stride, const f2 (&f)[2], int a, int nt, int left,
                                                 int lane) {
        T* to = p + tok(a, lane) * stride + ch(lane);
        if (kFull || (tok(a, lane) < nt && ch(lane) < left)) {
            if constexpr (kVec) {
                Vec<T, 4> q;
                q.set_pairs(f);
                q.store(to);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (kFull || ch(lane) + i < left) to[i] = from_f32<T>(i & 1 ? hi2(f[i / 2]) : lo2(f[i / 2]));
            }
        }
    }
    // a value per channel, as a lane's elements meet it
    __device__ __forceinline__ static void per_channel(const float* p, int left, int lane, f2 (&f)[2]) {
        const int c = ch(lane);
        float v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = p && c + i < left ? __ldg(p + c + i) : 0.0f;
        f[0] = pack2(v[0], v[1]);
        f[1] = pack2(v[2], v[3]);
    }
};

// kN raw values to float32, by one warp.
template <class T, int kN>
__device__ __forceinline__ void put_floats(float* s, const T* raw, int lane) {
    static_assert(kN % 4 == 0, "fours");
#pragma unroll
    for (int i = 0; i < (kN / 4 + 31) / 32; ++i) {
        const int q = lane + 32 * i;
        if (kN / 4 % 32 != 0 && q >= kN / 4) break;
        Vec<T, 4> v;
        v.load_rw(raw + 4 * q);
        *reinterpret_cast<ulonglong2*>(s + 4 * q) = make_ulonglong2(v.pair(0), v.pair(1));
    }
}

// A lane's channels at one token of a [tokens][CH] array as pairs, and its four
// states of a [tokens][NP] array of (v, v) pairs.
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

// Sum over the S lanes of a channel group: lane s < CPL of it gets channel s of
// the lane's CPL (the other lanes copies).
template <class G>
__device__ __forceinline__ float sum_states(const f2 (&v)[G::PC], int lane) {
    static_assert(G::PC == 2, "four channels");
    const bool b0 = lane & 1, b1 = lane & 2;
    const float a = lo2(v[0]), b = hi2(v[0]), c = lo2(v[G::PC - 1]), d = hi2(v[G::PC - 1]);
    const float x = (b0 ? b : a) + __shfl_xor_sync(0xffffffffu, b0 ? a : b, 1);
    const float y = (b0 ? d : c) + __shfl_xor_sync(0xffffffffu, b0 ? c : d, 1);
    float r = (b1 ? y : x) + __shfl_xor_sync(0xffffffffu, b1 ? x : y, 2);
#pragma unroll
    for (int m = 4; m < G::S; m <<= 1) r += __shfl_xor_sync(0xffffffffu, r, m);
    return r;
}
// A lane's part of a sum over states, for TileRows::get_sums; row: the token's.
template <class G>
__device__ __forceinline__ void put_sums(float* row, const f2 (&v)[G::PC], int lane) {
    const int s = lane % G::S, c = lane / G::S;
    if constexpr (!G::kParts) {
        const float r = sum_states<G>(v, lane);
        if (s < G::CPL) row[G::CPL * c + s] = r;
    } else if constexpr (G::PC == 2) {
        *reinterpret_cast<ulonglong2*>(row + G::place(s, G::CPL * c)) = make_ulonglong2(v[0], v[1]);
    } else {
        *reinterpret_cast<f2*>(row + G::place(s, G::CPL * c)) = v[0];
    }
}

// A lane's four states of each of its channels in the library's own arrays,
// [fours of states][channels][4]; p: the warp's first channel of the first four.
template <class G>
__device__ __forceinline__ void load_lane(const float* p, long long channels, int left, int lane,
                                          float (&v)[G::CPL][4]) {
    const int s = lane % G::S, c = lane / G::S;
#pragma unroll
    for (int j = 0; j < G::CPL; ++j) {
        float4 q = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (G::CPL * c + j < left) q = *reinterpret_cast<const float4*>(p + (s * channels + G::CPL * c + j) * 4);
        v[j][0] = q.x;
        v[j][1] = q.y;
        v[j][2] = q.z;
        v[j][3] = q.w;
    }
}
template <class G>
__device__ __forceinline__ void store_lane(float* p, long long channels, int left, int lane, const f2 (&v)[G::PC][4]) {
    const int s = lane % G::S, c = lane / G::S;
#pragma unroll
    for (int j = 0; j < G::CPL; ++j)
        if (G::CPL * c + j < left) {
            const f2(&r)[4] = v[j / 2];
            *reinterpret_cast<float4*>(p + (s * channels + G::CPL * c + j) * 4) =
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
__device__ __forceinline__ void to_pairs(const float (&v)[G::CPL][4], f2 (&o)[G::PC][4]) {
#pragma unroll
    for (int q = 0; q < G::PC; ++q)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[q][k] = pack2(v[2 * q][k], v[2 * q + 1][k]);
}
template <class G>
__device__ __forceinline__ void to_rates(const float (&A)[G::CPL][4], f2 (&o)[G::PC][4]) {
#pragma unroll
    for (int q = 0; q < G::PC; ++q)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[q][k] = pack2(rate(A[2 * q][k]), rate(A[2 * q + 1][k]));
}
// The lane, asked for anew: what is made of it, seldom used, is not kept in registers.
__device__ __forceinline__ int lane_anew() {
    int lane;
    asm volatile("mov.u32 %0, %%laneid;" : "=r"(lane));
    return lane;
}
// Zeros for a lane's states beyond `states`.
template <class G>
__device__ __forceinline__ void drop_padding(long long states, f2 (&v)[G::PC][4]) {
    const int real = (int)states - lane_anew() % G::S * 4;
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int q = 0; q < G::PC; ++q)
            if (k >= real) v[q][k] = 0ull;
}
template <class G>
__device__ __forceinline__ void clear(f2 (&v)[G::PC][4]) {
#pragma unroll
    for (int q = 0; q < G::PC; ++q)
#pragma unroll
        for (int k = 0; k < 4; ++k) v[q][k] = 0ull;
}

// Bit t: a segment starts at token t of the tile.
__device__ __forceinline__ unsigned tile_heads(const uint8_t* row, long long t0, int nt, int lane) {
    if (!row) return 0u;
    return __ballot_sync(0xffffffffu, lane < nt && row[t0 + (lane < nt ? lane : 0)] != 0);
}

// carry = decay of run j over its whole length * carry + what the run adds.  (One
// exponential for the run: without the nudge that makes up for hundreds of them.)
template <class G, bool kPadded>
__device__ __forceinline__ void fold_run(const SsmParams& p, const f2 (&A2)[G::PC][4], long long b, long long j,
                                         long long ch0, int left, int lane, f2 (&carry)[G::PC][4]) {
    const long long row = b * p.runs + j;
    float v[G::CPL][4], d[G::CPL];
    load_lane<G>(p.carry + row * p.channels * G::NP + ch0 * 4, p.channels, left, lane, v);
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
    if constexpr (kPadded) drop_padding<G>(p.states, carry);
}
// The run's own part, left for the others to fold.
template <class G>
__device__ __forceinline__ void leave_run(const SsmParams& p, long long b, long long run, long long ch0, int left,
                                          int lane, const f2 (&carry)[G::PC][4], const f2 (&sum_d)[G::PC]) {
    const long long row = b * p.runs + run;
    store_lane<G>(p.carry + row * p.channels * G::NP + ch0 * 4, p.channels, left, lane, carry);
    const int c = lane / G::S;
    if (lane % G::S == 0)
#pragma unroll
        for (int j = 0; j < G::CPL; ++j)
            if (G::CPL * c + j < left)
                p.sum_d[row * p.channels + ch0 + G::CPL * c + j] = j & 1 ? hi2(sum_d[j / 2]) : lo2(sum_d[j / 2]);
}

}  // namespace scg
