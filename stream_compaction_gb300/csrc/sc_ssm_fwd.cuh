// Forward selective scan.
//
// Per token, channel and state: one exponential, two products and two
// multiply-adds; per token and channel 4 elements of memory, a softplus and a
// SiLU.  With 16 states a warp's 32 channels take, per token, 64 clocks of its
// SM quarter's exponentials and as many of its multipliers (measured rates: 8
// exponentials, 32 multiply-adds a clock), and another 16 and 12 for the
// softplus and the SiLU.
//
// Two warps share 32 channels (of up to 16 states; 16 of up to 32, 8 of up to
// 64).  The element warp reads x, dt, B and C, makes d = softplus(..) and d * x
// and lays them out in shared memory one tile of kT tokens ahead, and turns the
// sums over states of the tile before into y; the token warp runs the
// recurrence, a lane one channel and 16 of its states.  One barrier a tile.  The
// raw elements are copied asynchronously, several tiles ahead, so that enough
// bytes are under way.
//
// 8 x 4096 tokens, 4096 channels, 16 states, float16: 761 us, where the
// exponentials alone take 230 (and the 1.1 GB 159): an SM's quarter issues in 57 %
// of its clocks, 122 instructions a token and 32 channels (the token warp 78), its
// multipliers work in 43 %, its exponentials in 35 %; the rest is what a token
// needs of the one before, and the barrier between the two warps' work.  Measured
// and slower: one warp for both parts (813), 8 states a lane and two token warps
// (817), 4 states of 4 channels a lane with sums across lanes (791), tiles of 16
// tokens (925: fewer CTAs fit).
//
// Where rows x channels give the machine too few warps the length is split
// into chunks: a first kernel scans each chunk from a zero state (kSummary: no
// C, no y), and the second folds the chunks before its own, h = exp(A * sum of
// d) * h + (their result), and scans its chunk from there.  The exponentials
// are computed twice then, which is why the split waits for idle SMs.
#pragma once
#include "sc_ssm.cuh"

namespace scg {

// 16, or 4, bytes on their way from memory to shared memory.
__device__ __forceinline__ void copy16(void* s, const void* g) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((unsigned)__cvta_generic_to_shared(s)), "l"(g)
                 : "memory");
}
__device__ __forceinline__ void copy4(void* s, const void* g) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"((unsigned)__cvta_generic_to_shared(s)), "l"(g)
                 : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>  // until at most kLeft groups are on their way
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory"); }

// A lane's share: SP states of one channel; S lanes share a channel.
template <int SP_, int S_>
struct FwdGeo {
    static constexpr int SP = SP_, S = S_, P = SP / 2;  // pairs of states
    static constexpr int CH = 32 / S;                   // channels of a warp: lane = s * CH + channel
    static constexpr int NP = SP * S;                   // padded states
    static constexpr int kT = CH == 8 ? 16 : 8;         // tokens that the warps hand over at a time
};

// The forward kernel's shared memory, in bytes.
template <class T, class G, bool kSummary>
struct FwdShared {
    static constexpr int kT = G::kT;
    // tiles of raw elements under way or in use: two behind, the rest ahead
    static constexpr int kRing = sizeof(T) == 4 || G::S == 4 ? 4 : 6;
    static constexpr int kRow = kT * G::CH, kStates = kT * G::NP;
    static constexpr int kRawX = kRow * (int)sizeof(T), kRawB = kStates * (int)sizeof(T);
    static constexpr int x = 0, dt = kRawX, z = 2 * kRawX, B = 3 * kRawX, C = B + kRawB, kRaw = C + kRawB;  // a ring place
    static constexpr int du = kRing * kRaw;                     // [2][kT][CH] of (d, d, d x, d x)
    static constexpr int fB = du + 2 * kRow * 16, fC = fB + 2 * kStates * 4;  // [2][kT][NP]
    static constexpr int y = fC + (kSummary ? 0 : 2 * kStates * 4);           // [2][kT][CH]
    static constexpr int kBytes = y + (kSummary ? 0 : 2 * kRow * 4);
    // Place of a channel's (d, d, d x, d x) in its token's row: neither the four
    // channels that an element lane writes nor the eight that a quarter of the
    // token warp reads meet in a bank.
    __device__ __forceinline__ static int place(int ch) { return ch ^ (ch >> 3); }
};

// Copies of kRows rows of kCols elements, `stride` apart in memory, to a dense
// array in shared memory by one warp, tile after tile; rows from nt on and
// columns from `cols` on get zeros (kFull: there are none).  kVec: row starts
// and cols in 16-byte steps.
template <class T, int kRows, int kCols, bool kVec>
struct RowCopy {
    static constexpr int kPer = kVec ? 16 / (int)sizeof(T) : 1;  // elements of one copy
    static constexpr int kLine = kCols / kPer, kAll = kRows * kLine;
    static_assert(kCols % kPer == 0, "whole copies");
    static_assert(kLine <= 32 ? 32 % kLine == 0 : kLine % 32 == 0, "lanes keep their columns");
    const T* at;
    long long stride;
    __device__ __forceinline__ RowCopy(const T* p, long long token, int lane)
        : at(p + lane / kLine * token + lane % kLine * kPer), stride(token) {}
    template <bool kFull>
    __device__ __forceinline__ void run(T* s, int nt, int cols, int lane) {
        T* to0 = s + lane * kPer;
#pragma unroll
        for (int i = 0; i < (kAll + 31) / 32; ++i) {
            if (kAll % 32 != 0 && lane + 32 * i >= kAll) break;
            const int row = 32 * i / kLine, col = kLine <= 32 ? 0 : 32 * i % kLine * kPer;  // beyond the lane's own
            T* to = to0 + 32 * i * kPer;
            const T* from = at + row * stride + col;
            if (kFull || (lane / kLine + row < nt && lane % kLine * kPer + col < cols)) {
                if constexpr (kVec) copy16(to, from);
                else if constexpr (sizeof(T) == 4) copy4(to, from);
                else *to = __ldg(from);
            } else if constexpr (kVec) {
                *reinterpret_cast<uint4*>(to) = make_uint4(0u, 0u, 0u, 0u);
            } else {
                *to = from_f32<T>(0.0f);
            }
        }
        at += kRows * stride;
    }
};

// Whether any of a warp's values is an infinity or NaN.
template <int kN>
__device__ __forceinline__ bool not_finite(const f2 (&v)[kN][2], const f2 (&w)[kN][2]) {
    f2 zero = 0ull;  // times 0: 0, or NaN
#pragma unroll
    for (int a = 0; a < kN; ++a)
#pragma unroll
        for (int i = 0; i < 2; ++i) zero = fma2(v[a][i], 0ull, fma2(w[a][i], 0ull, zero));
    return __any_sync(0xffffffffu, lo2(zero) + hi2(zero) != 0.0f);
}

// Beside a tile's segment starts (bits 0 .. kT - 1): an infinity or NaN, and padding.
constexpr unsigned kOdd = 1u << 31;

// kPadded: fewer states than the padded number.
template <class T, class G, bool kVec, bool kSummary, bool kPadded>
__global__ void __launch_bounds__(64) ssm_kernel(SsmParams p, int blocks_per_group, int grid_chunks) {
    using Sh = FwdShared<T, G, kSummary>;
    constexpr int kT = Sh::kT, kRing = Sh::kRing;
    using Elems = TileElems<T, G::CH, kT>;
    extern __shared__ __align__(16) unsigned char s_all[];
    __shared__ unsigned s_heads[2], s_flip;
    ulonglong2* s_du = reinterpret_cast<ulonglong2*>(s_all + Sh::du);
    float* s_y = reinterpret_cast<float*>(s_all + Sh::y);
    float *s_B = reinterpret_cast<float*>(s_all + Sh::fB), *s_C = reinterpret_cast<float*>(s_all + Sh::fC);
    const SsmPlace<G, 1> at(p, blocks_per_group, grid_chunks, 0);
    const int lane = threadIdx.x & 31, left = at.left;
    const long long b = at.b;
    const long long t_begin = at.chunk * p.chunk_tiles * kTile;
    const long long t_end = min(t_begin + p.chunk_tiles * kTile, p.length);
    const int n = (int)((t_end - t_begin + kT - 1) / kT);  // tiles
    // An SM gives its warp slots to its four quarters in turn, and a CTA two
    // neighbouring ones: with the roles by the thread index alone every token
    // warp would land on the same two quarters.  Every other pair of slots swaps
    // them (a hint: any outcome is correct, and both warps see warp 0's).
    if (threadIdx.x == 0) {
        unsigned slot;
        asm volatile("mov.u32 %0, %%warpid;" : "=r"(slot));
        s_flip = slot >> 2 & 1u;
    }
    __syncthreads();

    if ((threadIdx.x >> 5) != s_flip) {  // ------------------------------- the element warp
        f2 bias[2], D[2];
        Elems::per_channel(p.dt_bias ? p.dt_bias + at.ch0 : nullptr, left, lane, bias);
        Elems::per_channel(p.D ? p.D + at.ch0 : nullptr, left, lane, D);
        const bool gated = p.z != nullptr && !kSummary;
        const T* xp = static_cast<const T*>(p.x) + b * p.x_batch + t_begin * p.x_token + at.ch0;
        const T* dtp = static_cast<const T*>(p.dt) + b * p.dt_batch + t_begin * p.dt_token + at.ch0;
        const T* zp = gated ? static_cast<const T*>(p.z) + b * p.z_batch + t_begin * p.z_token + at.ch0 : nullptr;
        const T* Bp = static_cast<const T*>(p.B) + b * p.B_batch + t_begin * p.B_token + at.group * p.B_group;
        const T* Cp = static_cast<const T*>(p.C) + b * p.C_batch + t_begin * p.C_token + at.group * p.C_group;
        T* yp = kSummary ? nullptr : static_cast<T*>(p.y) + b * p.y_batch + t_begin * p.y_token + at.ch0;
        const uint8_t* heads = p.heads ? p.heads + b * p.length + t_begin : nullptr;
        const long long tokens = t_end - t_begin;
        bool odd = false;  // the staged tile has a d or d x that is not finite
        auto tile_len = [&](int k) { return (int)min((long long)kT, tokens - (long long)k * kT); };
        auto raw = [&](int k, int what) { return reinterpret_cast<T*>(s_all + (k % kRing) * Sh::kRaw + what); };
        // The copies of one tile, addresses as far as possible made beforehand: a
        // lane's first element of each tensor, moved on by a tile each time.
        const bool whole = left == G::CH;
        RowCopy<T, kT, G::CH, kVec> cx(xp, p.x_token, lane), cdt(dtp, p.dt_token, lane), cz(zp, p.z_token, lane);
        RowCopy<T, kT, G::NP, kVec> cB(Bp, p.B_token, lane), cC(Cp, p.C_token, lane);
        auto fetch = [&](int k) {
            if (k < n) {
                const int nt = tile_len(k);
                if (whole && nt == kT && p.states == G::NP) {
                    cx.template run<true>(raw(k, Sh::x), nt, left, lane);
                    cdt.template run<true>(raw(k, Sh::dt), nt, left, lane);
                    if (gated) cz.template run<true>(raw(k, Sh::z), nt, left, lane);
                    cB.template run<true>(raw(k, Sh::B), nt, G::NP, lane);
                    if constexpr (!kSummary) cC.template run<true>(raw(k, Sh::C), nt, G::NP, lane);
                } else {
                    cx.template run<false>(raw(k, Sh::x), nt, left, lane);
                    cdt.template run<false>(raw(k, Sh::dt), nt, left, lane);
                    if (gated) cz.template run<false>(raw(k, Sh::z), nt, left, lane);
                    cB.template run<false>(raw(k, Sh::B), nt, (int)p.states, lane);
                    if constexpr (!kSummary) cC.template run<false>(raw(k, Sh::C), nt, (int)p.states, lane);
                }
            }
            copies_commit();
        };
        // One step: d and d x of tile k + 1 (kStage), and y of tile k - 1
        // (kFinish), side by side so that the latencies of one hide the other's.
        // Every choice is made outside: a branch among the elements would keep
        // them apart.  kFull: whole tiles of whole channel groups.
        auto step = [&](int k, auto full, auto with_stage, auto with_finish, auto with_softplus, auto with_gate) {
            constexpr bool kFull = decltype(full)::value, kStage = decltype(with_stage)::value;
            constexpr bool kFinish = decltype(with_finish)::value && !kSummary, kGate = decltype(with_gate)::value;
            f2 d[Elems::NA][2], x[Elems::NA][2], y[Elems::NA][2], xe[Elems::NA][2], z[Elems::NA][2];
            const int ks = (k + 1) & 1, nts = kFull || !kStage ? kT : tile_len(k + 1);
            if constexpr (kStage) {
                copies_wait<kRing - 3>();  // tile k + 1 is there: that many groups were committed after its own
                __syncwarp();
#pragma unroll
                for (int a = 0; a < Elems::NA; ++a) {
                    Elems::get(raw(k + 1, Sh::dt) + a * 128, d[a], lane);
                    Elems::get(raw(k + 1, Sh::x) + a * 128, x[a], lane);
                }
            }
            if constexpr (kFinish) {
#pragma unroll
                for (int a = 0; a < Elems::NA; ++a) {
                    Elems::get(s_y + ((k - 1) & 1) * Sh::kRow + a * 128, y[a], lane);
                    Elems::get(raw(k - 1, Sh::x) + a * 128, xe[a], lane);
                    if constexpr (kGate) Elems::get(raw(k - 1, Sh::z) + a * 128, z[a], lane);
                }
            }
            if constexpr (kStage) {
                put_floats<T, Sh::kStates>(s_B + ks * Sh::kStates, raw(k + 1, Sh::B), lane);
                if constexpr (!kSummary) put_floats<T, Sh::kStates>(s_C + ks * Sh::kStates, raw(k + 1, Sh::C), lane);
            }
#pragma unroll
            for (int a = 0; a < Elems::NA; ++a)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    if constexpr (kStage) {
                        d[a][i] = add2(d[a][i], bias[i]);
                        if constexpr (decltype(with_softplus)::value) d[a][i] = softplus_2<T>(d[a][i]);
                        // past the end d = 0, whatever the bias
                        if constexpr (!kFull) d[a][i] = Elems::tok(a, lane) < nts ? d[a][i] : 0ull;
                        x[a][i] = mul2(d[a][i], x[a][i]);
                    }
                    if constexpr (kFinish) {
                        y[a][i] = fma2(D[i], xe[a][i], y[a][i]);
                        if constexpr (kGate) y[a][i] = mul2(y[a][i], mul2(z[a][i], sigmoid_2<T>(z[a][i])));
                    }
                }
            if constexpr (kStage) {
                if constexpr (kPadded) odd = not_finite(d, x);
                ulonglong2* out = s_du + ks * Sh::kRow;
#pragma unroll
                for (int a = 0; a < Elems::NA; ++a)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float dv = i & 1 ? hi2(d[a][i / 2]) : lo2(d[a][i / 2]);
                        const float uv = i & 1 ? hi2(x[a][i / 2]) : lo2(x[a][i / 2]);
                        out[Elems::tok(a, lane) * G::CH + Sh::place(Elems::ch(lane) + i)] =
                            make_ulonglong2(both(dv), both(uv));
                    }
            }
            if constexpr (kFinish) {
                const int nt = kFull ? kT : tile_len(k - 1);
#pragma unroll
                for (int a = 0; a < Elems::NA; ++a)
                    Elems::template store<kVec, kFull>(yp, p.y_token, y[a], a, nt, left, lane);
                yp += kT * p.y_token;
            }
        };
        using Yes = std::true_type;
        using No = std::false_type;
        auto any_step = [&](int k, auto full, auto with_stage, auto with_finish) {
            if (p.softplus) {
                if (gated) step(k, full, with_stage, with_finish, Yes{}, Yes{});
                else step(k, full, with_stage, with_finish, Yes{}, No{});
            } else {
                if (gated) step(k, full, with_stage, with_finish, No{}, Yes{});
                else step(k, full, with_stage, with_finish, No{}, No{});
            }
        };
        auto put_heads = [&](int k, bool head) {
            const unsigned mask = __ballot_sync(0xffffffffu, head);
            if (lane == 0) s_heads[k & 1] = kPadded && odd ? mask | kOdd : mask;
        };
        auto head_at = [&](int k) {
            const long long t = (long long)k * kT + lane;
            return heads && lane < kT && t < tokens && heads[t] != 0;
        };
#pragma unroll
        for (int k = 0; k < kRing - 2; ++k) fetch(k);
        any_step(-1, No{}, Yes{}, No{});  // stages tile 0
        put_heads(0, head_at(0));
        __syncthreads();
        for (int k = 0; k < n; ++k) {  // the token warp is at tile k
            const bool head = head_at(k + 1);
            fetch(k + kRing - 2);      // to the place of tile k - 2, which is finished
            if (k > 0 && k + 1 < n) {
                if (p.softplus && whole && (long long)(k + 2) * kT <= tokens) {
                    if (gated) step(k, Yes{}, Yes{}, Yes{}, Yes{}, Yes{});
                    else step(k, Yes{}, Yes{}, Yes{}, Yes{}, No{});
                } else {
                    any_step(k, No{}, Yes{}, Yes{});
                }
            } else {
                if (k + 1 < n) any_step(k, No{}, Yes{}, No{});
                if (k > 0) any_step(k, No{}, No{}, Yes{});
            }
            put_heads(k + 1, head);
            __syncthreads();
        }
        any_step(n, No{}, No{}, Yes{});
        return;
    }

    // -------------------------------------------------------------- the token warp
    const int s = lane / G::CH, c = lane % G::CH;
    const bool mine = c < left;
    const long long e = at.ch0 + c;
    f2 A2[G::P], h[G::P];
    float dsum = 0.0f;
#pragma unroll
    for (int i = 0; i < G::P; ++i) {
        const int n0 = s * G::SP + 2 * i;
        const float* Ap = p.A + e * p.states + n0;
        const float* hp = p.state ? p.state + (b * p.channels + e) * p.states + n0 : nullptr;
        const bool in0 = mine && n0 < p.states, in1 = mine && n0 + 1 < p.states;
        A2[i] = pack2(in0 ? rate(Ap[0]) : 0.0f, in1 ? rate(Ap[1]) : 0.0f);
        h[i] = kSummary || !hp ? 0ull : pack2(in0 ? hp[0] : 0.0f, in1 ? hp[1] : 0.0f);
    }
    // states of this lane in the library's own arrays: [fours of states][channels][4]
    auto own = [&](float* base, long long row) {
        return reinterpret_cast<ulonglong2*>(base) + (row * (G::NP / 4) + s * (G::SP / 4)) * p.channels + e;
    };
    // States past `states` have A = B = C = 0 and stay 0 by themselves while d and d x
    // are finite.  An infinity times their zeros would be NaN, and reach y: where a tile
    // has one they are set to 0, token by token.
    auto drop_padding = [&]() {
        const int real = (int)p.states - lane_anew() / G::CH * G::SP;  // the lane's states before the padding
#pragma unroll
        for (int i = 0; i < G::P; ++i) h[i] = pack2(2 * i < real ? lo2(h[i]) : 0.0f, 2 * i + 1 < real ? hi2(h[i]) : 0.0f);
    };
    if constexpr (!kSummary) {
        for (long long j = 0; j < at.chunk; ++j) {  // the chunks before this one
            const long long row = b * p.chunks + j;
            const ulonglong2* cp = own(p.carry, row);
            const f2 d = both(mine ? p.sum_d[row * p.channels + e] : 0.0f);
            const bool cut = p.cut[row] != 0;
#pragma unroll
            for (int i = 0; i < G::P / 2; ++i) {
                const ulonglong2 v = mine ? cp[i * p.channels] : make_ulonglong2(0ull, 0ull);
                h[2 * i] = cut ? v.x : fma2(ex2_2(mul2(d, A2[2 * i])), h[2 * i], v.x);
                h[2 * i + 1] = cut ? v.y : fma2(ex2_2(mul2(d, A2[2 * i + 1])), h[2 * i + 1], v.y);
            }
            if constexpr (kPadded) drop_padding();
        }
    }
    const long long saves = (p.length + kTile - 1) / kTile;
    unsigned cut = 0;
    __syncthreads();
    for (int k = 0; k < n; ++k) {
        const ulonglong2* ldu = s_du + (k & 1) * Sh::kRow + Sh::place(c);
        const ulonglong2* lB = reinterpret_cast<const ulonglong2*>(s_B + (k & 1) * Sh::kStates + s * G::SP);
        const ulonglong2* lC = reinterpret_cast<const ulonglong2*>(s_C + (k & 1) * Sh::kStates + s * G::SP);
        float* ly = s_y + (k & 1) * Sh::kRow + c;
        const unsigned hm = s_heads[k & 1];
        cut |= hm & ~kOdd;
        if (!kSummary && p.saved && k % (kTile / kT) == 0 && mine) {
            ulonglong2* sp = own(p.saved, b * saves + at.chunk * p.chunk_tiles + k / (kTile / kT));
#pragma unroll
            for (int i = 0; i < G::P / 2; ++i) sp[i * p.channels] = make_ulonglong2(h[2 * i], h[2 * i + 1]);
        }
        // One token ahead: the decays and inputs of token t + 1 are on their way
        // while token t is applied, so that neither the exponentials nor the
        // multipliers wait for the other.
        auto tokens = [&](auto with_care) {  // segment starts, or states to be kept at 0
            f2 a[G::P], ub[G::P];
            auto ahead = [&](int t) {
                const ulonglong2 du = ldu[t * G::CH];
#pragma unroll
                for (int i = 0; i < G::P / 2; ++i) {
                    const ulonglong2 Bv = lB[t * (G::NP / 4) + i];
                    a[2 * i] = decay_2(du.x, A2[2 * i]);
                    a[2 * i + 1] = decay_2(du.x, A2[2 * i + 1]);
                    ub[2 * i] = mul2(du.y, Bv.x);
                    ub[2 * i + 1] = mul2(du.y, Bv.y);
                }
                if constexpr (kSummary) dsum += lo2(du.x);
            };
            ahead(0);
#pragma unroll
            for (int t = 0; t < kT; ++t) {
                f2 now[G::P], in[G::P];
#pragma unroll
                for (int i = 0; i < G::P; ++i) {
                    now[i] = a[i];
                    in[i] = ub[i];
                }
                if (t + 1 < kT) ahead(t + 1);
                if (decltype(with_care)::value && (hm >> t & 1u)) {
#pragma unroll
                    for (int i = 0; i < G::P; ++i) h[i] = 0ull;
                }
#pragma unroll
                for (int i = 0; i < G::P; ++i) h[i] = fma2(now[i], h[i], in[i]);
                if (decltype(with_care)::value && kPadded && hm >= kOdd) drop_padding();
                if constexpr (!kSummary) {
                    f2 y0 = 0ull, y1 = 0ull;
#pragma unroll
                    for (int i = 0; i < G::P / 2; ++i) {
                        const ulonglong2 Cv = lC[t * (G::NP / 4) + i];
                        y0 = i ? fma2(Cv.x, h[2 * i], y0) : mul2(Cv.x, h[2 * i]);
                        y1 = i ? fma2(Cv.y, h[2 * i + 1], y1) : mul2(Cv.y, h[2 * i + 1]);
                    }
                    y0 = add2(y0, y1);
                    float y = lo2(y0) + hi2(y0);
#pragma unroll
                    for (int m = G::CH; m < 32; m <<= 1) y += __shfl_xor_sync(0xffffffffu, y, m);
                    if (G::S == 1 || s == 0) ly[t * G::CH] = y;
                }
            }
        };
        if (hm) tokens(std::true_type{});
        else tokens(std::false_type{});
        __syncthreads();
    }
    if constexpr (kSummary) {
        const long long row = b * p.chunks + at.chunk;
        if (mine) {
            ulonglong2* cp = own(p.carry, row);
#pragma unroll
            for (int i = 0; i < G::P / 2; ++i) cp[i * p.channels] = make_ulonglong2(h[2 * i], h[2 * i + 1]);
            if (s == 0) p.sum_d[row * p.channels + e] = dsum;
        }
        if (at.cblock == 0 && lane == 0) p.cut[row] = cut != 0;
    } else if (p.final_state && t_end == p.length && mine) {
        float* fp = p.final_state + (b * p.channels + e) * p.states + s * G::SP;
#pragma unroll
        for (int i = 0; i < G::SP; ++i)
            if (s * G::SP + i < p.states) fp[i] = i & 1 ? hi2(h[i / 2]) : lo2(h[i / 2]);
    }
}

template <class T, class G, bool kVec>
cudaError_t ssm_of(const SsmParams& p, const SsmPlan& plan, int* launches, cudaStream_t s) {
    const long long per = p.channels / p.groups;
    const int bpg = (int)((per + G::CH - 1) / G::CH);
    const long long ncb = bpg * p.groups;
    *launches = 1;
    auto go = [&](auto kernel, int bytes, int chunks) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e == cudaSuccess) kernel<<<(unsigned)(ncb * chunks * p.batch), 64, bytes, s>>>(p, bpg, chunks);
        return e;
    };
    const bool padded = p.states != G::NP;
    if (p.chunks > 1) {  // nobody waits for the last chunk's summary
        const int bytes = FwdShared<T, G, true>::kBytes;
        const cudaError_t e = padded ? go(ssm_kernel<T, G, kVec, true, true>, bytes, p.chunks - 1)
                                     : go(ssm_kernel<T, G, kVec, true, false>, bytes, p.chunks - 1);
        if (e != cudaSuccess) return e;
        *launches = 2;
    }
    const int bytes = FwdShared<T, G, false>::kBytes;
    const cudaError_t e = padded ? go(ssm_kernel<T, G, kVec, false, true>, bytes, p.chunks)
                                 : go(ssm_kernel<T, G, kVec, false, false>, bytes, p.chunks);
    if (e != cudaSuccess) return e;
    return cudaGetLastError();
}

template <class T>
cudaError_t ssm_type(const SsmParams& p, const SsmPlan& plan, int* launches, cudaStream_t s) {
    auto go = [&](auto g) {
        using G = decltype(g);
        return p.vec ? ssm_of<T, G, true>(p, plan, launches, s) : ssm_of<T, G, false>(p, plan, launches, s);
    };
    switch (plan.lanes) {
    case 2: return go(FwdGeo<8, 1>{});
    case 4: return go(FwdGeo<16, 1>{});
    case 8: return go(FwdGeo<16, 2>{});
    case 16: return go(FwdGeo<16, 4>{});
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace scg
