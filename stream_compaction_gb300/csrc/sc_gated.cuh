// The gated recurrence h[t] = f[t] h[t-1] + b[t], f = sigmoid(gate), b = (1 - f) x
// (or f = gate, b = x), its gradient and its form for one token: kernels, by element
// type in sc_gated_*.cu.
//
//   dh[t] = dy[t] + f[t+1] dh[t+1];  dx = dh (1 - f);  dgate = dh (h[t-1] - x) f (1 - f)
//
// Three elements moved forward and five backward for some ten operations each: bytes
// bound it, if the length is split.  A warp takes a tile of kTokens tokens by 32 or 64
// channels, a lane's channels side by side with all their tokens, so the recurrence
// needs no exchange inside a tile.  The warps of a CTA take consecutive tiles of the same
// channels, and the CTAs of a cluster consecutive runs of them; a round of kWarps x
// cluster tiles goes like a scan:
//
//   each warp   its tile's map h -> A h + B (A the product of f, B the recurrence from 0);
//   the CTA     the maps meet in shared memory; the CTA's own map goes to every CTA of
//               the cluster (distributed shared memory, writes that are counted there);
//   each warp   the state before its tile: the carry, through the maps before it in order;
//               then the recurrence again, on registers, and the results.
//
// So every element is read once and written once, no scratch memory is needed, and the
// order of all roundings is fixed.  Tiles come and results go by the copy engine, one
// instruction each, one or two rounds ahead in shared memory; rows that are not aligned
// to 16 bytes are loaded a round ahead into registers.
//
// The gradient runs the same rounds backwards on q[t] = f[t] dh[t], with the states
// recomputed from those that the forward pass saved (one in kTokens: 1/16 of an
// element's place in float32, where keeping h itself would cost an element read and
// rounding errors of 16 bits in dgate).
//
// 8 x 4096 tokens of 4096 bfloat16: forward 141 to 145 us (5.6 to 5.7 TB/s, a copy 6.5), 147
// to 151 with the states saved, gradient 246 to 250 (5.4 to 5.5); rows that are not aligned
// 2.4 to 4.6 TB/s.
#pragma once
#include <algorithm>

#include <cooperative_groups.h>

#include "sc_bulk.cuh"
#include "sc_cluster.h"
#include "sc_seq.cuh"
#include "sc_seq_launch.h"
#include "sc_tensor_map.h"

namespace scg {

namespace {

namespace cg = cooperative_groups;

constexpr int kTokens = SC_GATED_SAVE;
constexpr int kMaxCluster = 16;  // beyond 8 a launch has to ask for it

// Tensor maps of a call: forward x, gate and y; backward x, gate, dy, dx and dgate.
struct GatedMaps {
    CUtensorMap map[5];
};
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int c, int t, int b, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(c), "r"(t), "r"(b), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, int c, int t, int b, uint32_t src) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];"
                 ::"l"(reinterpret_cast<uint64_t>(map)), "r"(c), "r"(t), "r"(b), "r"(src)
                 : "memory");
}

// A lane's K channels of a token: as they lie in memory, and as one operand.
template <class T, int K> struct Raw { using type = unsigned short; };
template <> struct Raw<float, 1> { using type = float; };
template <> struct Raw<f16, 2> { using type = uint32_t; };
template <> struct Raw<bf16, 2> { using type = uint32_t; };

template <int K> struct Lane;
template <> struct Lane<1> {
    using V = float;
    static __device__ __forceinline__ V all(float v) { return v; }
    static __device__ __forceinline__ V mul(V a, V b) { return a * b; }
    static __device__ __forceinline__ V add(V a, V b) { return a + b; }
    static __device__ __forceinline__ V fma(V a, V b, V c) { return fmaf(a, b, c); }
    static __device__ __forceinline__ V load(const float* p) { return __ldg(p); }
    static __device__ __forceinline__ void store(float* p, V v) { *p = v; }
    static __device__ __forceinline__ bool nan(V v) { return v != v; }
    // `a` where `by` is NaN, else b
    static __device__ __forceinline__ V pick(V by, V a, V b) { return nan(by) ? a : b; }
};
template <> struct Lane<2> {
    using V = f2;
    static __device__ __forceinline__ V all(float v) { return both(v); }
    static __device__ __forceinline__ V mul(V a, V b) { return mul2(a, b); }
    static __device__ __forceinline__ V add(V a, V b) { return add2(a, b); }
    static __device__ __forceinline__ V fma(V a, V b, V c) { return fma2(a, b, c); }
    static __device__ __forceinline__ V load(const float* p) { return pack2(__ldg(p), __ldg(p + 1)); }
    static __device__ __forceinline__ void store(float* p, V v) {
        p[0] = lo2(v);
        p[1] = hi2(v);
    }
    static __device__ __forceinline__ bool nan(V v) { return lo2(v) != lo2(v) || hi2(v) != hi2(v); }
    static __device__ __forceinline__ V pick(V by, V a, V b) {
        return pack2(Lane<1>::pick(lo2(by), lo2(a), lo2(b)), Lane<1>::pick(hi2(by), hi2(a), hi2(b)));
    }
};

// A lane's tile: kTokens tokens of K channels in pairs, for two-lane arithmetic: a
// token's two channels, or two tokens of one channel.
template <int K> constexpr int kPairs = kTokens * K / 2;
template <int K>
__device__ __forceinline__ typename Lane<K>::V token(const f2 (&v)[kPairs<K>], int j) {
    if constexpr (K == 2) return v[j];
    else return j % 2 ? hi2(v[j / 2]) : lo2(v[j / 2]);
}
template <int K>
__device__ __forceinline__ void set_token(f2 (&v)[kPairs<K>], int j, typename Lane<K>::V t) {
    if constexpr (K == 2) v[j] = t;
    else v[j / 2] = j % 2 ? pack2(lo2(v[j / 2]), t) : pack2(t, hi2(v[j / 2]));
}

// Token j's part of the pair that it is in.
template <int K>
__device__ __forceinline__ typename Lane<K>::V half(f2 v, int j) {
    if constexpr (K == 2) return v;
    else return j % 2 ? hi2(v) : lo2(v);
}

// A lane's elements as they lie in memory, as an operand.
template <class T, class R>
__device__ __forceinline__ float one_of(R v) {
    if constexpr (sizeof(T) == 4) {
        return v;
    } else {
        T e;
        memcpy(&e, &v, 2);
        return to_f32(e);
    }
}
template <class T, int K>
struct Elements {
    using R = typename Raw<T, K>::type;
    using V = typename Lane<K>::V;
    static __device__ __forceinline__ V of(R v) {
        if constexpr (K == 2) {
            Vec<T, 2> e;
            e.w[0] = v;
            return e.pair(0);
        } else {
            return one_of<T>(v);
        }
    }
    static __device__ __forceinline__ f2 pair(R a, R b) { return pack2(one_of<T>(a), one_of<T>(b)); }
    static __device__ __forceinline__ void store(T* p, V v) {
        if constexpr (K == 2) {
            const float f[2] = {lo2(v), hi2(v)};
            Vec<T, 2> o;
            o.set(f);
            o.store(p);
        } else {
            *p = from_f32<T>(v);
        }
    }
};

// A warp's tile of one tensor in shared memory, 32 K channels a token: rounds ahead of
// its use without a register, where loads into registers had a third of that under way
// (8 x 4096 tokens of 4096 channels: 160 us, 141 so).
template <class T, int K>
struct Tile : Elements<T, K> {
    using E = Elements<T, K>;
    using R = typename E::R;
    static constexpr int kBytes = kTokens * 32 * (int)sizeof(R);
    R* at;  // the lane's channels of the first token
    __device__ __forceinline__ Tile(unsigned char* tile, int lane) : at(reinterpret_cast<R*>(tile) + lane) {}
    __device__ __forceinline__ f2 pair(int i) const {
        if constexpr (K == 2) return E::of(at[i * 32]);
        else return E::pair(at[2 * i * 32], at[(2 * i + 1) * 32]);
    }
    __device__ __forceinline__ typename E::V get(int j) const { return E::of(at[j * 32]); }
    // The result of token j in place of what was read there.
    __device__ __forceinline__ void put(int j, typename E::V v) const { E::store(reinterpret_cast<T*>(at + j * 32), v); }
};

// A warp's tile in registers, where rows are not aligned to 16 bytes; the next one is
// loaded when this one has been used.
template <class T, int K>
struct Held : Elements<T, K> {
    using E = Elements<T, K>;
    using R = typename E::R;
    R r[kTokens];
    const T* p;         // the lane's channels of the next tile's first token
    long long stride;   // of a token
    long long advance;  // from a tile to the warp's next
    __device__ __forceinline__ Held(const void* base, long long row, long long token, int tile, int step, long long ch)
        : p(static_cast<const T*>(base) + row + (long long)tile * kTokens * token + ch), stride(token),
          advance((long long)step * kTokens * token) {}
    // The next tile, of which the row has `left` tokens (zeros for the others).
    __device__ __forceinline__ void next(int left, bool live) {
        if (left >= kTokens && live) {
#pragma unroll
            for (int j = 0; j < kTokens; ++j) r[j] = __ldg(reinterpret_cast<const R*>(p + j * stride));
        } else {
#pragma unroll
            for (int j = 0; j < kTokens; ++j)
                r[j] = live && j < left ? __ldg(reinterpret_cast<const R*>(p + j * stride)) : R(0);
        }
        p += advance;
    }
    __device__ __forceinline__ f2 pair(int i) const {
        if constexpr (K == 2) return E::of(r[i]);
        else return E::pair(r[2 * i], r[2 * i + 1]);
    }
    __device__ __forceinline__ typename E::V get(int j) const { return E::of(r[j]); }
    __device__ __forceinline__ void put(int, typename E::V) const {}
};

// The smaller of f and 1 - f, e / (1 + e) with e = exp(-|g|), and the larger, for a pair.
// The smaller one has its relative error ((4 + |g|) 2^-24 in 16 bits, 9 x 2^-24 in
// float32; 0 where e is below 2^-126) however small it is: so has a closed gate's f, which
// dgate is proportional to, and an open gate's 1 - f, which x enters with.  The larger is
// off by as much absolutely, times the smaller: decays close to 1 are as good as rounded
// ones, however many are multiplied.  (f = 1 - e / (1 + e) with e = exp(-g) for all gates
// saves a selection, but keeps one or two digits of a gate of -12, none of one below -17.)
template <class T>
__device__ __forceinline__ void gate_parts(f2 g, f2& small, f2& large) {
    f2 e;
    if constexpr (kFine<T>) e = exp_minus_2<true>(g & 0x7fffffff7fffffffull);
    else e = pack2(ex2(fabsf(lo2(g)) * -kLog2e), ex2(fabsf(hi2(g)) * -kLog2e));
    small = mul2(e, rcp_2(add2(e, both(1.0f))));
    large = fma2(small, both(-1.0f), both(1.0f));
}
// By a gate's sign bit.
__device__ __forceinline__ bool closed(float g) { return __float_as_int(g) < 0; }
__device__ __forceinline__ f2 select2(f2 by, f2 shut, f2 open) {
    return pack2(closed(lo2(by)) ? lo2(shut) : lo2(open), closed(hi2(by)) ? hi2(shut) : hi2(open));
}
// f and 1 - f.
template <class T>
__device__ __forceinline__ void gates(f2 g, f2& f, f2& rest) {
    f2 small, large;
    gate_parts<T>(g, small, large);
    f = select2(g, small, large);
    rest = select2(g, large, small);
}
// f dh and (1 - f) dh from the smaller of f and 1 - f with the gate's sign.
__device__ __forceinline__ void shares(float part, float dh, float& f, float& rest) {
    const float a = fabsf(part), less = a * dh, more = fmaf(-a, dh, dh);
    f = closed(part) ? less : more;
    rest = closed(part) ? more : less;
}
__device__ __forceinline__ void shares(f2 part, f2 dh, f2& f, f2& rest) {
    float v[2][2];
    shares(lo2(part), lo2(dh), v[0][0], v[1][0]);
    shares(hi2(part), hi2(dh), v[0][1], v[1][1]);
    f = pack2(v[0][0], v[0][1]);
    rest = pack2(v[1][0], v[1][1]);
}

// A lane's flag of a tile's tokens, and the tokens where a segment starts, one bit each.
__device__ __forceinline__ uint8_t head_of(const uint8_t* heads, long long row, long long t0, long long length, int lane) {
    const long long t = t0 + lane;
    return lane < kTokens && t >= 0 && t < length ? __ldg(heads + row * length + t) : 0;
}
// (A tile that did not come is NaN from one end to the other, whatever starts in it.)
template <bool kTma>
__device__ __forceinline__ uint32_t cuts_of(uint8_t head, bool ok) {
    const uint32_t cuts = __ballot_sync(0xffffffffu, head != 0);
    return !kTma || __all_sync(0xffffffffu, ok) ? cuts : 0u;
}

// The map of a run of tokens on the value before it: h -> A h + B, or B alone where a
// segment starts inside (whatever h is, infinities too).
template <int K>
struct Map {
    typename Lane<K>::V A, B;
    __device__ __forceinline__ typename Lane<K>::V of(typename Lane<K>::V h) const { return Lane<K>::fma(A, h, B); }
    __device__ __forceinline__ typename Lane<K>::V of(typename Lane<K>::V h, bool cut) const { return cut ? B : of(h); }
};

// What the warps and CTAs of a round exchange.
template <int K, int kWarps>
struct Exchange {
    uint64_t bar[2];  // the other CTAs' maps have arrived
    int cut[2][kWarps], rank_cut[2][kMaxCluster];
    Map<K> warp[2][kWarps][32];
    Map<K> rank[1][32];  // [2][CTAs] of them; a CTA by itself needs none
    static __host__ __device__ constexpr size_t bytes(int ctas) {
        return sizeof(Exchange) + (ctas > 1 ? (2 * ctas - 1) * sizeof(Map<K>[32]) : 0);
    }
};

// Remote writes that are counted on a barrier of the CTA that they go to, so nothing has
// to be waited for but the data themselves (a cluster barrier's release waits for all
// that the CTA has written, results too: 8192 tokens of 2048 channels 41 us).
__device__ __forceinline__ uint32_t at_rank(uint32_t address, int rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(address), "r"(rank));
    return r;
}
__device__ __forceinline__ void send(uint32_t to, uint32_t bar, const Map<1>& m) {
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.b32 [%0], {%1, %2}, [%3];"
                 ::"r"(to), "r"(__float_as_uint(m.A)), "r"(__float_as_uint(m.B)), "r"(bar) : "memory");
}
__device__ __forceinline__ void send(uint32_t to, uint32_t bar, const Map<2>& m) {
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.b64 [%0], {%1, %2}, [%3];"
                 ::"r"(to), "l"(m.A), "l"(m.B), "r"(bar) : "memory");
}
__device__ __forceinline__ void send(uint32_t to, uint32_t bar, int v) {
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];"
                 ::"r"(to), "r"(v), "r"(bar) : "memory");
}
__device__ __forceinline__ bool arrived_from_cluster(uint32_t bar, uint32_t parity) {
    for (int i = 0; i < (1 << 20); ++i) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, 1000;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
        if (ok) return true;
    }
    return false;
}

// The round's tiles one by one, from `value` before it, for the channels where `odd` is NaN.
template <int K, int kWarps, class Walk>
__device__ __forceinline__ void one_by_one(Exchange<K, kWarps>& x, int turn, int warp, int lane, int rank, int ranks,
                                           typename Lane<K>::V odd, typename Lane<K>::V value, typename Lane<K>::V& in,
                                           typename Lane<K>::V& carry, Walk walk) {
    const cg::cluster_group cluster = cg::this_cluster();
    if (ranks > 1) cluster.sync();  // the maps are read
    else __syncthreads();
    for (int r = 0; r < ranks; ++r) {
        if (r == rank) {
            for (int w = 0; w < kWarps; ++w) {
                if (w == warp) {
                    in = Lane<K>::pick(odd, value, in);
                    x.warp[turn][w][lane].B = walk(value);
                }
                __syncthreads();
                value = x.warp[turn][w][lane].B;
            }
            if (ranks > 1 && warp == 0)
                for (int to = 0; to < ranks; ++to) *cluster.map_shared_rank(&x.rank[turn * ranks + r][lane].B, to) = value;
        }
        if (ranks > 1) {
            cluster.sync();
            value = x.rank[turn * ranks + r][lane].B;
        }
    }
    carry = Lane<K>::pick(odd, value, carry);
}

// One round: takes this warp's map, returns the value before its tile and moves
// `carry`, the value before the round, to behind it (the same in all warps).  Warps and
// CTAs count in the direction of the recurrence.  Buffers alternate: a warp writes for
// the next round while others still read this one's, and two rounds on a barrier lies
// between (in a cluster: a CTA sends for a round when all its warps are through with
// the one before, and gets no further until every other has).
// kCuts: segments may start anywhere.  kAny: decays of any size; where the product of some
// passes float32's range (or is NaN), its channel goes through the round's tiles one by one
// (walk: a value through this warp's), since infinity times a state of 0 is not 0.
template <int K, int kWarps, bool kCuts, bool kAny, class Walk>
__device__ __forceinline__ typename Lane<K>::V exchange(Exchange<K, kWarps>& x, int round, int warp, int lane, int rank,
                                                        int ranks, const Map<K>& map, bool cut,
                                                        typename Lane<K>::V& carry, Walk walk) {
    using V = typename Lane<K>::V;
    // odd: 0, or NaN where a product is not finite
    [[maybe_unused]] V before_all = carry, odd = Lane<K>::all(0.0f);
    const int turn = round & 1;
    x.warp[turn][warp][lane] = map;
    if (kCuts && lane == 0) x.cut[turn][warp] = cut;
    __syncthreads();
    V in = carry;
    if (ranks == 1) {
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const Map<K> m = x.warp[turn][w][lane];
            const bool c = kCuts && x.cut[turn][w] != 0;
            if (w < warp) in = m.of(in, c);
            carry = m.of(carry, c);
            if (kAny) odd = Lane<K>::fma(m.A, Lane<K>::all(0.0f), odd);
        }
        if (kAny && __any_sync(0xffffffffu, Lane<K>::nan(odd)))
            one_by_one(x, turn, warp, lane, rank, ranks, odd, before_all, in, carry, walk);
        return in;
    }
    // the maps of the warps before this one, and of the CTA
    Map<K> before{Lane<K>::all(1.0f), Lane<K>::all(0.0f)}, all = before;
    bool before_cut = false, all_cut = false;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w == warp) {
            before = all;
            before_cut = all_cut;
        }
        const Map<K> m = x.warp[turn][w][lane];
        const bool c = kCuts && x.cut[turn][w] != 0;
        all.B = m.of(all.B, c);
        all.A = Lane<K>::mul(m.A, all.A);
        all_cut |= c;
    }
    const uint32_t bar = smem_u32(&x.bar[turn]), to = smem_u32(&x.rank[turn * ranks + rank][lane]);
    if (threadIdx.x == 0) mbar_arrive_expect_tx(bar, (uint32_t)ranks * (32 * sizeof(Map<K>) + (kCuts ? 4 : 0)));
    for (int r = warp; r < ranks; r += kWarps) {
        send(at_rank(to, r), at_rank(bar, r), all);
        if (kCuts && lane == 0) send(at_rank(smem_u32(&x.rank_cut[turn][rank]), r), at_rank(bar, r), (int)all_cut);
    }
    const bool here = arrived_from_cluster(bar, (uint32_t)(round >> 1) & 1u);
    if (!here) carry = Lane<K>::all(not_a_number());
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r) {
        if (r >= ranks) break;
        if (r == rank) in = carry;
        carry = x.rank[turn * ranks + r][lane].of(carry, kCuts && here && x.rank_cut[turn][r] != 0);
        if (kAny) odd = Lane<K>::fma(x.rank[turn * ranks + r][lane].A, Lane<K>::all(0.0f), odd);
    }
    in = before.of(in, kCuts && before_cut);
    // (a wait that ran out: the CTAs may not have seen the same maps, and must not wait for one another)
    if (kAny && here && __any_sync(0xffffffffu, Lane<K>::nan(odd)))
        one_by_one(x, turn, warp, lane, rank, ranks, odd, before_all, in, carry, walk);
    return in;
}
// Before the first round: every CTA's barriers stand before another writes to it.
template <class E>
__device__ __forceinline__ void exchange_begin(E& x, int ranks) {
    if (ranks == 1) return;
    if (threadIdx.x == 0) {
        mbar_init(smem_u32(&x.bar[0]), 1);
        mbar_init(smem_u32(&x.bar[1]), 1);
        fence_mbar_init();
    }
    cg::this_cluster().sync();
}
// After the last: no CTA leaves while another writes to its shared memory.
__device__ __forceinline__ void exchange_end(int ranks) {
    if (ranks > 1) cg::this_cluster().sync();
}

// Where a CTA works: row b, the lane's first channel, the rounds.
struct Place {
    long long b, ch0, ch;  // ch0: the warp's first channel, ch: the lane's
    int rounds, tiles, rank, ranks, warp, lane;
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
    c.ch0 = (group - c.b * blocks) * 32 * K;
    c.ch = c.ch0 + c.lane * K;
    c.live = c.ch < p.channels;
    c.tiles = (int)((p.length + kTokens - 1) / kTokens);
    c.rounds = (c.tiles + c.ranks * kWarps - 1) / (c.ranks * kWarps);
    return c;
}

// A warp's ring of rounds, kTensors tiles each: whole tiles by the copy engine, one
// instruction of one lane, and results back the same way from where the elements lay.
template <class T, int K, int kTensors, int kStages>
struct Ring {
    using Tl = Tile<T, K>;
    static constexpr int kRound = kTensors * Tl::kBytes, kBytes = kStages * kRound;
    unsigned char *base, *fill, *take;
    uint32_t bar, phase = 0;  // the stages' barriers, the parity of the round to take
    __device__ __forceinline__ Ring(unsigned char* mem, uint64_t* bars, int lane)
        : base(mem), fill(mem), take(mem), bar(smem_u32(bars)) {
        if (bars && lane == 0) {
#pragma unroll
            for (int i = 0; i < kStages; ++i) mbar_init(bar + 8 * i, 1);
            fence_mbar_init();
        }
        __syncwarp();
    }
    __device__ __forceinline__ void next(unsigned char*& at) {
        at += kRound;
        if (at == base + kBytes) at = base;
    }
    // The tiles of the tokens from t0 of row b, by one lane; what the stage held has been
    // read, by the copies of results out of it, too.
    __device__ __forceinline__ void load(const GatedMaps& m, int ch0, int t0, int b) {
        bulk_wait_read_all();
        const uint32_t full = bar + (uint32_t)(fill - base) / kRound * 8, to = smem_u32(fill);
        mbar_arrive_expect_tx(full, kRound);
#pragma unroll
        for (int i = 0; i < kTensors; ++i) tma_load_3d(to + i * Tl::kBytes, &m.map[i], ch0, t0, b, full);
    }
    __device__ __forceinline__ bool wait() {
        const uint32_t full = bar + (uint32_t)(take - base) / kRound * 8;
        const bool ok = arrived(full, phase);
        if (take + kRound == base + kBytes) phase ^= 1;
        return ok;
    }
    __device__ __forceinline__ Tl tile(int i, int lane) const { return Tl(take + i * Tl::kBytes, lane); }
};
// Rows that are not aligned have no ring.
template <int K, int kWarps, class Ring, bool kTma> struct Shared {
    unsigned char ring[kTma ? kWarps : 1][kTma ? Ring::kBytes : 16];  // first: the copy engine wants 128 bytes' alignment
    uint64_t bars[kWarps][4];
    Exchange<K, kWarps> ex;  // last: its size goes by the cluster
    static __host__ __device__ constexpr size_t bytes(int ctas) {
        return sizeof(Shared) - sizeof(Exchange<K, kWarps>) + Exchange<K, kWarps>::bytes(ctas);
    }
};

// The tensor's tile of this round: in the ring, or as it was loaded.
template <bool kTma, class Ring, class Held>
__device__ __forceinline__ auto tile_of(const Ring& ring, const Held& held, int i, int lane) {
    if constexpr (kTma) return ring.tile(i, lane);
    else return held;
}

// ---------------------------------------------------------------- forward
template <class T, int K> using ForwardRing = Ring<T, K, 2, 3>;

template <class T, int K, bool kTma, bool kSigmoid, int kWarps, bool kCuts>
__global__ void __launch_bounds__(32 * kWarps, 16 / kWarps)
    gated_kernel(GatedParams p, const __grid_constant__ GatedMaps maps) {
    using L = Lane<K>;
    using V = typename L::V;
    using Sh = Shared<K, kWarps, ForwardRing<T, K>, kTma>;
    extern __shared__ __align__(128) unsigned char s_mem[];
    Sh& s = *reinterpret_cast<Sh*>(s_mem);
    const Place c = place_of<K, kWarps>(p);
    const int step = c.ranks * kWarps;
    int tile = c.rank * kWarps + c.warp;
    ForwardRing<T, K> ring(s.ring[kTma ? c.warp : 0], kTma ? s.bars[c.warp] : nullptr, c.lane);
    Held<T, K> x(p.x, c.b * p.x_batch, p.x_token, tile, step, c.ch);
    Held<T, K> g(p.gate, c.b * p.gate_batch, p.gate_token, tile, step, c.ch);
    T* y = static_cast<T*>(p.y) + c.b * p.y_batch + (long long)tile * kTokens * p.y_token + c.ch;
    float* saved = p.saved ? p.saved + (c.b * c.tiles + tile) * p.channels + c.ch : nullptr;
    int left = (int)p.length - tile * kTokens, left_ahead = left;  // tokens from a tile's start to the row's end
    uint8_t head = 0;
    auto fetch = [&] {
        if constexpr (kTma) {
            if (c.lane == 0 && left_ahead > 0) ring.load(maps, (int)c.ch0, (int)p.length - left_ahead, (int)c.b);
            ring.next(ring.fill);
        } else {
            x.next(left_ahead, c.live);
            g.next(left_ahead, c.live);
        }
        left_ahead -= step * kTokens;
    };
    fetch();
    if (kTma) fetch();
    if (kCuts) head = head_of(p.heads, c.b, tile * kTokens, p.length, c.lane);
    V carry = p.state && c.live ? L::load(p.state + c.b * p.channels + c.ch) : L::all(0.0f);
    exchange_begin(s.ex, c.ranks);
    for (int round = 0; round < c.rounds; ++round) {
        const bool ok = !kTma || left <= 0 || ring.wait();
        const auto xr = tile_of<kTma>(ring, x, 0, c.lane), gr = tile_of<kTma>(ring, g, 1, c.lane);
        f2 f[kPairs<K>], b[kPairs<K>];
        const uint32_t cut = kCuts ? cuts_of<kTma>(head, ok) : 0u;
        if (kCuts) head = head_of(p.heads, c.b, (long long)(tile + step) * kTokens, p.length, c.lane);
        const int valid = min(left, kTokens);
#pragma unroll
        for (int i = 0; i < kPairs<K>; ++i) {
            if constexpr (kSigmoid) {
                gates<T>(gr.pair(i), f[i], b[i]);
                b[i] = mul2(b[i], xr.pair(i));
            } else {
                f[i] = gr.pair(i);
                b[i] = xr.pair(i);
            }
        }
        if (valid < kTokens) {  // behind the row's end: the state stays
#pragma unroll
            for (int j = 0; j < kTokens; ++j)
                if (j >= valid) {
                    set_token<K>(f, j, L::all(1.0f));
                    set_token<K>(b, j, L::all(0.0f));
                }
        }
        if (!ok) set_token<K>(b, 0, L::all(not_a_number()));
        __syncwarp();  // every lane has read
        fetch();
        Map<K> map{token<K>(f, 0), token<K>(b, 0)};
        if (!kCuts || cut == 0) {
#pragma unroll
            for (int j = 1; j < kTokens; ++j) {
                map.A = L::mul(map.A, token<K>(f, j));
                map.B = L::fma(token<K>(f, j), map.B, token<K>(b, j));
            }
        } else {
            map.A = L::all(0.0f);
#pragma unroll
            for (int j = 1; j < kTokens; ++j)
                map.B = cut >> j & 1u ? token<K>(b, j) : L::fma(token<K>(f, j), map.B, token<K>(b, j));
        }
        auto through = [&](int j, V v) {
            return kCuts && (cut >> j & 1u) ? token<K>(b, j) : L::fma(token<K>(f, j), v, token<K>(b, j));
        };
        auto walk = [&](V v) {
#pragma unroll
            for (int j = 0; j < kTokens; ++j) v = through(j, v);
            return v;
        };
        V h = exchange<K, kWarps, kCuts, !kSigmoid>(s.ex, round, c.warp, c.lane, c.rank, c.ranks, map, cut != 0, carry, walk);
        // A warp without a tile leaves its stage as it is: the copy of earlier results out of
        // it is waited for only where the stage is filled again (Ring::load).
        if (valid > 0) {
            if (saved && c.live) L::store(saved, h);
            T* to = y;
#pragma unroll
            for (int j = 0; j < kTokens; ++j) {
                h = through(j, h);
                if constexpr (kTma) {
                    xr.put(j, h);
                } else {
                    if (c.live && j < valid) Elements<T, K>::store(to, h);
                    to += p.y_token;
                }
            }
            if constexpr (kTma) {
                fence_proxy_async();
                __syncwarp();
                if (c.lane == 0) {
                    tma_store_3d(&maps.map[2], (int)c.ch0, tile * kTokens, (int)c.b, smem_u32(ring.take));
                    bulk_commit();
                }
            }
        }
        if constexpr (kTma) ring.next(ring.take);
        if (saved) saved += step * p.channels;
        y += (long long)step * kTokens * p.y_token;
        tile += step;
        left -= step * kTokens;
    }
    if (p.final_state && c.live && c.rank == 0 && c.warp == 0) L::store(p.final_state + c.b * p.channels + c.ch, carry);
    if (kTma && c.lane == 0) bulk_wait_read_all();
    exchange_end(c.ranks);
}

// --------------------------------------------------------------- gradient
template <class T, int K> using BackwardRing = Ring<T, K, 3, 2>;

// Warps, CTAs and rounds count from the end of the row.  Three tensors in registers, two
// channels a lane: 12 warps an SM (4 x 4096 tokens of 4094 bfloat16: 182 us; with one
// channel a lane 221 or more).
template <class T, int K, bool kTma, bool kSigmoid, int kWarps, bool kCuts>
__global__ void __launch_bounds__(32 * kWarps, (kTma || K == 1 ? 16 : 12) / kWarps)
    gated_grad_kernel(GatedParams p, const __grid_constant__ GatedMaps maps) {
    using L = Lane<K>;
    using V = typename L::V;
    using Sh = Shared<K, kWarps, BackwardRing<T, K>, kTma>;
    extern __shared__ __align__(128) unsigned char s_mem[];
    Sh& s = *reinterpret_cast<Sh*>(s_mem);
    const Place c = place_of<K, kWarps>(p);
    const int step = c.ranks * kWarps;
    int tile = c.tiles - 1 - (c.rank * kWarps + c.warp);
    BackwardRing<T, K> ring(s.ring[kTma ? c.warp : 0], kTma ? s.bars[c.warp] : nullptr, c.lane);
    Held<T, K> x(p.x, c.b * p.x_batch, p.x_token, tile, -step, c.ch);
    Held<T, K> g(p.gate, c.b * p.gate_batch, p.gate_token, tile, -step, c.ch);
    Held<T, K> dy(p.dy, c.b * p.dy_batch, p.dy_token, tile, -step, c.ch);
    const long long to = (c.b * p.length + (long long)tile * kTokens) * p.channels + c.ch;
    T *dx = static_cast<T*>(p.dx) + to, *dg = static_cast<T*>(p.dgate) + to;
    // a warp's first tile ends with the row, those before the row's first are none
    int ahead = tile;
    auto tokens_of = [&](int t) { return t < 0 ? 0 : min(kTokens, (int)p.length - t * kTokens); };
    uint8_t head = 0;
    V start = L::all(0.0f);
    auto fetch = [&] {
        if constexpr (kTma) {
            if (c.lane == 0 && ahead >= 0) ring.load(maps, (int)c.ch0, ahead * kTokens, (int)c.b);
            ring.next(ring.fill);
        } else {
            const int n = tokens_of(ahead);
            x.next(n, c.live);
            g.next(n, c.live);
            dy.next(n, c.live);
        }
        ahead -= step;
    };
    const float* saved = p.saved + (c.b * c.tiles + tile) * p.channels + c.ch;
    auto fetch_small = [&](int t) {  // a round ahead, in registers
        if (c.live && t >= 0) start = L::load(saved);
        saved -= step * p.channels;
        if (kCuts) head = head_of(p.heads, c.b, (long long)t * kTokens, p.length, c.lane);
    };
    fetch();
    fetch_small(tile);
    V carry = p.dfinal && c.live ? L::load(p.dfinal + c.b * p.channels + c.ch) : L::all(0.0f);
    exchange_begin(s.ex, c.ranks);
    const V one = L::all(1.0f), minus = L::all(-1.0f), none = L::all(0.0f);
    for (int round = 0; round < c.rounds; ++round) {
        if (kTma) fetch();
        const bool ok = !kTma || tile < 0 || ring.wait();
        const auto xr = tile_of<kTma>(ring, x, 0, c.lane), gr = tile_of<kTma>(ring, g, 1, c.lane);
        const auto d = tile_of<kTma>(ring, dy, 2, c.lane);
        // u: what dh is multiplied with for dgate; w: the smaller of f and 1 - f with the
        // gate's sign (sigmoid), or f itself.  map: q behind the tile -> q before it, as the
        // sum over its tokens of dy times the product of f from the tile's start up to there.
        f2 u[kPairs<K>], w[kPairs<K>];
        const uint32_t cut = kCuts ? cuts_of<kTma>(head, ok) : 0u;
        const int valid = tokens_of(tile), until = kCuts && cut ? __ffs(cut) - 1 : kTokens;
        V h = start;
        fetch_small(tile - step);
        Map<K> map{one, none};
        if constexpr (kSigmoid) {
#pragma unroll
            for (int i = 0; i < kPairs<K>; ++i) {
                f2 small, large;
                const f2 g2 = gr.pair(i);
                gate_parts<T>(g2, small, large);
                const f2 fs = select2(g2, small, large), rests = select2(g2, large, small);
                const f2 product = mul2(small, large);
                w[i] = small | (g2 & 0x8000000080000000ull);
#pragma unroll
                for (int j = i * 2 / K; j < (i + 1) * 2 / K; ++j) {
                    const V f = half<K>(fs, j), xv = xr.get(j);
                    if (kCuts && (cut >> j & 1u)) h = none;
                    set_token<K>(u, j, L::mul(L::fma(xv, minus, h), half<K>(product, j)));
                    h = L::fma(f, h, L::mul(half<K>(rests, j), xv));
                    map.A = L::mul(map.A, f);
                    if (!kCuts || j < until) map.B = L::fma(map.A, d.get(j), map.B);
                }
            }
        } else {
#pragma unroll
            for (int j = 0; j < kTokens; ++j) {
                const V f = gr.get(j), xv = xr.get(j);
                if (kCuts && (cut >> j & 1u)) h = none;
                set_token<K>(w, j, f);
                set_token<K>(u, j, h);
                h = kCuts && (cut >> j & 1u) ? xv : L::fma(f, h, xv);
            }
        }
        if (valid < kTokens) {  // behind the row's end: q stays
            map.A = one;
#pragma unroll
            for (int j = 0; j < kTokens; ++j) {
                V more = map.A, unused;
                if (j >= valid) set_token<K>(w, j, kSigmoid ? none : one);
                else if constexpr (kSigmoid) shares(token<K>(w, j), map.A, more, unused);
                map.A = more;
            }
            if (valid <= 0) map.B = none;
        }
        if constexpr (!kSigmoid) {
            if (valid > 0) {
#pragma unroll
                for (int j = kTokens - 1; j >= 0; --j) {
                    const V f = token<K>(w, j);
                    map.A = L::mul(map.A, f);
                    map.B = L::mul(f, L::add(d.get(j), map.B));
                    if (kCuts && (cut >> j & 1u)) map.B = none;
                }
            }
        }
        if (!ok) {  // q and all that is made of it
            map.A = map.B = L::all(not_a_number());
            set_token<K>(w, kTokens - 1, map.A);
            set_token<K>(u, kTokens - 1, map.A);
        }
        if (!kTma) fetch();
        auto walk = [&](V v) {
            if (valid > 0) {
#pragma unroll
                for (int j = kTokens - 1; j >= 0; --j) {
                    v = L::mul(token<K>(w, j), L::add(d.get(j), v));
                    if (kCuts && (cut >> j & 1u)) v = none;
                }
            }
            return v;
        };
        V q = exchange<K, kWarps, kCuts, !kSigmoid>(s.ex, round, c.warp, c.lane, c.rank, c.ranks, map, cut != 0, carry, walk);
        if (!kSigmoid && !ok) q = L::all(not_a_number());  // (dx is dh itself)
        if (valid > 0) {  // as in the forward kernel
            T *tx = dx + (kTokens - 1) * p.channels, *tg = dg + (kTokens - 1) * p.channels;
#pragma unroll
            for (int j = kTokens - 1; j >= 0; --j) {
                const V dh = L::add(d.get(j), q);
                V og = L::mul(dh, token<K>(u, j)), ox = dh;
                if constexpr (kSigmoid) shares(token<K>(w, j), dh, q, ox);
                else q = L::mul(token<K>(w, j), dh);
                if (kCuts && (cut >> j & 1u)) {
                    q = none;
                    if (!kSigmoid) og = none;
                }
                if constexpr (kTma) {
                    xr.put(j, ox);
                    gr.put(j, og);
                } else {
                    if (c.live && j < valid) {
                        Elements<T, K>::store(tx, ox);
                        Elements<T, K>::store(tg, og);
                    }
                    tx -= p.channels;
                    tg -= p.channels;
                }
            }
            if constexpr (kTma) {
                fence_proxy_async();
                __syncwarp();
                if (c.lane == 0) {
                    const uint32_t from = smem_u32(ring.take);
                    tma_store_3d(&maps.map[3], (int)c.ch0, tile * kTokens, (int)c.b, from);
                    tma_store_3d(&maps.map[4], (int)c.ch0, tile * kTokens, (int)c.b, from + Tile<T, K>::kBytes);
                    bulk_commit();
                }
            }
        }
        if constexpr (kTma) ring.next(ring.take);
        tile -= step;
        dx -= (long long)step * kTokens * p.channels;
        dg -= (long long)step * kTokens * p.channels;
    }
    if (p.dstate && c.live && c.rank == 0 && c.warp == 0) L::store(p.dstate + c.b * p.channels + c.ch, carry);
    if (kTma && c.lane == 0) bulk_wait_read_all();
    exchange_end(c.ranks);
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
            f2 f, rest;
            gates<T>(both(g[k]), f, rest);
            h[k] = fmaf(lo2(f), h[k], lo2(rest) * x[k]);
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
// The machine holds 16 warps an SM (128 registers a thread; the gradient of 16-bit tiles spills
// 72 to 88 bytes so, rows that are not aligned up to 184, the most where segments start
// anywhere).  CTAs of 4 warps where the
// rows and channels alone make enough of them (a round's fold is half as long, and they
// fill the SMs more evenly), else of 8.  CTAs in a cluster: until there are 12 warps an
// SM or the length has no more tiles (16 of them only where all clusters are resident at
// once, which takes as many SMs of one part of the chip each: 8192 tokens of 384 bfloat16
// channels, 6 clusters, 20 us with 8 CTAs and 16 with 16; of 512, 8 clusters, 22, and 27 or more with 16);
// and while the last wave of CTAs is mostly empty, up to 4.
struct Split {
    int warps, ctas;
};
inline Split split_of(long long groups, long long tiles) {
    const long long sms = seq_sms();
    Split s{groups * 4 >= 12 * sms || tiles <= 4 ? 4 : 8, 1};
    const long long slots = 16 / s.warps * sms;
    auto more = [&] {
        if ((long long)s.ctas * s.warps >= tiles) return false;
        const long long n = groups * s.ctas;
        if (n * s.warps < 12 * sms) return s.ctas < 8 || (s.ctas == 8 && groups * kMaxCluster * 3 <= sms * 2);
        return n > slots && s.ctas < 4 && n * 5 < (n + slots - 1) / slots * slots * 4;
    };
    while (more()) s.ctas *= 2;
    return s;
}

// Channels x tokens x rows, in boxes of a tile.
template <class T, int K>
bool map_of(CUtensorMap* m, const void* base, const GatedParams& p, long long batch, long long token) {
    PFN_cuTensorMapEncodeTiled_v12000 enc = persist::tensor_map_encoder();
    if (!enc) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)p.channels, (cuuint64_t)p.length, (cuuint64_t)p.batch};
    // a stride that is not used (one row, one token) may be anything that the engine takes
    const cuuint64_t row = (cuuint64_t)p.channels * sizeof(T);
    const cuuint64_t strides[2] = {p.length > 1 ? (cuuint64_t)token * sizeof(T) : row,
                                   p.batch > 1 ? (cuuint64_t)batch * sizeof(T) : row};
    const cuuint32_t box[3] = {32 * K, kTokens, 1}, each[3] = {1, 1, 1};
    const CUtensorMapDataType type = sizeof(T) == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_UINT16;
    return enc(m, type, 3, const_cast<void*>(base), dims, strides, box, each, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
template <class T, int K>
bool maps_of(GatedMaps* m, const GatedParams& p, bool grad) {
    if (!map_of<T, K>(&m->map[0], p.x, p, p.x_batch, p.x_token) ||
        !map_of<T, K>(&m->map[1], p.gate, p, p.gate_batch, p.gate_token))
        return false;
    if (!grad) return map_of<T, K>(&m->map[2], p.y, p, p.y_batch, p.y_token);
    const long long row = p.length * p.channels;
    return map_of<T, K>(&m->map[2], p.dy, p, p.dy_batch, p.dy_token) && map_of<T, K>(&m->map[3], p.dx, p, row, p.channels) &&
           map_of<T, K>(&m->map[4], p.dgate, p, row, p.channels);
}

template <class T, int K, bool kTma, bool kSigmoid, int kWarps, bool kCuts>
cudaError_t go(const GatedParams& p, const GatedMaps& maps, bool grad, long long groups, int ctas, cudaStream_t s) {
    const void* kernel = grad ? (const void*)gated_grad_kernel<T, K, kTma, kSigmoid, kWarps, kCuts>
                              : (const void*)gated_kernel<T, K, kTma, kSigmoid, kWarps, kCuts>;
    auto bytes = [&](int n) {
        return (int)(grad ? Shared<K, kWarps, BackwardRing<T, K>, kTma>::bytes(n)
                          : Shared<K, kWarps, ForwardRing<T, K>, kTma>::bytes(n));
    };
    // the limit is one per device: always the largest, whatever this call needs
    cudaError_t e = cudaSuccess;
    if (bytes(ctas) > kDefaultShared)
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes(kMaxCluster));
    if (e == cudaSuccess && ctas > 8)
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute a{};
    a.id = cudaLaunchAttributeClusterDimension;
    a.val.clusterDim.y = a.val.clusterDim.z = 1;
    cfg.blockDim = dim3(32 * kWarps);
    cfg.stream = s;
    cfg.attrs = &a;
    cfg.numAttrs = 1;
    auto size = [&](int n) {
        a.val.clusterDim.x = (unsigned)n;
        cfg.gridDim = dim3((unsigned)(groups * n));
        cfg.dynamicSmemBytes = (size_t)bytes(n);
    };
    size(ctas);
    static LargeClusters large[2];
    if (ctas > 8 && !large[grad].fit(kernel, cfg)) size(8);
    void* args[] = {const_cast<GatedParams*>(&p), const_cast<GatedMaps*>(&maps)};
    e = cudaLaunchKernelExC(&cfg, kernel, args);
    count_launches(1);
    return e;
}

template <class T, int K, bool kTma, bool kSigmoid>
cudaError_t by_length(const GatedParams& p, const GatedMaps& maps, bool grad, cudaStream_t s) {
    const long long tiles = (p.length + kTokens - 1) / kTokens, groups = p.batch * ((p.channels + 32 * K - 1) / (32 * K));
    const Split split = split_of(groups, tiles);
    if (split.warps == 4)
        return p.heads ? go<T, K, kTma, kSigmoid, 4, true>(p, maps, grad, groups, split.ctas, s)
                       : go<T, K, kTma, kSigmoid, 4, false>(p, maps, grad, groups, split.ctas, s);
    return p.heads ? go<T, K, kTma, kSigmoid, 8, true>(p, maps, grad, groups, split.ctas, s)
                   : go<T, K, kTma, kSigmoid, 8, false>(p, maps, grad, groups, split.ctas, s);
}

template <class T, int K, bool kTma>
cudaError_t by_gate(const GatedParams& p, const GatedMaps& maps, bool grad, cudaStream_t s) {
    return p.sigmoid ? by_length<T, K, kTma, true>(p, maps, grad, s) : by_length<T, K, kTma, false>(p, maps, grad, s);
}

template <class T>
cudaError_t launch_gated_as(const GatedParams& p, bool grad, cudaStream_t s) {
    constexpr int K = 4 / (int)sizeof(T);  // 4 bytes a lane
    GatedMaps maps{};
    if (p.wide && maps_of<T, K>(&maps, p, grad)) return by_gate<T, K, true>(p, maps, grad, s);
    if constexpr (K == 2) {
        if (p.pairs) return by_gate<T, 2, false>(p, maps, grad, s);
    }
    return by_gate<T, 1, false>(p, maps, grad, s);
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
