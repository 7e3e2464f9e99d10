// The norm of a token's channels (with the residual sum in front of it) and its
// gradient: kernels, by element type in sc_norm_*.cu.
//
//   s = x + residual, rounded;  n = (s - m) r;  y = n weight + bias
//   dn = dy weight;  dx = r (dn - mean(dn) - n mean(dn n)) + dsum
//   dweight = sum over tokens of dy n;  dbias = sum over tokens of dy
// (rms: m = 0, and mean(dn) drops out.)
//
// A row lies in the registers of kLanes threads, N elements each, so each tensor is
// read and written once: bytes are all that the operator costs.  The variance is of the
// centred row, a second sum over registers, not a difference of moments.  Rows of up to
// 32 vectors of 16 bytes take part of a warp or one, wider ones up to 1024 threads, which
// then meet in shared memory.  Rows beyond kRowMax elements are read again for each of
// their sums.
//
// CTAs stay and take rows in turns, with the parameters (and the gradient's sums over
// tokens) in registers.  A team, the threads of a wide row or a warp with several
// narrow ones, has a ring of rows in shared memory that bulk copies fill some turns
// ahead; rows that are not aligned to 16 bytes, and calls of one turn, are loaded into
// registers, the next row's while this one is worked on.  (Unaligned rows through the
// ring, their ends by themselves: 17367 rows of 636 bfloat16 43 us forward, 23 so.)
//
// Should a copy not come, its row is NaN, and so are the ring's later ones.  One flag for
// all turns costs nothing; leaving the later waits or loads out made the gradient of 262144
// rows of 128 float16 55 us in place of 45, as a ring's state then differs between lanes.
//
// 4 x 4096 rows of 4096 bfloat16 with a residual: forward 85 us, gradient 87 and its sums
// 8 (6.2 TB/s; a copy 6.5).
//
// The gradient's sums over tokens: a CTA's columns' sums over all its rows become one row
// of partial sums, and a second kernel adds those in the order of the CTAs: the same bits
// on every run.
#pragma once
#include <algorithm>

#include "sc_bulk.cuh"
#include "sc_seq.cuh"
#include "sc_seq_launch.h"

namespace scg {

namespace {

constexpr long long kRowMax = 8192;

template <class T> constexpr int kWidth = 16 / (int)sizeof(T);  // elements of a vector

// A row's first element: rows of `length` tokens, or all in one stride (length >= rows).
__device__ __forceinline__ long long at(uint32_t row, uint32_t length, long long sb, long long st) {
    if (row < length) return (long long)row * st;
    const uint32_t b = row / length;
    return (long long)b * sb + (long long)(row - b * length) * st;
}

// How rows come: by the widest accesses that all of them are aligned to, single 16-bit
// elements, 4 bytes, or vectors of 16; or by vectors through the ring.
enum Way { kElements, kUnits, kVectors, kRing };
template <Way kWay> constexpr bool kByVectors = kWay == kVectors || kWay == kRing;
template <class T, Way kWay>  // elements of an access
constexpr int kAccess = kByVectors<kWay> ? kWidth<T> : kWay == kUnits ? 4 / (int)sizeof(T) : 1;

// Element j of vector i of a lane: the lanes' accesses lie side by side.
template <class T, Way kWay, int kLanes>
__device__ __forceinline__ int column(int i, int j, int lane) {
    constexpr int A = kAccess<T, kWay>;
    return ((i * (kWidth<T> / A) + j / A) * kLanes + lane) * A + j % A;
}

template <class T, Way kWay, int kLanes, int NV>
struct Row {
    static constexpr int W = kWidth<T>, A = kAccess<T, kWay>;
    Vec<T, W> v[NV];
    __device__ __forceinline__ void load(const T* p, int lane, int channels) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if constexpr (kByVectors<kWay>) {
                const int c = column<T, kWay, kLanes>(i, 0, lane);
                if (c < channels) v[i].load(p + c);
                else v[i].zero();
            } else if constexpr (kWay == kUnits) {
#pragma unroll
                for (int j = 0; j < W; j += A) {
                    const int c = column<T, kWay, kLanes>(i, j, lane);
                    v[i].w[j / A] = c < channels ? __ldg(reinterpret_cast<const uint32_t*>(p + c)) : 0u;
                }
            } else {
                T e[W];
#pragma unroll
                for (int j = 0; j < W; ++j) {
                    const int c = column<T, kWay, kLanes>(i, j, lane);
                    e[j] = c < channels ? __ldg(p + c) : from_f32<T>(0.0f);
                }
                memcpy(v[i].w, e, 16);
            }
        }
    }
    __device__ __forceinline__ void load_shared(const unsigned char* row, int lane, int channels) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = column<T, kRing, kLanes>(i, 0, lane);
            if (c < channels) v[i].load_rw(reinterpret_cast<const T*>(row) + c);
            else v[i].zero();
        }
    }
    // NaN in every element, of whichever type.
    __device__ __forceinline__ void spoil() {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < Vec<T, W>::kWords; ++j) v[i].w[j] = 0x7fff7fffu;
    }
    // Elements 2 j and 2 j + 1 of vector i.
    __device__ __forceinline__ f2 pair(int i, int j) const { return v[i].pair(j); }
    // The elements of f (as pairs, vector by vector) to a row, rounded; `rounded`: and back in f.
    template <bool kRounded = false>
    __device__ __forceinline__ static void store(T* p, int lane, int channels, f2 (&f)[NV * W / 2]) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            Vec<T, W> o;
#pragma unroll
            for (int j = 0; j < W / 2; ++j) set_pair(o, j, f[i * W / 2 + j]);
            if (kRounded)
#pragma unroll
                for (int j = 0; j < W / 2; ++j) f[i * W / 2 + j] = o.pair(j);
            if constexpr (kByVectors<kWay>) {
                const int c = column<T, kWay, kLanes>(i, 0, lane);
                if (c < channels) o.store(p + c);
            } else {
                T e[W];
                memcpy(e, o.w, 16);
#pragma unroll
                for (int j = 0; j < W; j += A) {
                    const int c = column<T, kWay, kLanes>(i, j, lane);
                    if (c >= channels) continue;
                    if constexpr (kWay == kUnits) *reinterpret_cast<uint32_t*>(p + c) = o.w[j / A];
                    else p[c] = e[j];
                }
            }
        }
    }
    __device__ __forceinline__ static void set_pair(Vec<T, W>& o, int j, f2 v) {
        if constexpr (sizeof(T) == 4) {
            o.w[2 * j] = __float_as_uint(lo2(v));
            o.w[2 * j + 1] = __float_as_uint(hi2(v));
        } else if constexpr (std::is_same<T, bf16>::value) {
            const __nv_bfloat162 e = __floats2bfloat162_rn(lo2(v), hi2(v));
            memcpy(&o.w[j], &e, 4);
        } else {
            const __half2 e = __floats2half2_rn(lo2(v), hi2(v));
            memcpy(&o.w[j], &e, 4);
        }
    }
};
__device__ __forceinline__ float sum2(f2 v) { return lo2(v) + hi2(v); }
// 1 / sqrt(v): the instruction's result and a step of Newton's, which would make NaN of 0
// and of infinity (rounding: within 1.5 units of 2^-23; the instruction's is 2).
__device__ __forceinline__ float inverse_root(float v) {
    const float r = rsqrtf(v), n = fmaf(0.5f * r, fmaf(-v * r, r, 1.0f), r);
    return n == n ? n : r;
}

template <class T>
__device__ __forceinline__ float parameter(const void* p, int f32, int c) {
    return f32 ? __ldg(static_cast<const float*>(p) + c) : to_f32(__ldg(static_cast<const T*>(p) + c));
}

// The sum of K values over the kLanes threads of a row, in a fixed order.  `slot`:
// shared memory of the row's own, for this sum; two calls in turn take two slots, since
// a thread may be at the next sum while another still reads this one's.
template <int kLanes, int K>
__device__ __forceinline__ void row_sum(float (&v)[K], float* slot, int lane, int group) {
#pragma unroll
    for (int o = 1; o < (kLanes < 32 ? kLanes : 32); o <<= 1)
#pragma unroll
        for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
    if constexpr (kLanes > 32) {
        constexpr int kWarps = kLanes / 32;
        if ((lane & 31) == 0) {
#pragma unroll
            for (int k = 0; k < K; ++k) slot[k * kWarps + (lane >> 5)] = v[k];
        }
        asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "n"(kLanes) : "memory");
#pragma unroll
        for (int k = 0; k < K; ++k) {
            float s[kWarps];
            constexpr int kAtOnce = kWarps < 4 ? kWarps : 4;
#pragma unroll
            for (int w = 0; w < kWarps; w += kAtOnce) {
                if constexpr (kAtOnce == 4) {
                    const float4 q = *reinterpret_cast<const float4*>(slot + k * kWarps + w);
                    s[w] = q.x, s[w + 1] = q.y, s[w + 2] = q.z, s[w + 3] = q.w;
                } else {
                    const float2 q = *reinterpret_cast<const float2*>(slot + k * kWarps + w);
                    s[w] = q.x, s[w + 1] = q.y;
                }
            }
            // in pairs, then their sums, for a short chain
#pragma unroll
            for (int o = 1; o < kWarps; o *= 2)
#pragma unroll
                for (int w = 0; w < kWarps; w += 2 * o) s[w] += s[w + o];
            v[k] = s[0];
        }
    }
}

template <int kLanes> constexpr int kThreads = kLanes < 256 ? 256 : kLanes;

// A team: the threads of a row, or a warp with kSide rows side by side, and two of them
// one behind the other where they are short (four: 262144 rows of 128 16-bit channels 31 us
// forward, 29 so, and the gradient spills).
template <class T, Way kWay, int kLanes, int NV> struct Team {
    static constexpr int W = kWidth<T>, N = NV * W, NT = kThreads<kLanes>;
    static constexpr int kSize = kLanes > 32 ? kLanes : 32, kTeams = NT / kSize;
    static constexpr int kSide = kLanes < 32 ? 32 / kLanes : 1, kDeep = NV == 1 && kLanes <= 32 && kWay == kRing ? 2 : 1;
    static constexpr int kRows = kSide * kDeep;  // of a turn
    static constexpr int kGroups = NT / kLanes;
};

// A team's ring: stages of kTensors x kRows rows.
template <class T, int kTensors, int kRows>
struct RowRing {
    const T* from[kTensors];
    long long sb[kTensors], st[kTensors];
    uint32_t row_bytes, length;
    unsigned char* base;
    uint32_t bar;  // of stage 0
    int stages, fill = 0, take = 0, tensors;
    uint32_t phase = 0;
    bool dense;  // all rows follow one another

    __device__ __forceinline__ int bytes() const { return tensors * kRows * (int)row_bytes; }
    __device__ __forceinline__ void begin(unsigned char* mem, uint64_t* bars, int n, int thread) {
        base = mem;
        bar = smem_u32(bars);
        stages = n;
        if (thread == 0) {
            for (int i = 0; i < n; ++i) mbar_init(bar + 8 * i, 1);
            fence_mbar_init();
        }
    }
    // The rows [r0, r0 + n) into the next stage; by the team's first warp, when the whole
    // team has read what was there.
    __device__ __forceinline__ void load(uint32_t r0, int n, int lane) {
        const uint32_t full = bar + 8 * fill, to = smem_u32(base) + fill * bytes();
        if (lane == 0) mbar_arrive_expect_tx(full, (uint32_t)(tensors * n) * row_bytes);
#pragma unroll
        for (int i = 0; i < kTensors; ++i) {
            if (i >= tensors) break;
            const uint32_t dst = to + i * kRows * row_bytes;
            if (kRows == 1 || dense) {
                if (lane == 0) bulk_load(dst, from[i] + at(r0, length, sb[i], st[i]), n * row_bytes, full);
            } else if (lane < n) {
                bulk_load(dst + lane * row_bytes, from[i] + at(r0 + lane, length, sb[i], st[i]), row_bytes, full);
            }
        }
        if (++fill == stages) fill = 0;
    }
    __device__ __forceinline__ bool wait() const { return arrived(bar + 8 * take, phase); }
    __device__ __forceinline__ const unsigned char* row(int i, int r) const {
        return base + take * bytes() + (i * kRows + r) * row_bytes;
    }
    __device__ __forceinline__ void taken() {
        if (++take == stages) {
            take = 0;
            phase ^= 1;
        }
    }
};

// The rows of a team's turns, of 1 or 2 tensors forward, 2 or 3 backward.
template <class T, Way kWay, int kLanes, int NV, int kTensors>
struct Turns {
    using G = Team<T, kWay, kLanes, NV>;
    using R = Row<T, kWay, kLanes, NV>;
    RowRing<T, kTensors, G::kRows> ring;
    R next[kWay == kRing ? 1 : kTensors][kWay == kRing ? 1 : G::kDeep];
    uint32_t rows, step, ahead;  // below 2^31; a turn behind the last stays below 2^32
    int thread, lane, side, channels;  // thread: of the team

    __device__ __forceinline__ void begin(const NormParams& p, unsigned char* mem, const void* const* from,
                                          const long long* sb, const long long* st, int tensors) {
        const int team = threadIdx.x / G::kSize;
        thread = threadIdx.x % G::kSize;
        lane = threadIdx.x % kLanes;
        side = kLanes < 32 ? thread / kLanes : 0;
        channels = (int)p.channels;
        rows = p.rows;
        ahead = first();
        step = gridDim.x * (uint32_t)(G::kTeams * G::kRows);
        ring.tensors = tensors;
        ring.length = p.length;
        ring.dense = p.dense;
        ring.row_bytes = (uint32_t)(channels * sizeof(T));
#pragma unroll
        for (int i = 0; i < kTensors; ++i) {
            ring.from[i] = static_cast<const T*>(from[i]);
            ring.sb[i] = sb[i];
            ring.st[i] = st[i];
        }
        if constexpr (kWay == kRing) {
            uint64_t* bars = reinterpret_cast<uint64_t*>(mem + (long long)G::kTeams * p.stages * ring.bytes());
            ring.begin(mem + (long long)team * p.stages * ring.bytes(), bars + team * p.stages, p.stages, thread);
            __syncthreads();
            for (int i = 0; i < p.stages; ++i) fetch();
        } else {
            fetch();
        }
    }
    __device__ __forceinline__ uint32_t first() const {
        return (blockIdx.x * G::kTeams + threadIdx.x / G::kSize) * (uint32_t)G::kRows;
    }
    // This thread's row d of the turn that begins with `base`.
    __device__ __forceinline__ uint32_t row(uint32_t base, int d) const { return base + d * G::kSide + side; }
    // The turn after those under way.
    __device__ __forceinline__ void fetch() {
        if (ahead >= rows) return;
        if constexpr (kWay == kRing) {
            if (thread < 32) ring.load(ahead, (int)min((uint32_t)G::kRows, rows - ahead), thread);
        } else {
#pragma unroll
            for (int i = 0; i < kTensors; ++i) {
                if (i >= ring.tensors) break;
#pragma unroll
                for (int d = 0; d < G::kDeep; ++d) {
                    const uint32_t r = row(ahead, d);
                    const bool live = r < rows;
                    next[i][d].load(ring.from[i] + at(live ? r : 0u, ring.length, ring.sb[i], ring.st[i]), lane,
                                    live ? channels : 0);
                }
            }
        }
        ahead += step;
    }
    // The turn's rows of tensor i, when wait() says that they are there.
    __device__ __forceinline__ bool wait() const {
        if constexpr (kWay == kRing) return ring.wait();
        else return true;
    }
    __device__ __forceinline__ void take(int i, uint32_t base, R (&to)[G::kDeep]) const {
#pragma unroll
        for (int d = 0; d < G::kDeep; ++d) {
            if constexpr (kWay == kRing)
                to[d].load_shared(ring.row(i, d * G::kSide + side), lane, row(base, d) < rows ? channels : 0);
            else
                to[d] = next[i][d];
        }
    }
    // Every thread of the team has taken its rows (a barrier lies between): the next turn's
    // may come.
    __device__ __forceinline__ void done() {
        if constexpr (kWay == kRing) {
            if constexpr (kLanes <= 32) __syncwarp();
            ring.taken();
            fetch();
        }
    }
};

// ---------------------------------------------------------------- forward
// Threads that an SM's 65536 registers hold, 80 a thread through the ring, 128 with 16
// elements of a row and of the next, 64 with 8; and CTAs of them.
template <class T, Way kWay> constexpr int kHeld = kWay == kRing ? 768 : kWay == kVectors && sizeof(T) == 2 ? 512 : 1024;
template <class T, Way kWay, int kLanes>
constexpr int kResident = kHeld<T, kWay> > kThreads<kLanes> ? kHeld<T, kWay> / kThreads<kLanes> : 1;

template <class T, Way kWay, int kLanes, int NV>
__global__ void __launch_bounds__(kThreads<kLanes>, kResident<T, kWay, kLanes>) norm_kernel(NormParams p) {
    using G = Team<T, kWay, kLanes, NV>;
    using R = Row<T, kWay, kLanes, NV>;
    constexpr int W = G::W, N = G::N, D = G::kDeep;
    __shared__ __align__(16) float s_sum[G::kGroups][2][2][kLanes > 32 ? kLanes / 32 : 1];
    extern __shared__ __align__(128) unsigned char s_mem[];
    const int group = threadIdx.x / kLanes, channels = (int)p.channels;
    Turns<T, kWay, kLanes, NV, 2> turns;
    {
        const void* const from[2] = {p.x, p.residual};
        const long long sb[2] = {p.x_batch, p.residual_batch}, st[2] = {p.x_token, p.residual_token};
        turns.begin(p, s_mem, from, sb, st, p.residual ? 2 : 1);
    }
    const int lane = turns.lane;
    f2 w[N / 2], b[N / 2];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < W; j += 2) {
            float v[2][2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int c = column<T, kWay, kLanes>(i, j + h, lane);
                v[0][h] = c < channels && p.weight ? parameter<T>(p.weight, p.params_f32, c) : 1.0f;
                v[1][h] = c < channels && p.bias ? parameter<T>(p.bias, p.params_f32, c) : 0.0f;
            }
            w[(i * W + j) / 2] = pack2(v[0][0], v[0][1]);
            b[(i * W + j) / 2] = pack2(v[1][0], v[1][1]);
        }
    const float per = 1.0f / (float)channels;
    const bool full = channels == kLanes * N;
    int turn = 0;
    bool good = true;  // all rows up to here came
    for (uint32_t base = turns.first(); base < turns.rows; base += turns.step) {
        good = turns.wait() && good;
        R x[D];
        turns.take(0, base, x);
        if (!good) {
#pragma unroll
            for (int d = 0; d < D; ++d) x[d].spoil();
        }
        f2 f[D][N / 2];
#pragma unroll
        for (int d = 0; d < D; ++d)
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int j = 0; j < W / 2; ++j) f[d][i * W / 2 + j] = x[d].pair(i, j);
        if (p.residual) {
            turns.take(1, base, x);
#pragma unroll
            for (int d = 0; d < D; ++d) {
#pragma unroll
                for (int i = 0; i < NV; ++i)
#pragma unroll
                    for (int j = 0; j < W / 2; ++j) f[d][i * W / 2 + j] = add2(f[d][i * W / 2 + j], x[d].pair(i, j));
                const uint32_t r = turns.row(base, d);
                const bool live = r < turns.rows;
                R::template store<true>(static_cast<T*>(p.sum) + at(live ? r : 0u, p.length, p.sum_batch, p.sum_token),
                                        lane, live ? channels : 0, f[d]);
            }
        }
        if constexpr (kWay != kRing) turns.fetch();
        float mean[D], q[D];
#pragma unroll
        for (int d = 0; d < D; ++d) mean[d] = 0.0f;
        if (!p.rms) {
#pragma unroll
            for (int d = 0; d < D; ++d) {
                f2 sum = f[d][0];
#pragma unroll
                for (int i = 1; i < N / 2; ++i) sum = add2(sum, f[d][i]);
                mean[d] = sum2(sum);
            }
            row_sum<kLanes, D>(mean, &s_sum[group][turn][0][0], lane, group);
#pragma unroll
            for (int d = 0; d < D; ++d) {
                mean[d] *= per;
#pragma unroll
                for (int i = 0; i < N / 2; ++i) f[d][i] = add2(f[d][i], both(-mean[d]));
            }
            if (!full) {  // behind the row's end: not minus the mean
#pragma unroll
                for (int d = 0; d < D; ++d)
#pragma unroll
                    for (int i = 0; i < NV; ++i)
#pragma unroll
                        for (int j = 0; j < W / 2; ++j) {
                            f2& v = f[d][i * W / 2 + j];
                            if (kAccess<T, kWay> > 1) v = column<T, kWay, kLanes>(i, 2 * j, lane) < channels ? v : 0ull;
                            else v = pack2(column<T, kWay, kLanes>(i, 2 * j, lane) < channels ? lo2(v) : 0.0f,
                                           column<T, kWay, kLanes>(i, 2 * j + 1, lane) < channels ? hi2(v) : 0.0f);
                        }
            }
        }
#pragma unroll
        for (int d = 0; d < D; ++d) {
            f2 sum = mul2(f[d][0], f[d][0]);
#pragma unroll
            for (int i = 1; i < N / 2; ++i) sum = fma2(f[d][i], f[d][i], sum);
            q[d] = sum2(sum);
        }
        row_sum<kLanes, D>(q, &s_sum[group][turn][1][0], lane, group);
        turn ^= 1;
        turns.done();
#pragma unroll
        for (int d = 0; d < D; ++d) {
            const uint32_t r = turns.row(base, d);
            const bool live = r < turns.rows;
            const float rstd = inverse_root(fmaf(q[d], per, p.eps));
            if (p.saved && lane == 0 && live) reinterpret_cast<float2*>(p.saved)[r] = make_float2(mean[d], rstd);
#pragma unroll
            for (int i = 0; i < N / 2; ++i) f[d][i] = fma2(mul2(f[d][i], both(rstd)), w[i], b[i]);
            R::store(static_cast<T*>(p.y) + at(live ? r : 0u, p.length, p.y_batch, p.y_token), lane, live ? channels : 0,
                     f[d]);
        }
    }
}

// --------------------------------------------------------------- gradient
// 128 registers a thread (64 of 1024 threads); 80 where a thread has 8 elements of one row
// and two tensors (3003 rows of 2047 float32: 27 us with two CTAs an SM, 25 with three; two
// 16-bit rows a thread spill so, and take 55 us in place of 49).  kSum: dsum is there.
// Of the gradients with dsum, those that load 16 elements a thread and tensor into registers
// spill 24 to 52 bytes (16 bits, calls of one turn), and with 1024 threads 16 to 64 (16 bits,
// unaligned) and 176 to 208 (float32, 4097 to 8192 channels; without dsum 32 to 72).
template <class T, Way kWay, int kLanes, int NV, bool kSum>
constexpr int kGradResident = kThreads<kLanes> > 256                                                        ? 1
                              : kWidth<T> * NV == 8 && !kSum && (kWay != kRing || sizeof(T) == 4) ? 3
                                                                                                   : 2;

template <class T, Way kWay, int kLanes, int NV, bool kSum>
__global__ void __launch_bounds__(kThreads<kLanes>, kGradResident<T, kWay, kLanes, NV, kSum>) norm_grad_kernel(NormParams p) {
    using G = Team<T, kWay, kLanes, NV>;
    using R = Row<T, kWay, kLanes, NV>;
    constexpr int W = G::W, N = G::N, D = G::kDeep, NT = G::NT, kGroups = G::kGroups;
    __shared__ __align__(16) float s_sum[kGroups][2][2 * D * (kLanes > 32 ? kLanes / 32 : 1)];
    extern __shared__ __align__(128) unsigned char s_mem[];
    const int group = threadIdx.x / kLanes, channels = (int)p.channels;
    constexpr int kTensors = kSum ? 3 : 2;
    Turns<T, kWay, kLanes, NV, kTensors> turns;
    {
        const void* from[kTensors] = {p.x, p.dy};
        long long sb[kTensors] = {p.x_batch, p.dy_batch}, st[kTensors] = {p.x_token, p.dy_token};
        if constexpr (kSum) {
            from[2] = p.dsum;
            sb[2] = p.dsum_batch;
            st[2] = p.dsum_token;
        }
        turns.begin(p, s_mem, from, sb, st, kTensors);
    }
    const int lane = turns.lane;
    f2 w[N / 2], dw[N / 2], db[N / 2];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < W; j += 2) {
            float v[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int c = column<T, kWay, kLanes>(i, j + h, lane);
                v[h] = c >= channels ? 0.0f : p.weight ? parameter<T>(p.weight, p.params_f32, c) : 1.0f;
            }
            w[(i * W + j) / 2] = pack2(v[0], v[1]);
            dw[(i * W + j) / 2] = db[(i * W + j) / 2] = 0ull;
        }
    const float per = 1.0f / (float)channels;
    float2 stat[D];
    auto fetch_stat = [&](uint32_t base) {
#pragma unroll
        for (int d = 0; d < D; ++d) {
            const uint32_t r = turns.row(base, d);
            stat[d] = r < turns.rows ? __ldg(reinterpret_cast<const float2*>(p.saved) + r) : make_float2(0.0f, 0.0f);
        }
    };
    int turn = 0;
    bool good = true;  // all rows up to here came
    fetch_stat(turns.first());
    for (uint32_t base = turns.first(); base < turns.rows; base += turns.step) {
        good = turns.wait() && good;
        R x[D], dy[D], ds[kSum ? D : 1];
        turns.take(0, base, x);
        turns.take(1, base, dy);
        if constexpr (kSum) turns.take(2, base, ds);
        float mean[D], rstd[D], s[2 * D];
#pragma unroll
        for (int d = 0; d < D; ++d) {
            mean[d] = stat[d].x;
            rstd[d] = good ? stat[d].y : not_a_number();
        }
        fetch_stat(base + turns.step);
        if constexpr (kWay != kRing) turns.fetch();
#pragma unroll
        for (int d = 0; d < D; ++d) {
            f2 a = 0ull, b = 0ull;
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int j = 0; j < W / 2; ++j) {
                    const int k = i * W / 2 + j;
                    const f2 n = mul2(add2(x[d].pair(i, j), both(-mean[d])), both(rstd[d]));
                    const f2 g = dy[d].pair(i, j), dn = mul2(g, w[k]);
                    a = add2(a, dn);
                    b = fma2(dn, n, b);  // w = 0 behind the row's end, where n is not 0
                    db[k] = add2(db[k], g);
                    dw[k] = fma2(g, n, dw[k]);
                }
            s[2 * d] = sum2(a);
            s[2 * d + 1] = sum2(b);
        }
        row_sum<kLanes, 2 * D>(s, s_sum[group][turn], lane, group);
        turn ^= 1;
        turns.done();
#pragma unroll
        for (int d = 0; d < D; ++d) {
            const f2 a = both(p.rms ? 0.0f : -s[2 * d] * per), b = both(-s[2 * d + 1] * per);
            f2 o[N / 2];
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int j = 0; j < W / 2; ++j) {
                    const int k = i * W / 2 + j;
                    const f2 n = mul2(add2(x[d].pair(i, j), both(-mean[d])), both(rstd[d]));
                    o[k] = fma2(n, b, fma2(dy[d].pair(i, j), w[k], a));
                }
            if constexpr (kSum) {
#pragma unroll
                for (int i = 0; i < NV; ++i)
#pragma unroll
                    for (int j = 0; j < W / 2; ++j) o[i * W / 2 + j] = fma2(o[i * W / 2 + j], both(rstd[d]), ds[d].pair(i, j));
            } else {
#pragma unroll
                for (int k = 0; k < N / 2; ++k) o[k] = mul2(o[k], both(rstd[d]));
            }
            const uint32_t r = turns.row(base, d);
            const bool live = r < turns.rows;
            R::store(static_cast<T*>(p.dx) + (long long)(live ? r : 0u) * channels, lane, live ? channels : 0, o);
        }
    }
    if (!p.partials) return;
    if (!good) {  // dy of rows that did not come
#pragma unroll
        for (int k = 0; k < N / 2; ++k) db[k] = both(not_a_number());
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the kernel that adds the partial sums may get ready
    // one row of partial sums a CTA: over its groups, in their order
    float* s_col = reinterpret_cast<float*>(s_mem);
    auto put = [&](int which, const f2 (&v)[N / 2]) {
        auto element = [&](int k) { return k % 2 ? hi2(v[k / 2]) : lo2(v[k / 2]); };
        float* to = p.partials + ((long long)blockIdx.x * 2 + which) * channels;
        if constexpr (kGroups == 1) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int j = 0; j < W; ++j) {
                    const int c = column<T, kWay, kLanes>(i, j, lane);
                    if (c < channels) to[c] = element(i * W + j);
                }
        } else {
            __syncthreads();
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int j = 0; j < W; ++j)
                    s_col[group * (kLanes * N) + column<T, kWay, kLanes>(i, j, lane)] = element(i * W + j);
            __syncthreads();
            for (int c = threadIdx.x; c < channels; c += NT) {
                float sum = 0.0f;
#pragma unroll
                for (int g = 0; g < kGroups; ++g) sum += s_col[g * (kLanes * N) + c];
                to[c] = sum;
            }
        }
    };
    if (p.dweight) put(0, dw);
    if (p.dbias) put(1, db);
}

// ------------------------------------------------------------- wide rows
// One CTA a row, the row read once for each of its sums (the second time from L2).
constexpr int kWideNT = 1024;

template <int K>
__device__ __forceinline__ void cta_sum(float (&v)[K], float* slot) {
    row_sum<kWideNT, K>(v, slot, threadIdx.x, 0);
}

// f(column, element of each row) over a row, 16 bytes a thread where rows are aligned
template <class T, bool kVec, class F>
__device__ __forceinline__ void each(long long channels, F f) {
    constexpr int W = kVec ? kWidth<T> : 1;
    for (long long c = (long long)threadIdx.x * W; c < channels; c += kWideNT * W) f(c);
}
template <class T, bool kVec> constexpr int kEach = kVec ? kWidth<T> : 1;
template <class T, bool kVec>
__device__ __forceinline__ void take(const T* p, float (&f)[kEach<T, kVec>]) {
    if constexpr (kVec) {
        Vec<T, kWidth<T>> v;
        v.load_rw(p);
#pragma unroll
        for (int i = 0; i < kWidth<T>; ++i) f[i] = v.get(i);
    } else {
        f[0] = to_f32(*p);
    }
}
template <class T, bool kVec>
__device__ __forceinline__ void give(T* p, const float (&f)[kEach<T, kVec>]) {
    if constexpr (kVec) {
        Vec<T, kWidth<T>> v;
        v.set(f);
        v.store(p);
    } else {
        *p = from_f32<T>(f[0]);
    }
}

template <class T, bool kVec>
__global__ void __launch_bounds__(kWideNT) norm_wide_kernel(NormParams p) {
    constexpr int E = kEach<T, kVec>;
    __shared__ __align__(16) float slot[2][kWideNT / 32];
    const uint32_t r = blockIdx.x;
    const T* x = static_cast<const T*>(p.x) + at(r, p.length, p.x_batch, p.x_token);
    T* y = static_cast<T*>(p.y) + at(r, p.length, p.y_batch, p.y_token);
    const long long ch = p.channels;
    const float per = 1.0f / (float)ch;
    float s[1] = {0.0f};
    if (p.residual) {
        const T* e = static_cast<const T*>(p.residual) + at(r, p.length, p.residual_batch, p.residual_token);
        T* sum = static_cast<T*>(p.sum) + at(r, p.length, p.sum_batch, p.sum_token);
        each<T, kVec>(ch, [&](long long c) {
            float f[E], g[E];
            take<T, kVec>(x + c, f);
            take<T, kVec>(e + c, g);
            for (int i = 0; i < E; ++i) {
                f[i] = to_f32(from_f32<T>(f[i] + g[i]));
                s[0] += f[i];
            }
            give<T, kVec>(sum + c, f);
        });
        x = sum;  // each thread reads what it wrote itself
    } else if (!p.rms) {
        each<T, kVec>(ch, [&](long long c) {
            float f[E];
            take<T, kVec>(x + c, f);
            for (int i = 0; i < E; ++i) s[0] += f[i];
        });
    }
    float mean = 0.0f;
    if (!p.rms) {
        cta_sum<1>(s, slot[0]);
        mean = s[0] * per;
    }
    float q[1] = {0.0f};
    each<T, kVec>(ch, [&](long long c) {
        float f[E];
        take<T, kVec>(x + c, f);
        for (int i = 0; i < E; ++i) q[0] = fmaf(f[i] - mean, f[i] - mean, q[0]);
    });
    cta_sum<1>(q, slot[1]);
    const float rstd = inverse_root(fmaf(q[0], per, p.eps));
    if (p.saved && threadIdx.x == 0) reinterpret_cast<float2*>(p.saved)[r] = make_float2(mean, rstd);
    each<T, kVec>(ch, [&](long long c) {
        float f[E];
        take<T, kVec>(x + c, f);
        for (int i = 0; i < E; ++i) {
            const float w = p.weight ? parameter<T>(p.weight, p.params_f32, c + i) : 1.0f;
            const float n = (f[i] - mean) * rstd;
            f[i] = p.bias ? fmaf(n, w, parameter<T>(p.bias, p.params_f32, c + i)) : n * w;
        }
        give<T, kVec>(y + c, f);
    });
}

template <class T, bool kVec>
__global__ void __launch_bounds__(kWideNT) norm_grad_wide_kernel(NormParams p) {
    constexpr int E = kEach<T, kVec>;
    __shared__ __align__(16) float slot[2 * kWideNT / 32];
    const uint32_t r = blockIdx.x;
    const T* x = static_cast<const T*>(p.x) + at(r, p.length, p.x_batch, p.x_token);
    const T* dy = static_cast<const T*>(p.dy) + at(r, p.length, p.dy_batch, p.dy_token);
    const T* ds = p.dsum ? static_cast<const T*>(p.dsum) + at(r, p.length, p.dsum_batch, p.dsum_token) : nullptr;
    T* dx = static_cast<T*>(p.dx) + (long long)r * p.channels;
    const long long ch = p.channels;
    const float2 stat = __ldg(reinterpret_cast<const float2*>(p.saved) + r);
    const float mean = stat.x, rstd = stat.y, per = 1.0f / (float)ch;
    float s[2] = {0.0f, 0.0f};
    each<T, kVec>(ch, [&](long long c) {
        float f[E], g[E];
        take<T, kVec>(x + c, f);
        take<T, kVec>(dy + c, g);
        for (int i = 0; i < E; ++i) {
            const float dn = p.weight ? g[i] * parameter<T>(p.weight, p.params_f32, c + i) : g[i];
            s[0] += dn;
            s[1] = fmaf(dn, (f[i] - mean) * rstd, s[1]);
        }
    });
    cta_sum<2>(s, slot);
    const float a = p.rms ? 0.0f : s[0] * per, b = s[1] * per;
    each<T, kVec>(ch, [&](long long c) {
        float f[E], g[E], h[E];
        take<T, kVec>(x + c, f);
        take<T, kVec>(dy + c, g);
        if (ds) take<T, kVec>(ds + c, h);
        for (int i = 0; i < E; ++i) {
            const float dn = p.weight ? g[i] * parameter<T>(p.weight, p.params_f32, c + i) : g[i];
            f[i] = fmaf(-(f[i] - mean) * rstd, b, dn - a) * rstd;
            if (ds) f[i] += h[i];
        }
        give<T, kVec>(dx + c, f);
    });
}

// Columns' sums over the rows blockIdx.y, + parts, ...: into partials.
constexpr int kColumnNT = 256, kColumnParts = 32;
template <class T>
__global__ void __launch_bounds__(kColumnNT) norm_columns_kernel(NormParams p) {
    const long long c = (long long)blockIdx.x * kColumnNT + threadIdx.x;
    if (c >= p.channels) return;
    float dw = 0.0f, db = 0.0f;
    for (long long row = blockIdx.y; row < p.rows; row += p.parts) {
        const uint32_t r = (uint32_t)row;
        const float g = to_f32(static_cast<const T*>(p.dy)[at(r, p.length, p.dy_batch, p.dy_token) + c]);
        const float2 stat = __ldg(reinterpret_cast<const float2*>(p.saved) + r);
        const float n = (to_f32(static_cast<const T*>(p.x)[at(r, p.length, p.x_batch, p.x_token) + c]) - stat.x) * stat.y;
        dw = fmaf(g, n, dw);
        db += g;
    }
    float* to = p.partials + (long long)blockIdx.y * 2 * p.channels + c;
    to[0] = dw;
    to[p.channels] = db;
}

// ---------------------------------------------------------------- launch
// Shared memory of an SM that its rings share, and of a CTA's ring at most.
constexpr int kRingBytes = 200 * 1024;

template <class T, Way kWay, int kLanes, int NV, bool kGrad, bool kSum>
cudaError_t launch_as(NormParams& p, cudaStream_t s) {
    using G = Team<T, kWay, kLanes, NV>;
    const long long turns = (p.rows + (long long)G::kTeams * G::kRows - 1) / (G::kTeams * G::kRows);
    const int resident = kGrad ? kGradResident<T, kWay, kLanes, NV, kSum> : kResident<T, kWay, kLanes>;
    const int tensors = kGrad ? (kSum ? 3 : 2) : p.residual ? 2 : 1;
    int bytes = kGrad && G::kGroups > 1 ? (int)sizeof(float) * G::NT * G::N : 0;  // the columns' sums
    if (kWay == kRing) {
        const int stage = G::kTeams * tensors * G::kRows * (int)(p.channels * sizeof(T));
        p.stages = std::clamp(kRingBytes / resident / stage, 2, 8);
        bytes = std::max(bytes, p.stages * (stage + G::kTeams * 8));
    }
    p.parts = std::min(turns, seq_sms() * resident);
    const void* kernel;
    if constexpr (kGrad) kernel = (const void*)norm_grad_kernel<T, kWay, kLanes, NV, kSum>;
    else kernel = (const void*)norm_kernel<T, kWay, kLanes, NV>;
    // the limit is one per device: always the largest, whatever this call needs
    if (bytes > kDefaultShared) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes + 8192);
        if (e != cudaSuccess) return e;
    }
    void* args[] = {&p};
    return cudaLaunchKernel(kernel, dim3((unsigned)p.parts), dim3(G::NT), args, (size_t)bytes, s);
}
template <class T, Way kWay, int kLanes, int NV>
cudaError_t go(NormParams& p, bool grad, cudaStream_t s) {
    if (!grad) return launch_as<T, kWay, kLanes, NV, false, false>(p, s);
    return p.dsum ? launch_as<T, kWay, kLanes, NV, true, true>(p, s) : launch_as<T, kWay, kLanes, NV, true, false>(p, s);
}

// Through the ring where CTAs have several turns to take.
template <class T, int kLanes, int NV>
cudaError_t vectors(NormParams& p, bool grad, cudaStream_t s) {
    using G = Team<T, kVectors, kLanes, NV>;
    const int resident = !grad    ? kResident<T, kVectors, kLanes>
                         : p.dsum ? kGradResident<T, kVectors, kLanes, NV, true>
                                  : kGradResident<T, kVectors, kLanes, NV, false>;
    const long long held = seq_sms() * resident * G::kTeams * G::kRows;
    if (p.rows <= held) return go<T, kVectors, kLanes, NV>(p, grad, s);
    return go<T, kRing, kLanes, NV>(p, grad, s);
}

// Rows that are not aligned to 16 bytes; 16-bit elements 8 a thread (with 16 the gradient's
// rows do not fit the registers).
template <class T, Way kWay>
cudaError_t narrow(NormParams& p, long long n, bool grad, cudaStream_t s) {
    if constexpr (sizeof(T) == 4 && kWay == kElements) {
        return cudaErrorInvalidValue;
    } else {
        constexpr int NV = sizeof(T) == 4 ? 2 : 1;
        if (n <= 8) return go<T, kWay, 8, 1>(p, grad, s);
        if (n <= 16) return go<T, kWay, 16, 1>(p, grad, s);
        if (n <= 32) return go<T, kWay, 32, 1>(p, grad, s);
        if (n <= 32 * NV) return go<T, kWay, 32, NV>(p, grad, s);
        if (n <= 64 * NV) return go<T, kWay, 64, NV>(p, grad, s);
        if (n <= 128 * NV) return go<T, kWay, 128, NV>(p, grad, s);
        if (n <= 256 * NV) return go<T, kWay, 256, NV>(p, grad, s);
        if (n <= 512 * NV) return go<T, kWay, 512, NV>(p, grad, s);
        return go<T, kWay, 1024, NV>(p, grad, s);
    }
}

template <class T>
cudaError_t by_width(NormParams& p, bool grad, cudaStream_t s) {
    const long long n = (p.channels + kWidth<T> - 1) / kWidth<T>;
    if (!p.vec) return sizeof(T) == 4 || p.pairs ? narrow<T, kUnits>(p, n, grad, s) : narrow<T, kElements>(p, n, grad, s);
    if (n <= 8) return vectors<T, 8, 1>(p, grad, s);
    if (n <= 16) return vectors<T, 16, 1>(p, grad, s);
    if (n <= 32) return vectors<T, 32, 1>(p, grad, s);
    if (n <= 64) return vectors<T, 32, 2>(p, grad, s);
    if (n <= 128) return vectors<T, 64, 2>(p, grad, s);
    if (n <= 256) return vectors<T, 128, 2>(p, grad, s);
    if (n <= 512) return vectors<T, 256, 2>(p, grad, s);
    if (n <= 1024) return vectors<T, 512, 2>(p, grad, s);
    if constexpr (sizeof(T) == 4) return vectors<T, 1024, 2>(p, grad, s);
    return cudaErrorInvalidValue;
}

template <class T>
cudaError_t launch_norm_as(NormParams& p, bool grad, cudaStream_t s) {
    if (p.channels <= kRowMax) {
        const cudaError_t e = by_width<T>(p, grad, s);
        count_launches(1);
        return e;
    }
    if (!grad) {
        if (p.vec) norm_wide_kernel<T, true><<<p.rows, kWideNT, 0, s>>>(p);
        else norm_wide_kernel<T, false><<<p.rows, kWideNT, 0, s>>>(p);
        count_launches(1);
        return cudaGetLastError();
    }
    if (p.vec) norm_grad_wide_kernel<T, true><<<p.rows, kWideNT, 0, s>>>(p);
    else norm_grad_wide_kernel<T, false><<<p.rows, kWideNT, 0, s>>>(p);
    count_launches(1);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !p.partials) return e;
    p.parts = std::min<long long>(p.rows, kColumnParts);
    const dim3 grid((unsigned)((p.channels + kColumnNT - 1) / kColumnNT), (unsigned)p.parts);
    norm_columns_kernel<T><<<grid, kColumnNT, 0, s>>>(p);
    count_launches(1);
    return cudaGetLastError();
}

}  // namespace

// By element type, one translation unit each.
cudaError_t launch_norm_f32(NormParams& p, bool grad, cudaStream_t s);
cudaError_t launch_norm_f16(NormParams& p, bool grad, cudaStream_t s);
cudaError_t launch_norm_bf16(NormParams& p, bool grad, cudaStream_t s);

}  // namespace scg
