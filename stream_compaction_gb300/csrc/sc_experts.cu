// Tokens to their experts and back: the stable sort of the entries (token, choice) by
// expert, rows moved into that order and summed back with weights, and the gradients.
//
// The sort is one counting pass, since there is one digit: the expert.  One cluster of
// up to 16 CTAs, without scratch memory:
//   count   a warp counts its run of consecutive entries by expert (shared memory);
//   scan    per expert over the CTA's warps, over the CTAs (distributed shared
//           memory), then over the experts;
//   place   a warp goes through its run again, 32 entries at a time: an entry's row is
//           its expert's start + those before it in other warps and rounds + the lanes
//           below with the same expert.
// Entries of no expert are one more bin behind the others, so order and place are
// permutations and every row of an output has exactly one writer.
//
// The rows: bytes alone.  All kernels go by tokens, through place: a token's row is read
// (or written) once, and its entries' rows wherever they lie.  No atomics; a token's sum
// goes in the order of its choices.  16384 tokens, 2 of 64 experts, rows of 4096 bfloat16:
// sort 11 us, rows there 57, back 62, their gradients 61 and 100 (6.5 to 7 TB/s).
#include <algorithm>

#include <cooperative_groups.h>

#include "sc_bulk.cuh"
#include "sc_cluster.h"
#include "sc_seq.cuh"
#include "sc_seq_launch.h"

namespace scg {

namespace {

namespace cg = cooperative_groups;

// ------------------------------------------------------------------ sort
constexpr int kSortMaxWarps = 32, kSortMaxCtas = 16;
constexpr int kRounds = 4;  // of 32 entries, loaded together
constexpr int kMaxBins = SC_EXPERT_MAX + 1;

struct SortParams {
    const void* ids;
    int ids64, experts, bits;  // bits: of a bin, and of the number behind the last
    long long entries, run;    // of a warp, a multiple of 32
    int32_t *order, *place;
    int64_t* offsets;
};

// The lanes whose bin equals this one's, by one ballot a bit: a match instruction takes
// about 60 cycles of a unit that the SM has once, whatever the number of bins (262144
// entries of 512 experts: 65 us with it).
__device__ __forceinline__ uint32_t same_bin(int bin, int bits) {
    uint32_t same = 0xffffffffu;
    for (int b = 0; b < bits; ++b) {
        const uint32_t bit = (uint32_t)bin >> b & 1u, on = __ballot_sync(0xffffffffu, bit);
        same &= on ^ (bit - 1u);
    }
    return same;
}

__device__ __forceinline__ int bin_of(const SortParams& p, long long i) {
    const long long id = p.ids64 ? __ldg(static_cast<const long long*>(p.ids) + i)
                                 : (long long)__ldg(static_cast<const int*>(p.ids) + i);
    return id >= 0 && id < p.experts ? (int)id : p.experts;
}

// Shared memory: [warps][bins] counts, then starts.
__global__ void __launch_bounds__(32 * kSortMaxWarps) expert_sort_kernel(SortParams p) {
    extern __shared__ uint32_t s_count[];
    __shared__ uint32_t s_total[kMaxBins], s_before[kMaxBins], s_all[kMaxBins], s_warp[kSortMaxWarps];
    const cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank(), ranks = (int)cluster.num_blocks();
    const int threads = blockDim.x, warps = threads / 32, tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int bins = p.experts + 1;
    uint32_t* mine = s_count + warp * bins;
    for (int d = lane; d < bins; d += 32) mine[d] = 0u;
    __syncwarp();
    const long long first = ((long long)rank * warps + warp) * p.run, last = min(p.entries, first + p.run);
    for (long long i0 = first; i0 < last; i0 += 32 * kRounds) {
        int d[kRounds];
#pragma unroll
        for (int r = 0; r < kRounds; ++r) {
            const long long i = i0 + r * 32 + lane;
            d[r] = i < last ? bin_of(p, i) : -1;
        }
#pragma unroll
        for (int r = 0; r < kRounds; ++r)
            if (d[r] >= 0) atomicAdd(&mine[d[r]], 1u);
    }
    __syncthreads();
    // per bin: the entries of earlier warps, and the CTA's
    for (int d = tid; d < bins; d += threads) {
        uint32_t sum = 0;
        for (int w0 = 0; w0 < warps; w0 += 8) {
            uint32_t c[8];
#pragma unroll
            for (int w = 0; w < 8; ++w) c[w] = w0 + w < warps ? s_count[(w0 + w) * bins + d] : 0u;
#pragma unroll
            for (int w = 0; w < 8; ++w) {
                if (w0 + w < warps) s_count[(w0 + w) * bins + d] = sum;
                sum += c[w];
            }
        }
        s_total[d] = sum;
    }
    cluster.sync();
    // per bin: the entries in earlier CTAs, and in all
    for (int d = tid; d < bins; d += threads) {
        uint32_t before = 0, all = 0;
        for (int r = 0; r < ranks; ++r) {
            const uint32_t c = *cluster.map_shared_rank(&s_total[d], r);
            if (r < rank) before += c;
            all += c;
        }
        s_before[d] = before;
        s_all[d] = all;
    }
    cluster.sync();  // nobody reads totals any more
    // a thread's bins, side by side, over the threads
    const int per = (bins + threads - 1) / threads, d0 = min(bins, tid * per), d1 = min(bins, d0 + per);
    uint32_t sum = 0;
    for (int d = d0; d < d1; ++d) sum += s_all[d];
    uint32_t incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) s_warp[warp] = incl;
    __syncthreads();
    uint32_t start = incl - sum;
    for (int w = 0; w < warp; ++w) start += s_warp[w];
    for (int d = d0; d < d1; ++d) {
        s_total[d] = start + s_before[d];
        if (rank == 0) p.offsets[d] = start;
        start += s_all[d];
    }
    __syncthreads();
    for (int d = lane; d < bins; d += 32) mine[d] += s_total[d];
    __syncwarp();
    for (long long i0 = first; i0 < last; i0 += 32 * kRounds) {
        int d[kRounds];
#pragma unroll
        for (int r = 0; r < kRounds; ++r) {
            const long long i = i0 + r * 32 + lane;
            d[r] = i < last ? bin_of(p, i) : bins;
        }
        uint32_t same_[kRounds];
#pragma unroll
        for (int r = 0; r < kRounds; ++r) same_[r] = same_bin(d[r], p.bits);
#pragma unroll
        for (int r = 0; r < kRounds; ++r) {
            const uint32_t same = same_[r];
            const bool live = d[r] < bins;
            const uint32_t begin = live ? mine[d[r]] : 0u;
            __syncwarp();
            if (live) {
                const uint32_t row = begin + __popc(same & ((1u << lane) - 1u));
                const long long i = i0 + r * 32 + lane;
                p.place[i] = (int32_t)row;
                p.order[row] = (int32_t)i;
                if (lane == __ffs(same) - 1) mine[d[r]] = begin + __popc(same);
            }
            __syncwarp();
        }
    }
}

// ------------------------------------------------------------------ rows
constexpr int kNT = 256;

// A lane's elements of a row in one access: the widest of 16, 4 and (16-bit elements) 2
// bytes that every row is aligned to.  kAhead: the entries of a token that are loaded
// together, 2 or 4; kColumns: the accesses of a row that are, more where they are narrow.
template <class T, int kBytes, int kAhead_>
struct Part {
    static constexpr int W = kBytes / (int)sizeof(T), kAhead = kAhead_;
    static constexpr int kColumns = (kBytes == 16 ? 4 : 16) / kAhead;
    using Narrow = typename std::conditional<kBytes == 4, uint32_t, unsigned short>::type;
    using U = typename std::conditional<kBytes == 16, uint4, Narrow>::type;
    U v;
    __device__ __forceinline__ void load(const T* p) { v = __ldg(reinterpret_cast<const U*>(p)); }
    __device__ __forceinline__ void store(T* p) const { *reinterpret_cast<U*>(p) = v; }
    __device__ __forceinline__ void zero() { memset(&v, 0, sizeof(v)); }
    __device__ __forceinline__ void get(float (&f)[W]) const {
        if constexpr (kBytes == 16) {
            Vec<T, W> r;
            memcpy(r.w, &v, 16);
#pragma unroll
            for (int i = 0; i < W; ++i) f[i] = r.get(i);
        } else {
            T e[W];
            memcpy(e, &v, sizeof(v));
#pragma unroll
            for (int i = 0; i < W; ++i) f[i] = to_f32(e[i]);
        }
    }
    __device__ __forceinline__ void set(const float (&f)[W]) {
        if constexpr (kBytes == 16) {
            Vec<T, W> r;
            r.set(f);
            memcpy(&v, r.w, 16);
        } else {
            T e[W];
#pragma unroll
            for (int i = 0; i < W; ++i) e[i] = from_f32<T>(f[i]);
            memcpy(&v, e, sizeof(v));
        }
    }
};

// `lanes` threads a token, the token's group within the CTA; the CTAs of a column of the
// grid share a token's row.
struct Where {
    long long token;
    int lane;
};
__device__ __forceinline__ Where where(int lanes) {
    const int group = threadIdx.x / lanes;
    return {(long long)blockIdx.x * (kNT / lanes) + group, (int)threadIdx.x - group * lanes};
}
// Entries that have an expert; their rows come first.
__device__ __forceinline__ long long kept_of(const ExpertParams& p) {
    return min((long long)__ldg(reinterpret_cast<const long long*>(p.kept)), p.entries);
}
template <class T>
__device__ __forceinline__ float weight_of(const ExpertParams& p, long long entry) {
    if (!p.weights) return 1.0f;
    return p.weights_f32 ? __ldg(static_cast<const float*>(p.weights) + entry)
                         : to_f32(__ldg(static_cast<const T*>(p.weights) + entry));
}
// The row of an entry; -1: passed over.
__device__ __forceinline__ long long row_of(const ExpertParams& p, long long entry) {
    const long long row = __ldg(p.place + entry);
    return row < p.entries ? row : -1;
}

template <class T, class P>
__global__ void __launch_bounds__(kNT) expert_gather_kernel(ExpertParams p, int lanes) {
    const Where at = where(lanes);
    if (at.token >= p.tokens) return;
    const long long kept = kept_of(p);
    const T* x = static_cast<const T*>(p.in) + at.token * p.ld_in;
    const int step = lanes * P::W;
    const long long stride = (long long)step * P::kColumns;
    for (long long c0 = blockIdx.y * stride + at.lane * P::W; c0 < p.dim; c0 += gridDim.y * stride) {
        P v[P::kColumns], none;
        none.zero();
#pragma unroll
        for (int k = 0; k < P::kColumns; ++k)
            if (c0 + k * step < p.dim) v[k].load(x + c0 + k * step);
        for (long long j = 0; j < p.choices; ++j) {
            const long long row = row_of(p, at.token * p.choices + j);
            if (row < 0) continue;
            T* to = static_cast<T*>(p.out) + row * p.ld_out + c0;
#pragma unroll
            for (int k = 0; k < P::kColumns; ++k)
                if (c0 + k * step < p.dim) (row < kept ? v[k] : none).store(to + k * step);
        }
    }
}

// out[t] = sum over j of weights[t,j] rows[place[t,j]].  64 registers a thread, for four CTAs
// an SM (8000 tokens, 2 of 2047 float32: 59 us with three, 51 so).
template <class T, class P>
__global__ void __launch_bounds__(kNT, 4) expert_combine_kernel(ExpertParams p, int lanes) {
    constexpr int W = P::W, C = P::kColumns, kAhead = P::kAhead;
    const Where at = where(lanes);
    if (at.token >= p.tokens) return;
    const long long kept = kept_of(p);
    const long long entry = at.token * p.choices;
    const int step = lanes * W;
    const long long stride = (long long)step * C;
    for (long long c0 = blockIdx.y * stride + at.lane * W; c0 < p.dim; c0 += gridDim.y * stride) {
        float sum[C][W];
#pragma unroll
        for (int k = 0; k < C; ++k)
#pragma unroll
            for (int i = 0; i < W; ++i) sum[k][i] = 0.0f;
        for (long long j0 = 0; j0 < p.choices; j0 += kAhead) {
            P v[kAhead][C];
            bool live[kAhead];
#pragma unroll
            for (int a = 0; a < kAhead; ++a) {
                const long long row = j0 + a < p.choices ? row_of(p, entry + j0 + a) : -1;
                live[a] = row >= 0 && row < kept;
                const T* from = static_cast<const T*>(p.in) + row * p.ld_in + c0;
#pragma unroll
                for (int k = 0; k < C; ++k)
                    if (live[a] && c0 + k * step < p.dim) v[a][k].load(from + k * step);
            }
#pragma unroll
            for (int a = 0; a < kAhead; ++a) {
                if (!live[a]) continue;
                const float w = weight_of<T>(p, entry + j0 + a);
#pragma unroll
                for (int k = 0; k < C; ++k) {
                    float f[W];
                    v[a][k].get(f);
#pragma unroll
                    for (int i = 0; i < W; ++i) sum[k][i] = fmaf(w, f[i], sum[k][i]);
                }
            }
        }
        T* to = static_cast<T*>(p.out) + at.token * p.ld_out + c0;
#pragma unroll
        for (int k = 0; k < C; ++k) {
            P o;
            o.set(sum[k]);
            if (c0 + k * step < p.dim) o.store(to + k * step);
        }
    }
}

// drows[place[t,j]] = weights[t,j] dout[t];  dweights[t,j] = dout[t] . rows[place[t,j]]
template <class T, class P>
__global__ void __launch_bounds__(kNT) expert_combine_grad_kernel(ExpertParams p, int lanes) {
    constexpr int W = P::W, C = P::kColumns, kAhead = P::kAhead;
    __shared__ float s_dot[kNT / 32][kAhead];
    const Where at = where(lanes);
    const bool here = at.token < p.tokens;  // all stay for the sums over threads
    const long long kept = kept_of(p), entry = (here ? at.token : 0) * p.choices;
    const T* dout = static_cast<const T*>(p.in) + (here ? at.token : 0) * p.ld_in;
    const T* rows = static_cast<const T*>(p.rows);
    const int step = lanes * W;
    for (long long j0 = 0; j0 < p.choices; j0 += kAhead) {
        long long row[kAhead];
        float w[kAhead], dot[kAhead];
#pragma unroll
        for (int a = 0; a < kAhead; ++a) {
            row[a] = here && j0 + a < p.choices ? row_of(p, entry + j0 + a) : -1;
            dot[a] = 0.0f;
        }
#pragma unroll
        for (int a = 0; a < kAhead; ++a) w[a] = row[a] >= 0 && row[a] < kept ? weight_of<T>(p, entry + j0 + a) : 0.0f;
        for (long long c0 = (long long)at.lane * W; here && c0 < p.dim; c0 += step * C) {
            P g[C], v[kAhead][C];
#pragma unroll
            for (int k = 0; k < C; ++k) {
                if (c0 + k * step >= p.dim) break;
                g[k].load(dout + c0 + k * step);
#pragma unroll
                for (int a = 0; a < kAhead; ++a)
                    if (rows && row[a] >= 0 && row[a] < kept) v[a][k].load(rows + row[a] * p.ld_rows + c0 + k * step);
            }
#pragma unroll
            for (int k = 0; k < C; ++k) {
                if (c0 + k * step >= p.dim) break;
                float d[W];
                g[k].get(d);
#pragma unroll
                for (int a = 0; a < kAhead; ++a) {
                    if (row[a] < 0) continue;
                    const bool live = row[a] < kept;
                    float f[W];
                    if (rows && live) {
                        v[a][k].get(f);
#pragma unroll
                        for (int i = 0; i < W; ++i) dot[a] = fmaf(d[i], f[i], dot[a]);
                    }
                    P o;
#pragma unroll
                    for (int i = 0; i < W; ++i) f[i] = w[a] * d[i];
                    o.set(f);
                    if (!live) o.zero();
                    o.store(static_cast<T*>(p.out) + row[a] * p.ld_out + c0 + k * step);
                }
            }
        }
        if (!p.dweights) continue;
        for (int o = 1; o < min(lanes, 32); o <<= 1)
#pragma unroll
            for (int a = 0; a < kAhead; ++a) dot[a] += __shfl_xor_sync(0xffffffffu, dot[a], o);
        if (lanes > 32) {
            __syncthreads();  // the sums of the choices before are read
            if (threadIdx.x % 32 == 0) {
#pragma unroll
                for (int a = 0; a < kAhead; ++a) s_dot[threadIdx.x / 32][a] = dot[a];
            }
            __syncthreads();
        }
        if (here && at.lane < kAhead && j0 + at.lane < p.choices) {
            float v = 0.0f;
            if (lanes > 32) {
                const int w0 = ((int)threadIdx.x - at.lane) / 32;
                for (int i = 0; i < lanes / 32; ++i) v += s_dot[w0 + i][at.lane];
            } else {
#pragma unroll
                for (int a = 0; a < kAhead; ++a)
                    if (a == at.lane) v = dot[a];
            }
            const long long e = entry + j0 + at.lane;
            if (p.weights_f32) static_cast<float*>(p.dweights)[e] = v;
            else static_cast<T*>(p.dweights)[e] = from_f32<T>(v);
        }
    }
}

// ------------------------------------------------- rows through a ring
// The two kernels that read a token's entries' rows from wherever they lie, for aligned
// rows: CTAs stay and teams of 32 to 256 threads take tokens in turns; the rows of the
// next ones are under way, one bulk copy each, into a ring of stages in shared memory.
// A stage: (the gradient: the token's row of dout,) the rows of its entries that have an
// expert, and for each entry its row's number and its weight.
struct Entry {
    int row;  // of the sorted order; -1: passed over
    float weight;
};
constexpr int kMaxChoices = 32;  // a lane of the filling warp each

struct TeamRing {
    unsigned char* stage0;
    uint32_t bar, row_bytes, stage_bytes, phase = 0;
    int stages, fill = 0, take = 0;
    long long kept;
    // of the token to fill next, loaded a turn ahead: this lane's entry
    int row = -1;
    float weight = 0.0f;

    template <class T>
    __device__ __forceinline__ void peek(const ExpertParams& p, long long token, int lane) {
        row = -1;
        weight = 0.0f;
        if (token >= p.tokens || lane >= p.choices) return;
        const long long r = __ldg(p.place + token * p.choices + lane);
        row = r >= 0 && r < p.entries ? (int)r : -1;
        weight = weight_of<T>(p, token * p.choices + lane);
    }
    __device__ __forceinline__ Entry* entries(int stage) const {
        return reinterpret_cast<Entry*>(stage0 + (size_t)stage * stage_bytes);
    }
    __device__ __forceinline__ unsigned char* rows(int stage) const {
        return stage0 + (size_t)stage * stage_bytes + sizeof(Entry) * kMaxChoices;
    }
    // The token's rows into the next stage, by the team's first warp.
    template <class T, bool kGrad>
    __device__ __forceinline__ void load(const ExpertParams& p, long long token, int lane) {
        const uint32_t full = bar + 8 * fill;
        const bool live = row >= 0 && row < kept && (!kGrad || p.rows);
        if (lane < p.choices) entries(fill)[lane] = {row, weight};
        const int copies = __popc(__ballot_sync(0xffffffffu, live)) + (kGrad ? 1 : 0);  // after the entries are written
        __syncwarp();
        if (lane == 0) mbar_arrive_expect_tx(full, copies * row_bytes);
        const uint32_t to = smem_u32(rows(fill));
        const T* from = static_cast<const T*>(kGrad ? p.rows : p.in);
        if (live)
            bulk_load(to + (lane + (kGrad ? 1 : 0)) * row_bytes, from + row * (kGrad ? p.ld_rows : p.ld_in), row_bytes, full);
        if (kGrad && lane == 0) bulk_load(to, static_cast<const T*>(p.in) + token * p.ld_in, row_bytes, full);
        if (++fill == stages) fill = 0;
    }
    __device__ __forceinline__ bool wait() const { return arrived(bar + 8 * take, phase); }
    __device__ __forceinline__ void taken() {
        if (++take == stages) {
            take = 0;
            phase ^= 1;
        }
    }
};

__device__ __forceinline__ void team_sync(int team, int size) {
    if (size == 32) __syncwarp();
    else asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "r"(size) : "memory");
}

template <class T, bool kGrad>
__global__ void __launch_bounds__(kNT) expert_ring_kernel(ExpertParams p, int size, int stages, uint32_t stage_bytes) {
    extern __shared__ __align__(128) unsigned char s_mem[];
    __shared__ float s_dot[kNT / 32][kMaxChoices];
    constexpr int W = 16 / (int)sizeof(T);
    using P = Part<T, 16, 4>;
    const int teams = kNT / size, team = threadIdx.x / size, thread = threadIdx.x - team * size, lane = threadIdx.x % 32;
    const int choices = (int)p.choices;
    const long long step = (long long)gridDim.x * teams;
    long long token = (long long)blockIdx.x * teams + team, ahead = token;
    TeamRing ring;
    ring.stage0 = s_mem + (size_t)team * stages * stage_bytes;
    ring.bar = smem_u32(s_mem + (size_t)teams * stages * stage_bytes + team * stages * 8);
    ring.row_bytes = (uint32_t)(p.dim * sizeof(T));
    ring.stage_bytes = stage_bytes;
    ring.stages = stages;
    ring.kept = kept_of(p);
    if (thread == 0) {
        for (int i = 0; i < stages; ++i) mbar_init(ring.bar + 8 * i, 1);
        fence_mbar_init();
    }
    __syncthreads();
    auto fetch = [&] {  // the first warp of the team
        if (ahead < p.tokens) ring.load<T, kGrad>(p, ahead, lane);
        ahead += step;
        ring.peek<T>(p, ahead, lane);
    };
    if (thread < 32) {
        ring.peek<T>(p, ahead, lane);
        for (int i = 0; i < stages; ++i) fetch();
    }
    for (; token < p.tokens; token += step) {
        const bool ok = ring.wait();
        const Entry* entry = ring.entries(ring.take);
        const T* rows = reinterpret_cast<const T*>(ring.rows(ring.take));
        if constexpr (!kGrad) {
            for (long long c = (long long)thread * W; c < p.dim; c += size * W) {
                float sum[W];
#pragma unroll
                for (int i = 0; i < W; ++i) sum[i] = ok ? 0.0f : not_a_number();
#pragma unroll 4
                for (int j = 0; j < choices; ++j) {
                    const Entry e = entry[j];
                    if (e.row < 0 || e.row >= ring.kept) continue;
                    Vec<T, W> v;
                    v.load_rw(rows + j * p.dim + c);
#pragma unroll
                    for (int i = 0; i < W; ++i) sum[i] = fmaf(e.weight, v.get(i), sum[i]);
                }
                P o;
                o.set(sum);
                o.store(static_cast<T*>(p.out) + token * p.ld_out + c);
            }
        } else {
            for (int j = 0; j < choices; ++j) {
                const Entry e = entry[j];
                const bool live = e.row >= 0 && e.row < ring.kept;
                float dot = 0.0f;
                if (e.row >= 0) {
                    T* to = static_cast<T*>(p.out) + e.row * p.ld_out;
#pragma unroll 2
                    for (long long c = (long long)thread * W; c < p.dim; c += size * W) {
                        Vec<T, W> g, v;
                        P o;
                        o.zero();
                        if (live) {
                            g.load_rw(rows + c);
                            if (p.rows) {
                                v.load_rw(rows + (j + 1) * p.dim + c);
#pragma unroll
                                for (int i = 0; i < W; ++i) dot = fmaf(g.get(i), v.get(i), dot);
                            }
                            float f[W];
                            const float w = ok ? e.weight : not_a_number();
#pragma unroll
                            for (int i = 0; i < W; ++i) f[i] = w * g.get(i);
                            o.set(f);
                        }
                        o.store(to + c);
                    }
                }
                if (p.dweights) {
#pragma unroll
                    for (int o = 1; o < 32; o <<= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
                    if (lane == 0) s_dot[threadIdx.x / 32][j] = ok ? dot : not_a_number();
                }
            }
        }
        team_sync(team, size);  // the stage is read, and the parts of the products are there
        if (kGrad && p.dweights && thread < choices) {
            float v = 0.0f;
            for (int w = 0; w < size / 32; ++w) v += s_dot[team * (size / 32) + w][thread];
            const long long at = token * p.choices + thread;
            if (p.weights_f32) static_cast<float*>(p.dweights)[at] = v;
            else static_cast<T*>(p.dweights)[at] = from_f32<T>(v);
        }
        ring.taken();
        if (thread < 32) fetch();
        if (kGrad && p.dweights) team_sync(team, size);  // the parts are read
    }
}

// Threads a token: a Part's columns each, up to a whole CTA.
template <class P>
int lanes_of(long long dim) {
    const long long n = (dim + P::W * P::kColumns - 1) / (P::W * P::kColumns);
    int lanes = 8;
    while (lanes < kNT && lanes < n) lanes *= 2;
    return lanes;
}
enum { kGather, kCombine, kCombineGrad };

// Through a ring where CTAs have several turns and two stages fit a team's share of the
// shared memory; and where a token has few entries: with four or more a lane's direct
// loads are as much under way, without a stage of that many rows (16384 tokens with 8
// entries of 4096 bfloat16: gradient 608 us through the ring, 348 directly, sum 275 and
// 211; 32768 with 8 of 512: gradient 152 and 111, sum 59 and 68).
template <class T, bool kGrad>
bool ring_as(const ExpertParams& p, cudaStream_t s, cudaError_t* e) {
    constexpr int kShared = 200 * 1024;
    const long long vectors = p.dim * (long long)sizeof(T) / 16, row = p.dim * (long long)sizeof(T);
    if (p.choices < 1 || p.choices > kMaxChoices || row > kShared) return false;
    if (p.choices > 3 && (kGrad || vectors >= kNT)) return false;
    int size = 32;
    while (size < kNT && size < vectors) size *= 2;
    const int teams = kNT / size;
    const long long stage = (sizeof(Entry) * kMaxChoices + (p.choices + (kGrad ? 1 : 0)) * row + 127) / 128 * 128;
    int resident = 4;
    while (resident > 1 && stage * teams * 2 > kShared / resident) --resident;
    const int stages = (int)std::min<long long>(kShared / resident / (stage * teams), 8);
    if (stages < 2 || p.tokens <= seq_sms() * resident * teams) return false;
    const int bytes = stages * teams * ((int)stage + 8);
    auto kernel = expert_ring_kernel<T, kGrad>;
    // the limit is one per device: always the largest, whatever this call needs
    *e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kShared + 1024);
    if (*e != cudaSuccess) return true;
    const unsigned grid = (unsigned)std::min<long long>((p.tokens + teams - 1) / teams, seq_sms() * resident);
    kernel<<<grid, kNT, bytes, s>>>(p, size, stages, (uint32_t)stage);
    count_launches(1);
    *e = cudaGetLastError();
    return true;
}

template <class T, class P>
cudaError_t launch_rows(int what, const ExpertParams& p, cudaStream_t s) {
    const int lanes = lanes_of<P>(p.dim);
    const unsigned grid = (unsigned)((p.tokens + kNT / lanes - 1) / (kNT / lanes));
    // rows of more than one turn are shared where there are few tokens for the machine
    const long long turns = (p.dim + (long long)lanes * P::W * P::kColumns - 1) / ((long long)lanes * P::W * P::kColumns);
    const dim3 shared(grid, (unsigned)std::min<long long>(turns, 1 + 4 * seq_sms() / grid));
    if (what == kGather) expert_gather_kernel<T, P><<<shared, kNT, 0, s>>>(p, lanes);
    else if (what == kCombine) expert_combine_kernel<T, P><<<shared, kNT, 0, s>>>(p, lanes);
    else expert_combine_grad_kernel<T, P><<<grid, kNT, 0, s>>>(p, lanes);
    count_launches(1);
    return cudaGetLastError();
}
template <class T, int kBytes>
cudaError_t rows_as(int what, const ExpertParams& p, cudaStream_t s) {
    return p.choices <= 2 ? launch_rows<T, Part<T, kBytes, 2>>(what, p, s) : launch_rows<T, Part<T, kBytes, 4>>(what, p, s);
}
template <class T>
cudaError_t rows_of(int what, const ExpertParams& p, cudaStream_t s) {
    if (p.vec) {
        cudaError_t e;
        if ((what == kCombine && ring_as<T, false>(p, s, &e)) || (what == kCombineGrad && ring_as<T, true>(p, s, &e))) return e;
        return rows_as<T, 16>(what, p, s);
    }
    if constexpr (sizeof(T) == 2) {
        if (!p.pairs) return rows_as<T, 2>(what, p, s);
    }
    return rows_as<T, 4>(what, p, s);
}
cudaError_t rows(int dtype, int what, const ExpertParams& p, cudaStream_t s) {
    return dtype == SC_F32 ? rows_of<float>(what, p, s) : dtype == SC_F16 ? rows_of<f16>(what, p, s)
                                                                         : rows_of<bf16>(what, p, s);
}

}  // namespace

cudaError_t launch_expert_sort(const void* ids, int ids64, long long entries, int experts, int32_t* order, int32_t* place,
                               int64_t* offsets, cudaStream_t s) {
    // a warp per 32 entries up to 16 CTAs of 32 warps, then longer runs
    const long long least = (entries + 31) / 32;
    int ctas = 1;
    while (ctas < kSortMaxCtas && (long long)ctas * kSortMaxWarps < least) ctas *= 2;
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute a{};
    a.id = cudaLaunchAttributeClusterDimension;
    a.val.clusterDim.y = a.val.clusterDim.z = 1;
    cfg.attrs = &a;
    cfg.numAttrs = 1;
    cfg.stream = s;
    // the limit is one per device: always the whole, whatever this call needs
    constexpr int kShared = kSortMaxWarps * kMaxBins * (int)sizeof(uint32_t);
    cudaError_t e = cudaSuccess;
    auto allow = [&] { return cudaFuncSetAttribute(expert_sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kShared); };
    if (ctas > 8) {
        e = cudaFuncSetAttribute(expert_sort_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e == cudaSuccess) e = allow();
        if (e != cudaSuccess) return e;
        static LargeClusters large;
        a.val.clusterDim.x = (unsigned)ctas;
        cfg.gridDim = dim3((unsigned)ctas);
        cfg.blockDim = dim3(32 * kSortMaxWarps);
        cfg.dynamicSmemBytes = kShared;
        if (!large.fit((const void*)expert_sort_kernel, cfg)) ctas = 8;
    }
    // (a thread has two bins at most where a CTA can have as many threads)
    const long long wanted = std::max<long long>((least + ctas - 1) / ctas, experts / 64 + 1);
    const int warps = (int)std::min<long long>(wanted, kSortMaxWarps);
    SortParams p{ids, ids64, experts, 0, entries, 0, order, place, offsets};
    while (experts + 1 >> p.bits) ++p.bits;
    p.run = ((entries + (long long)ctas * warps - 1) / ((long long)ctas * warps) + 31) / 32 * 32;
    const size_t bytes = (size_t)warps * (experts + 1) * sizeof(uint32_t);
    if (ctas <= 8 && bytes > kDefaultShared - 8 * 1024) {
        e = allow();
        if (e != cudaSuccess) return e;
    }
    a.val.clusterDim.x = (unsigned)ctas;
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(32 * warps);
    cfg.dynamicSmemBytes = bytes;
    e = cudaLaunchKernelEx(&cfg, expert_sort_kernel, p);
    count_launches(1);
    return e;
}

cudaError_t launch_expert_gather(int dtype, const ExpertParams& p, cudaStream_t s) { return rows(dtype, kGather, p, s); }
cudaError_t launch_expert_combine(int dtype, const ExpertParams& p, cudaStream_t s) { return rows(dtype, kCombine, p, s); }
cudaError_t launch_expert_combine_grad(int dtype, const ExpertParams& p, cudaStream_t s) {
    return rows(dtype, kCombineGrad, p, s);
}

}  // namespace scg
