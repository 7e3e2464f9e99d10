// Token embedding, out[t] = scale * weight[ids[t]], and its gradient
// dweight[v] = scale * sum of dout[t] over ids[t] == v.
//
// Both move rows and compute next to nothing: the floor is their bytes.  The
// gradient writes each row of dweight once and reads each row of dout once:
//
//   sort       the (id, t) pairs by id, stable, least significant digit first,
//              at most 10 bits a pass (so two passes below 2^20 ids).  Up to
//              kClusterKeys tokens: one launch, one cluster of up to 8 CTAs whose
//              digit counts meet in distributed shared memory (16384 tokens:
//              18 us against 38 us of the four launches below).  Beyond: per
//              tile digit counts, their sums over tiles, the placement.  Then
//              where each id's run starts and ends.
//   long runs  tokens of one id may be a large part of all (padding, a frequent
//              word): runs longer than kRun are cut at multiples of kRun of the
//              sorted order and each piece summed by a CTA of its own;
//   rows       each CTA takes up to kRowsPerCta rows of dweight: first it writes the
//              zeros of those without a token, which wait for nothing, then the
//              sums of at most kRun rows of dout, or of the row's pieces.
// 16384 tokens of 4096 bfloat16 in a table of 131072: the lookup 44 us (6.1 TB/s),
// the gradient 214: sort 18, long runs 16, rows 180 (1.2 GB, 6.7 TB/s); 5003 tokens
// of 1000 float32 in 50021: 12, 10 and 38 us.  The rows begun while the long runs are
// summed (a programmatic launch): 301 us for all of the first case, 266 one after the
// other.  kRun 64 or 128 leaves a CTA's one
// frequent id to the end of the launch (94 us for all of the second case, 79 so).
//
// Sums are float32 in a fixed order, so a result is the same on every run, whatever
// the schedule (no atomics on values): a short run in the order of t, a long one piece
// by piece (with few columns a piece's rows in shares of their own, then the shares).
// Pieces are cut by position in the sorted order, so the rounding of a long run also
// depends on how many tokens smaller ids have.
#include <algorithm>

#include <cooperative_groups.h>

#include "sc_seq.cuh"
#include "sc_seq_launch.h"

namespace scg {

namespace {

constexpr int kNT = 256;
constexpr int kSortKeys = 8;                    // keys per thread of a sort tile
constexpr int kSortTile = kNT * kSortKeys;      // 2048
constexpr int kSortWarps = kNT / 32;
constexpr int kMaxDigit = 1024;
constexpr int kClusterNT = 1024, kClusterWarps = kClusterNT / 32, kClusterCtas = 8;
constexpr long long kClusterKeys = 8ll * kClusterNT * kClusterCtas;  // 8 a thread: 65536
// A launch asks for its digits' share of this.  The kernels' limit is always the
// whole: it is one per device, and another host thread's call between a call's own
// limit and its launch would have the launch refused.
constexpr int kClusterShared = kClusterWarps * kMaxDigit * 2;
constexpr int kRun = 32;
constexpr int kRowsPerCta = 32;

__device__ __forceinline__ long long load_id(const void* ids, int ids64, long long i) {
    return ids64 ? __ldg(static_cast<const long long*>(ids) + i) : (long long)__ldg(static_cast<const int*>(ids) + i);
}

// ---------------------------------------------------------------- lookup
template <class T, bool kVec>
__global__ void __launch_bounds__(kNT) embed_kernel(EmbedParams p, int tpr) {
    constexpr int W = 16 / sizeof(T);
    const int sub = threadIdx.x / tpr, lane = threadIdx.x % tpr;
    const long long t = (long long)blockIdx.x * (kNT / tpr) + sub;
    if (t >= p.tokens) return;
    const long long id = load_id(p.ids, p.ids64, t);
    const bool ok = id >= 0 && id < p.vocab;
    const T* src = static_cast<const T*>(p.weight) + (ok ? id : 0) * p.ldw;
    T* dst = static_cast<T*>(p.out) + t * p.ldo;
    const long long col0 = (long long)blockIdx.y * tpr * W;
    if constexpr (kVec) {
        const long long c = col0 + (long long)lane * W;
        if (c >= p.dim) return;
        Vec<T, W> v;
        if (ok) v.load(src + c);
        float f[W];
#pragma unroll
        for (int i = 0; i < W; ++i) f[i] = ok ? v.get(i) * p.scale : 0.0f;
        v.set(f);
        v.store(dst + c);
    } else {
#pragma unroll
        for (int i = 0; i < W; ++i) {
            const long long c = col0 + (long long)i * tpr + lane;
            if (c < p.dim) dst[c] = from_f32<T>(ok ? to_f32(src[c]) * p.scale : 0.0f);
        }
    }
}

// ------------------------------------------------------------------ sort
// Key i of a pass: on the first pass the id itself, ids outside [0, vocab) as
// `vocab`, behind every row.
__device__ __forceinline__ uint32_t sort_key(const EmbedParams& p, const uint32_t* keys, long long i) {
    if (keys) return keys[i];
    const long long id = load_id(p.ids, p.ids64, i);
    return id >= 0 && id < p.vocab ? (uint32_t)id : (uint32_t)p.vocab;
}

// counts[tile][digit]
__global__ void __launch_bounds__(kNT) sort_count_kernel(EmbedParams p, const uint32_t* keys, int shift, int bits,
                                                         uint32_t* counts) {
    __shared__ uint32_t h[kMaxDigit];
    const int digits = 1 << bits;
    for (int d = threadIdx.x; d < digits; d += kNT) h[d] = 0u;
    __syncthreads();
    const long long t0 = (long long)blockIdx.x * kSortTile;
#pragma unroll
    for (int j = 0; j < kSortKeys; ++j) {
        const long long i = t0 + j * kNT + threadIdx.x;
        if (i < p.tokens) atomicAdd(&h[(sort_key(p, keys, i) >> shift) & (digits - 1)], 1u);
    }
    __syncthreads();
    for (int d = threadIdx.x; d < digits; d += kNT) counts[(long long)blockIdx.x * digits + d] = h[d];
}

// counts[tile][digit] -> the digit's count in the tiles before; row `tiles`: totals.
__global__ void __launch_bounds__(kNT) sort_columns_kernel(uint32_t* counts, long long tiles, int digits) {
    const int d = blockIdx.x * kNT + threadIdx.x;
    if (d >= digits) return;
    uint32_t sum = 0;
    long long t = 0;
    for (; t + 8 <= tiles; t += 8) {
        uint32_t c[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) c[j] = counts[(t + j) * digits + d];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            counts[(t + j) * digits + d] = sum;
            sum += c[j];
        }
    }
    for (; t < tiles; ++t) {
        const uint32_t c = counts[t * digits + d];
        counts[t * digits + d] = sum;
        sum += c;
    }
    counts[tiles * digits + d] = sum;
}

// Stable placement of one tile: the warps rank their keys (a warp has 256
// consecutive keys, 32 at a time in order) with running counts per warp and
// digit; a key goes to (keys of smaller digits) + (its digit's keys in earlier
// tiles) + (in earlier warps) + its rank.
__global__ void __launch_bounds__(kNT) sort_place_kernel(EmbedParams p, const uint32_t* keys, const uint32_t* vals,
                                                         int shift, int bits, const uint32_t* counts, long long tiles,
                                                         uint32_t* keys_out, uint32_t* vals_out) {
    __shared__ uint32_t s_cnt[kSortWarps][kMaxDigit];
    __shared__ uint32_t s_warp[kSortWarps];
    constexpr int kPer = kMaxDigit / kNT;
    const int digits = 1 << bits, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    for (int i = tid; i < kSortWarps * kMaxDigit; i += kNT) (&s_cnt[0][0])[i] = 0u;
    __syncthreads();
    const long long base = (long long)blockIdx.x * kSortTile + warp * (32 * kSortKeys);
    uint32_t key[kSortKeys], rank[kSortKeys];
#pragma unroll
    for (int j = 0; j < kSortKeys; ++j) {
        const long long i = base + j * 32 + lane;
        key[j] = i < p.tokens ? sort_key(p, keys, i) : 0u;
    }
#pragma unroll
    for (int j = 0; j < kSortKeys; ++j) {
        const bool live = base + j * 32 + lane < p.tokens;
        const uint32_t d = (key[j] >> shift) & (uint32_t)(digits - 1);
        // lanes past the end match nobody's digit
        const uint32_t m = __match_any_sync(0xffffffffu, live ? d : 0xffffffffu);
        const uint32_t before = live ? s_cnt[warp][d] : 0u;
        __syncwarp();
        rank[j] = before + __popc(m & ((1u << lane) - 1u));
        if (live && lane == __ffs(m) - 1) s_cnt[warp][d] = before + __popc(m);
        __syncwarp();
    }
    __syncthreads();
    // thread tid: digits kPer * tid ..: keys of its digits in earlier tiles, and in all
    uint32_t prev[kPer], total[kPer], sum = 0;
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
        const int d = kPer * tid + q;
        prev[q] = total[q] = 0u;
        if (d < digits) {
            prev[q] = __ldg(counts + (long long)blockIdx.x * digits + d);
            total[q] = __ldg(counts + tiles * digits + d);
        }
        sum += total[q];
    }
    uint32_t incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    if (lane == 31) s_warp[warp] = incl;
    __syncthreads();
    uint32_t at = incl - sum;
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w) at += w < warp ? s_warp[w] : 0u;
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
        const int d = kPer * tid + q;
        if (d < digits) {
            uint32_t run = at + prev[q];
#pragma unroll
            for (int w = 0; w < kSortWarps; ++w) {
                const uint32_t c = s_cnt[w][d];
                s_cnt[w][d] = run;
                run += c;
            }
        }
        at += total[q];
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kSortKeys; ++j) {
        const long long i = base + j * 32 + lane;
        if (i < p.tokens) {
            const uint32_t to = s_cnt[warp][(key[j] >> shift) & (uint32_t)(digits - 1)] + rank[j];
            if (to < (uint32_t)p.tokens) {  // holds by construction
                keys_out[to] = key[j];
                vals_out[to] = vals ? vals[i] : (uint32_t)i;
            }
        }
    }
}

// Token positions [first, last) of each id in the sorted order; last == 0 (set
// beforehand) where an id has none.
struct Runs {
    uint32_t *first, *last;
};
__device__ __forceinline__ void mark_run(const uint32_t* keys, long long i, long long n, uint32_t vocab, const Runs& runs) {
    const uint32_t k = keys[i];
    if (k >= vocab) return;
    if (i == 0 || keys[i - 1] != k) runs.first[k] = (uint32_t)i;
    if (i + 1 == n || keys[i + 1] != k) runs.last[k] = (uint32_t)(i + 1);
}
__global__ void __launch_bounds__(kNT) sort_runs_kernel(const uint32_t* keys, long long n, uint32_t vocab, Runs runs) {
    const long long i = (long long)blockIdx.x * kNT + threadIdx.x;
    if (i < n) mark_run(keys, i, n, vocab, runs);
}

// The whole sort by one cluster: CTA r has the keys [r, r + 1) * kClusterNT * K of
// each pass's input, K as few as 8 CTAs allow.  As in the kernels above, but the
// CTAs' digit counts are read from one another's shared memory, and a barrier of
// the cluster stands between one pass's placement and the next pass's loads.
// Lanes with the same digit find one another by a ballot per bit.
template <int K>
__global__ void __launch_bounds__(kClusterNT) sort_cluster_kernel(EmbedParams p, int passes, int bits, uint32_t* keys0,
                                                                  uint32_t* vals0, uint32_t* keys1, uint32_t* vals1,
                                                                  Runs runs, bool zero_last) {
    namespace cg = cooperative_groups;
    extern __shared__ uint16_t s_cnt[];  // [kClusterWarps][digits]
    __shared__ uint32_t s_total[kMaxDigit], s_base[kMaxDigit], s_warp[kClusterWarps];
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank(), ctas = (int)cluster.num_blocks();
    const int digits = 1 << bits, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t mask = (uint32_t)digits - 1;
    const long long base = (long long)rank * (kClusterNT * K) + warp * (32 * K);
    uint32_t *kin = nullptr, *vin = nullptr;
    if (zero_last)  // the cluster's barriers stand between these and the marks below
        for (long long i = (long long)rank * kClusterNT + tid; i < p.vocab; i += (long long)ctas * kClusterNT)
            runs.last[i] = 0u;
    for (int pass = 0; pass < passes; ++pass) {
        const int shift = pass * bits;
        uint32_t *ko = pass & 1 ? keys1 : keys0, *vo = pass & 1 ? vals1 : vals0;
        uint32_t key[K], val[K], rk[K];
#pragma unroll
        for (int j = 0; j < K; ++j) {
            const long long i = base + j * 32 + lane;
            key[j] = val[j] = 0u;
            if (i < p.tokens) {
                key[j] = sort_key(p, kin, i);
                val[j] = vin ? vin[i] : (uint32_t)i;
            }
        }
        for (int i = tid; i < kClusterWarps * digits / 2; i += kClusterNT) reinterpret_cast<uint32_t*>(s_cnt)[i] = 0u;
        __syncthreads();
        uint16_t* mine = s_cnt + warp * digits;
#pragma unroll
        for (int j = 0; j < K; ++j) {
            const bool live = base + j * 32 + lane < p.tokens;
            const uint32_t d = (key[j] >> shift) & mask;
            uint32_t m = __ballot_sync(0xffffffffu, live);
            for (int q = 0; q < bits; ++q) {
                const uint32_t one = __ballot_sync(0xffffffffu, d >> q & 1u);
                m &= d >> q & 1u ? one : ~one;
            }
            const uint32_t before = live ? mine[d] : 0u;
            __syncwarp();
            rk[j] = before + __popc(m & ((1u << lane) - 1u));
            if (live && lane == __ffs(m) - 1) mine[d] = (uint16_t)(before + __popc(m));
            __syncwarp();
        }
        __syncthreads();
        if (tid < digits) {  // the warps before, per digit; the CTA's total
            uint32_t run = 0;
#pragma unroll 8
            for (int w = 0; w < kClusterWarps; ++w) {
                const uint32_t c = s_cnt[w * digits + tid];
                s_cnt[w * digits + tid] = (uint16_t)run;
                run += c;
            }
            s_total[tid] = run;
        }
        cluster.sync();
        uint32_t prev = 0, total = 0;
        if (tid < digits)
        {
            uint32_t c[kClusterCtas];  // all asked for at once
#pragma unroll
            for (int r = 0; r < kClusterCtas; ++r) c[r] = r < ctas ? cluster.map_shared_rank(s_total, r)[tid] : 0u;
#pragma unroll
            for (int r = 0; r < kClusterCtas; ++r) {
                prev += r < rank ? c[r] : 0u;
                total += c[r];
            }
        }
        uint32_t incl = total;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += y;
        }
        if (lane == 31) s_warp[warp] = incl;
        __syncthreads();
        const uint32_t at = incl - total + prev + __reduce_add_sync(0xffffffffu, lane < warp ? s_warp[lane] : 0u);
        if (tid < digits) s_base[tid] = at;
        __syncthreads();
#pragma unroll
        for (int j = 0; j < K; ++j) {
            if (base + j * 32 + lane < p.tokens) {
                const uint32_t d = (key[j] >> shift) & mask, to = s_base[d] + mine[d] + rk[j];
                if (to < (uint32_t)p.tokens) {  // holds by construction
                    ko[to] = key[j];
                    vo[to] = val[j];
                }
            }
        }
        cluster.sync();  // the pass's output is there, and nobody reads s_total any more
        kin = ko;
        vin = vo;
    }
#pragma unroll
    for (int j = 0; j < K; ++j) {
        const long long i = base + j * 32 + lane;
        if (i < p.tokens) mark_run(kin, i, p.tokens, (uint32_t)p.vocab, runs);
    }
}

// ----------------------------------------------------------------- sums
// acc += the rows of dout at sorted positions [lo, hi), in order, for this
// thread's columns: kVec: c .. c + W - 1, else c, c + step, ...
template <class T, int W, bool kVec>
__device__ __forceinline__ void add_rows(const T* dout, long long ldd, const uint32_t* vals, long long lo, long long hi,
                                         long long c, int step, long long dim, float (&acc)[W]) {
    long long i = lo;
    if constexpr (kVec) {
        if (c >= dim) return;
        for (; i + 16 <= hi; i += 16) {
            Vec<T, W> v[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) v[j].load(dout + (long long)vals[i + j] * ldd + c);
#pragma unroll
            for (int j = 0; j < 16; ++j)
#pragma unroll
                for (int k = 0; k < W; ++k) acc[k] += v[j].get(k);
        }
        for (; i + 4 <= hi; i += 4) {
            Vec<T, W> v[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j].load(dout + (long long)vals[i + j] * ldd + c);
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int k = 0; k < W; ++k) acc[k] += v[j].get(k);
        }
        for (; i < hi; ++i) {
            Vec<T, W> v;
            v.load(dout + (long long)vals[i] * ldd + c);
#pragma unroll
            for (int k = 0; k < W; ++k) acc[k] += v.get(k);
        }
    } else {
        for (; i < hi; i += 4) {
            T v[4][W];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const T* row = dout + (i + j < hi ? (long long)vals[i + j] : 0) * ldd + c;
#pragma unroll
                for (int k = 0; k < W; ++k)
                    v[j][k] = i + j < hi && c + (long long)k * step < dim ? __ldg(row + (long long)k * step)
                                                                         : from_f32<T>(0.0f);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int k = 0; k < W; ++k) acc[k] += to_f32(v[j][k]);
        }
    }
}

// Piece blockIdx.x of the sorted tokens, [kRun * x, kRun * (x + 1)): where its
// first or its last token belongs to a run longer than kRun, the sum of that
// run's part of the piece, into partial row 2x (the run holds the piece's first
// token) or 2x + 1 (it starts inside).
template <class T, int W, bool kVec>
__global__ void __launch_bounds__(kNT) embed_pieces_kernel(EmbedParams p, const uint32_t* keys, const uint32_t* vals,
                                                           Runs runs, float* partials, int tpr) {
    __shared__ long long s_lo[2], s_hi[2];
    __shared__ uint32_t s_vals[kRun];
    __shared__ float s_sum[W * kNT];
    const long long b0 = (long long)blockIdx.x * kRun, b1 = min(b0 + kRun, p.tokens);
    if (threadIdx.x >= 32 && threadIdx.x < 32 + kRun && b0 + threadIdx.x - 32 < b1)
        s_vals[threadIdx.x - 32] = vals[b0 + threadIdx.x - 32];
    if (threadIdx.x < 2) {
        const uint32_t k = keys[threadIdx.x == 0 ? b0 : b1 - 1];
        long long lo = 0, hi = 0;
        if (k < (uint32_t)p.vocab) {
            lo = runs.first[k];
            hi = runs.last[k];
        }
        if (hi - lo <= kRun) lo = hi = 0;
        s_lo[threadIdx.x] = lo;
        s_hi[threadIdx.x] = hi;
    }
    __syncthreads();
    // with few columns the piece's rows go to several thread rows, whose sums are
    // then added in order
    const int sub = threadIdx.x / tpr, lane = threadIdx.x % tpr, subs = kNT / tpr, share = (kRun + subs - 1) / subs;
    const long long c = (long long)blockIdx.y * tpr * W + (long long)lane * (kVec ? W : 1);
    for (int which = 0; which < 2; ++which) {
        const long long lo = s_lo[which], hi = s_hi[which];
        if (hi == lo) continue;
        if (which == 1 && lo <= b0) continue;  // the same run as `which == 0`
        float acc[W];
#pragma unroll
        for (int k = 0; k < W; ++k) acc[k] = 0.0f;
        const long long from = max(lo, b0) - b0 + sub * share, to = min(min(hi, b1) - b0, from + share);
        add_rows<T, W, kVec>(static_cast<const T*>(p.weight), p.ldw, s_vals, from, to, c, tpr, p.dim, acc);
        if (subs > 1) {
            __syncthreads();
#pragma unroll
            for (int k = 0; k < W; ++k) s_sum[k * kNT + threadIdx.x] = acc[k];
            __syncthreads();
            if (sub != 0) continue;
            for (int q = 1; q < subs; ++q)
#pragma unroll
                for (int k = 0; k < W; ++k) acc[k] += s_sum[k * kNT + q * tpr + lane];
        }
        float* row = partials + (2 * (long long)blockIdx.x + which) * p.dim;
#pragma unroll
        for (int k = 0; k < W; ++k) {
            const long long cc = c + (long long)k * (kVec ? 1 : tpr);
            if (cc < p.dim) row[cc] = acc[k];
        }
    }
}

template <class T, class O, int W, bool kVec>
__global__ void __launch_bounds__(kNT) embed_rows_kernel(EmbedParams p, const uint32_t* vals, Runs runs,
                                                         const float* partials, int tpr, int per_cta) {
    __shared__ uint32_t s_first[kRowsPerCta], s_last[kRowsPerCta];
    const long long row0 = (long long)blockIdx.x * per_cta;
    if (threadIdx.x < per_cta) {
        const bool in = row0 + threadIdx.x < p.vocab;
        s_last[threadIdx.x] = in ? runs.last[row0 + threadIdx.x] : 0u;
        s_first[threadIdx.x] = in ? runs.first[row0 + threadIdx.x] : 0u;  // anything where last is 0
    }
    __syncthreads();
    const int sub = threadIdx.x / tpr, lane = threadIdx.x % tpr, step = kNT / tpr;
    const int rows = (int)min((long long)per_cta, p.vocab - row0);
    const long long c = (long long)blockIdx.y * tpr * W + (long long)lane * (kVec ? W : 1);
    if (kVec && c >= p.dim) return;
    O* out0 = static_cast<O*>(p.out) + row0 * p.ldo + c;
    if (!kVec && !p.accumulate && p.ldo == p.dim && gridDim.y == 1) {
        // rows without gaps, but not in 16-byte words: zeros over the CTA's whole
        // stretch, in words as far as it has them, then the sums over those
        O* begin = static_cast<O*>(p.out) + row0 * p.ldo;
        const long long n = (long long)rows * p.dim;
        const long long head = min((long long)((16 - reinterpret_cast<uintptr_t>(begin) % 16) % 16 / sizeof(O)), n);
        const long long words = (n - head) / (16 / (int)sizeof(O)), tail = head + words * (16 / (int)sizeof(O));
        for (long long i = threadIdx.x; i < words; i += kNT)
            reinterpret_cast<uint4*>(begin + head)[i] = make_uint4(0u, 0u, 0u, 0u);
        if (threadIdx.x < head) begin[threadIdx.x] = from_f32<O>(0.0f);
        if (tail + threadIdx.x < n) begin[tail + threadIdx.x] = from_f32<O>(0.0f);
        __syncthreads();
    } else if (!p.accumulate) {
        for (int r = sub; r < rows; r += step) {
            if (s_last[r] != 0u) continue;
            O* out = out0 + r * p.ldo;
            if constexpr (kVec) {
                Vec<O, W> v;
                v.zero();
                v.store(out);
            } else {
#pragma unroll
                for (int k = 0; k < W; ++k)
                    if (c + (long long)k * tpr < p.dim) out[(long long)k * tpr] = from_f32<O>(0.0f);
            }
        }
    }
    for (int r = sub; r < rows; r += step) {
        const long long lo = s_first[r], hi = s_last[r];
        if (hi == 0) continue;
        float acc[W];
#pragma unroll
        for (int k = 0; k < W; ++k) acc[k] = 0.0f;
        if (hi - lo <= kRun) {
            add_rows<T, W, kVec>(static_cast<const T*>(p.weight), p.ldw, vals, lo, hi, c, tpr, p.dim, acc);
        } else {
#pragma unroll 4
            for (long long piece = lo / kRun; piece * kRun < hi; ++piece) {
                const float* row = partials + (2 * piece + (lo <= piece * kRun ? 0 : 1)) * p.dim;
#pragma unroll
                for (int k = 0; k < W; ++k) {
                    const long long cc = c + (long long)k * (kVec ? 1 : tpr);
                    if (cc < p.dim) acc[k] += __ldg(row + cc);
                }
            }
        }
        O* out = out0 + r * p.ldo;
        if constexpr (kVec) {
            Vec<O, W> v;
            if (p.accumulate) v.load_rw(out);
#pragma unroll
            for (int k = 0; k < W; ++k) acc[k] = acc[k] * p.scale + (p.accumulate ? v.get(k) : 0.0f);
            v.set(acc);
            v.store(out);
        } else {
#pragma unroll
            for (int k = 0; k < W; ++k) {
                const long long o = (long long)k * tpr;
                if (c + o < p.dim) out[o] = from_f32<O>(acc[k] * p.scale + (p.accumulate ? to_f32(out[o]) : 0.0f));
            }
        }
    }
}

// Threads per row for rows of `dim` elements, W of them a thread: a power of two.
int threads_per_row(long long dim, int w) {
    int t = 1;
    while (t < kNT && (long long)t * w < dim) t *= 2;
    return t;
}

long long ceil_div(long long a, long long b) { return (a + b - 1) / b; }

template <class T>
cudaError_t embed_of(const EmbedParams& p, cudaStream_t s) {
    constexpr int W = 16 / sizeof(T);
    const int tpr = threads_per_row(p.dim, W);
    const dim3 grid((unsigned)ceil_div(p.tokens, kNT / tpr), (unsigned)ceil_div(p.dim, (long long)tpr * W));
    if (p.vec) embed_kernel<T, true><<<grid, kNT, 0, s>>>(p, tpr);
    else embed_kernel<T, false><<<grid, kNT, 0, s>>>(p, tpr);
    return cudaGetLastError();
}

template <class T, class O>
cudaError_t sums_of(const EmbedParams& p, const uint32_t* keys, const uint32_t* vals, const Runs& runs, float* partials,
                    cudaStream_t s) {
    constexpr int W = 16 / sizeof(T);
    const int tpr = threads_per_row(p.dim, W);
    const unsigned slices = (unsigned)ceil_div(p.dim, (long long)tpr * W);
    if (p.tokens > kRun) {
        const dim3 grid((unsigned)ceil_div(p.tokens, kRun), slices);
        if (p.vec) embed_pieces_kernel<T, W, true><<<grid, kNT, 0, s>>>(p, keys, vals, runs, partials, tpr);
        else embed_pieces_kernel<T, W, false><<<grid, kNT, 0, s>>>(p, keys, vals, runs, partials, tpr);
        count_launches(1);
    }
    // fewer rows a CTA, down to one for each of its thread rows, where 32 would
    // leave SMs without a CTA
    int per_cta = kRowsPerCta;
    const long long enough = 8 * seq_sms();
    while (per_cta > std::max(kNT / tpr / 2, 1) && ceil_div(p.vocab, per_cta) * slices < enough) per_cta /= 2;
    const dim3 grid((unsigned)ceil_div(p.vocab, per_cta), slices);
    if (p.vec) embed_rows_kernel<T, O, W, true><<<grid, kNT, 0, s>>>(p, vals, runs, partials, tpr, per_cta);
    else embed_rows_kernel<T, O, W, false><<<grid, kNT, 0, s>>>(p, vals, runs, partials, tpr, per_cta);
    count_launches(1);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_embed(int dtype, const EmbedParams& p, cudaStream_t s) {
    count_launches(1);
    switch (dtype) {
    case SC_F32: return embed_of<float>(p, s);
    case SC_F16: return embed_of<f16>(p, s);
    case SC_BF16: return embed_of<bf16>(p, s);
    default: return cudaErrorInvalidValue;
    }
}

EmbedGradPlan embed_grad_plan(long long tokens, long long vocab, long long dim) {
    EmbedGradPlan g{};
    int bits = 1;
    while ((vocab >> bits) != 0) ++bits;  // keys 0 .. vocab
    g.passes = (bits + 9) / 10;
    g.digit_bits = (bits + g.passes - 1) / g.passes;
    g.tiles = ceil_div(std::max(tokens, 1ll), kSortTile);
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t o = at;
        at += (bytes + 255) / 256 * 256;
        return o;
    };
    g.keys0 = take((size_t)tokens * 4);
    g.keys1 = take((size_t)tokens * 4);
    g.vals0 = take((size_t)tokens * 4);
    g.vals1 = take((size_t)tokens * 4);
    g.first = take((size_t)vocab * 4);
    g.last = take((size_t)vocab * 4);
    g.counts = take(tokens <= kClusterKeys ? 0 : (size_t)(g.tiles + 1) * (size_t)(1 << g.digit_bits) * 4);
    g.partials = take(tokens > kRun ? (size_t)ceil_div(tokens, kRun) * 2 * (size_t)dim * 4 : 0);
    g.total = at;
    return g;
}

sc_status launch_embed_grad(int dtype, int wtype, const EmbedParams& p, const EmbedGradPlan& g, unsigned char* base,
                            cudaStream_t s) {
    uint32_t* keys[2] = {reinterpret_cast<uint32_t*>(base + g.keys0), reinterpret_cast<uint32_t*>(base + g.keys1)};
    uint32_t* vals[2] = {reinterpret_cast<uint32_t*>(base + g.vals0), reinterpret_cast<uint32_t*>(base + g.vals1)};
    uint32_t* counts = reinterpret_cast<uint32_t*>(base + g.counts);
    float* partials = reinterpret_cast<float*>(base + g.partials);
    const Runs runs{reinterpret_cast<uint32_t*>(base + g.first), reinterpret_cast<uint32_t*>(base + g.last)};
    const uint32_t *kin = nullptr, *vin = nullptr;
    // The cluster clears `last` on its way while that is little work (16 words a
    // thread): a launch less (300 tokens of 5000 ids, lookup and gradient: 23.6 us
    // so, 26.8 with a launch that clears).
    const long long each = ceil_div(p.tokens, (long long)kClusterNT * kClusterCtas);
    const long long k = each <= 2 ? std::max(each, 1ll) : each <= 4 ? 4 : 8, ctas = ceil_div(p.tokens, kClusterNT * k);
    const bool in_cluster = p.tokens > 0 && p.tokens <= kClusterKeys, zero_last = in_cluster && p.vocab <= 16 * kClusterNT * ctas;
    if (!zero_last) {
        const sc_status st = status_of(cudaMemsetAsync(runs.last, 0, (size_t)p.vocab * 4, s));
        if (st != SC_OK) return st;
    }
    if (in_cluster) {
        auto go = [&](auto kernel) {
            const int bytes = kClusterWarps * (1 << g.digit_bits) * 2;
            cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kClusterShared);
            if (e != cudaSuccess) return e;
            cudaLaunchAttribute attr{};
            attr.id = cudaLaunchAttributeClusterDimension;
            attr.val.clusterDim = {(unsigned)ctas, 1, 1};
            cudaLaunchConfig_t cfg{};
            cfg.gridDim = dim3(attr.val.clusterDim.x);
            cfg.blockDim = dim3(kClusterNT);
            cfg.dynamicSmemBytes = (size_t)bytes;
            cfg.stream = s;
            cfg.attrs = &attr;
            cfg.numAttrs = 1;
            return cudaLaunchKernelEx(&cfg, kernel, p, g.passes, g.digit_bits, keys[0], vals[0], keys[1], vals[1], runs,
                                      zero_last);
        };
        const cudaError_t e = k == 1   ? go(sort_cluster_kernel<1>)
                              : k == 2 ? go(sort_cluster_kernel<2>)
                              : k == 4 ? go(sort_cluster_kernel<4>)
                                       : go(sort_cluster_kernel<8>);
        if (e != cudaSuccess) return status_of(e);
        count_launches(1);
        kin = keys[(g.passes - 1) & 1];
        vin = vals[(g.passes - 1) & 1];
    } else if (p.tokens > 0) {
        const int digits = 1 << g.digit_bits;
        for (int pass = 0; pass < g.passes; ++pass) {
            const int shift = pass * g.digit_bits;
            uint32_t *ko = keys[pass & 1], *vo = vals[pass & 1];
            sort_count_kernel<<<(unsigned)g.tiles, kNT, 0, s>>>(p, kin, shift, g.digit_bits, counts);
            sort_columns_kernel<<<(unsigned)ceil_div(digits, kNT), kNT, 0, s>>>(counts, g.tiles, digits);
            sort_place_kernel<<<(unsigned)g.tiles, kNT, 0, s>>>(p, kin, vin, shift, g.digit_bits, counts, g.tiles, ko, vo);
            count_launches(3);
            kin = ko;
            vin = vo;
        }
        sort_runs_kernel<<<(unsigned)ceil_div(p.tokens, kNT), kNT, 0, s>>>(kin, p.tokens, (uint32_t)p.vocab, runs);
        count_launches(1);
        if (cudaGetLastError() != cudaSuccess) return SC_ERR_CUDA;
    }
    cudaError_t e = cudaErrorInvalidValue;
    if (dtype == SC_F32) e = sums_of<float, float>(p, kin, vin, runs, partials, s);
    else if (dtype == SC_F16) e = wtype == SC_F32 ? sums_of<f16, float>(p, kin, vin, runs, partials, s)
                                                  : sums_of<f16, f16>(p, kin, vin, runs, partials, s);
    else if (dtype == SC_BF16) e = wtype == SC_F32 ? sums_of<bf16, float>(p, kin, vin, runs, partials, s)
                                                   : sums_of<bf16, bf16>(p, kin, vin, runs, partials, s);
    return status_of(e);
}

}  // namespace scg
