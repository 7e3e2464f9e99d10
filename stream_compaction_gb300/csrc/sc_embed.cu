// Token embedding, out[t] = scale * weight[ids[t]], and its gradient
// dweight[v] = scale * sum of dout[t] over ids[t] == v.
//
// Both move rows and compute next to nothing: the floor is their bytes.  The
// gradient writes each row of dweight once and reads each row of dout once:
//
//   sort       the (id, t) pairs by id, stable, least significant digit first,
//              at most 10 bits a pass (so two passes below 2^20 ids): per tile
//              digit counts, then the placement, whose CTAs add up the counts
//              of the earlier tiles themselves (beyond kFoldTiles tiles a
//              kernel of its own scans them);
//   long runs  tokens of one id may be a large part of all (padding, a frequent
//              word): runs longer than kRun are cut at multiples of kRun of the
//              sorted order and each piece summed by a CTA of its own;
//   rows       each CTA takes kRowsPerCta rows of dweight, finds their runs in
//              the sorted ids by binary search, and writes zeros, a sum of at
//              most kRun rows of dout, or the sum of the row's pieces.
// Sums are taken in the order of t in float32, so a result is the same on
// every run, whatever the schedule (no atomics on values).
#include <algorithm>

#include "sc_seq.cuh"
#include "sc_seq_launch.h"

namespace scg {

namespace {

constexpr int kNT = 256;
constexpr int kSortKeys = 8;                    // keys per thread of a sort tile
constexpr int kSortTile = kNT * kSortKeys;      // 2048
constexpr int kSortWarps = kNT / 32;
constexpr int kMaxDigit = 1024;
constexpr int kFoldTiles = 16;
constexpr int kRun = 128;
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
template <bool kFold>
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
            if constexpr (kFold) {
                for (long long t = 0; t < tiles; ++t) {
                    const uint32_t c = __ldg(counts + t * digits + d);
                    total[q] += c;
                    prev[q] += t < blockIdx.x ? c : 0u;
                }
            } else {
                prev[q] = __ldg(counts + (long long)blockIdx.x * digits + d);
                total[q] = __ldg(counts + tiles * digits + d);
            }
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

// ----------------------------------------------------------------- sums
// First position of the sorted keys that is >= v.
__device__ __forceinline__ long long lower_bound(const uint32_t* keys, long long n, uint32_t v) {
    long long lo = 0, hi = n;
    while (lo < hi) {
        const long long mid = (lo + hi) >> 1;
        if (__ldg(keys + mid) < v) lo = mid + 1;
        else hi = mid;
    }
    return lo;
}

// acc += the rows of dout at sorted positions [lo, hi), in order, for this
// thread's columns: kVec: c .. c + W - 1, else c, c + step, ...
template <class T, int W, bool kVec>
__device__ __forceinline__ void add_rows(const T* dout, long long ldd, const uint32_t* vals, long long lo, long long hi,
                                         long long c, int step, long long dim, float (&acc)[W]) {
    long long i = lo;
    if constexpr (kVec) {
        if (c >= dim) return;
        for (; i + 4 <= hi; i += 4) {
            Vec<T, W> v[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j].load(dout + (long long)__ldg(vals + i + j) * ldd + c);
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int k = 0; k < W; ++k) acc[k] += v[j].get(k);
        }
        for (; i < hi; ++i) {
            Vec<T, W> v;
            v.load(dout + (long long)__ldg(vals + i) * ldd + c);
#pragma unroll
            for (int k = 0; k < W; ++k) acc[k] += v.get(k);
        }
    } else {
        for (; i < hi; ++i) {
            const T* row = dout + (long long)__ldg(vals + i) * ldd;
#pragma unroll
            for (int k = 0; k < W; ++k) {
                const long long cc = c + (long long)k * step;
                if (cc < dim) acc[k] += to_f32(__ldg(row + cc));
            }
        }
    }
}

// Piece blockIdx.x of the sorted tokens, [kRun * x, kRun * (x + 1)): where its
// first or its last token belongs to a run longer than kRun, the sum of that
// run's part of the piece, into partial row 2x (the run holds the piece's first
// token) or 2x + 1 (it starts inside).
template <class T, int W, bool kVec>
__global__ void __launch_bounds__(kNT) embed_pieces_kernel(EmbedParams p, const uint32_t* keys, const uint32_t* vals,
                                                           float* partials, int tpr) {
    __shared__ long long s_lo[2], s_hi[2];
    const long long b0 = (long long)blockIdx.x * kRun, b1 = min(b0 + kRun, p.tokens);
    if (threadIdx.x < 2) {
        const uint32_t k = keys[threadIdx.x == 0 ? b0 : b1 - 1];
        long long lo = 0, hi = 0;
        if (k < (uint32_t)p.vocab) {
            lo = lower_bound(keys, p.tokens, k);
            hi = lower_bound(keys, p.tokens, k + 1);
        }
        if (hi - lo <= kRun) lo = hi = 0;
        s_lo[threadIdx.x] = lo;
        s_hi[threadIdx.x] = hi;
    }
    __syncthreads();
    const int sub = threadIdx.x / tpr, lane = threadIdx.x % tpr;
    // with few columns the threads left over take the second run's sum
    for (int which = sub; which < 2; which += kNT / tpr) {
        const long long lo = s_lo[which], hi = s_hi[which];
        if (hi == lo) continue;
        if (which == 1 && lo <= b0) continue;  // the same run as `which == 0`
        float acc[W];
#pragma unroll
        for (int k = 0; k < W; ++k) acc[k] = 0.0f;
        const long long c = (long long)blockIdx.y * tpr * W + (long long)lane * (kVec ? W : 1);
        add_rows<T, W, kVec>(static_cast<const T*>(p.weight), p.ldw, vals, max(lo, b0), min(hi, b1), c, tpr, p.dim, acc);
        float* row = partials + (2 * (long long)blockIdx.x + which) * p.dim;
#pragma unroll
        for (int k = 0; k < W; ++k) {
            const long long cc = c + (long long)k * (kVec ? 1 : tpr);
            if (cc < p.dim) row[cc] = acc[k];
        }
    }
}

template <class T, class O, int W, bool kVec>
__global__ void __launch_bounds__(kNT) embed_rows_kernel(EmbedParams p, const uint32_t* keys, const uint32_t* vals,
                                                         const float* partials, int tpr) {
    __shared__ long long s_at[kRowsPerCta + 1];
    const long long row0 = (long long)blockIdx.x * kRowsPerCta;
    if (threadIdx.x <= kRowsPerCta)
        s_at[threadIdx.x] = lower_bound(keys, p.tokens, (uint32_t)min(row0 + threadIdx.x, p.vocab));
    __syncthreads();
    const int sub = threadIdx.x / tpr, lane = threadIdx.x % tpr;
    const long long c = (long long)blockIdx.y * tpr * W + (long long)lane * (kVec ? W : 1);
    for (int r = sub; r < kRowsPerCta && row0 + r < p.vocab; r += kNT / tpr) {
        const long long lo = s_at[r], hi = s_at[r + 1];
        if (lo == hi && p.accumulate) continue;
        float acc[W];
#pragma unroll
        for (int k = 0; k < W; ++k) acc[k] = 0.0f;
        if (hi - lo <= kRun) {
            add_rows<T, W, kVec>(static_cast<const T*>(p.weight), p.ldw, vals, lo, hi, c, tpr, p.dim, acc);
        } else {
            for (long long piece = lo / kRun; piece * kRun < hi; ++piece) {
                const float* row = partials + (2 * piece + (lo <= piece * kRun ? 0 : 1)) * p.dim;
#pragma unroll
                for (int k = 0; k < W; ++k) {
                    const long long cc = c + (long long)k * (kVec ? 1 : tpr);
                    if (cc < p.dim) acc[k] += __ldg(row + cc);
                }
            }
        }
        O* out = static_cast<O*>(p.out) + (row0 + r) * p.ldo;
        if constexpr (kVec) {
            if (c >= p.dim) continue;
            Vec<O, W> v;
            if (p.accumulate) v.load_rw(out + c);
#pragma unroll
            for (int k = 0; k < W; ++k) acc[k] = acc[k] * p.scale + (p.accumulate ? v.get(k) : 0.0f);
            v.set(acc);
            v.store(out + c);
        } else {
#pragma unroll
            for (int k = 0; k < W; ++k) {
                const long long cc = c + (long long)k * tpr;
                if (cc < p.dim) out[cc] = from_f32<O>(acc[k] * p.scale + (p.accumulate ? to_f32(out[cc]) : 0.0f));
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
cudaError_t sums_of(const EmbedParams& p, const uint32_t* keys, const uint32_t* vals, float* partials, cudaStream_t s) {
    constexpr int W = 16 / sizeof(T);
    const int tpr = threads_per_row(p.dim, W);
    const unsigned slices = (unsigned)ceil_div(p.dim, (long long)tpr * W);
    if (p.tokens > kRun) {
        const dim3 grid((unsigned)ceil_div(p.tokens, kRun), slices);
        if (p.vec) embed_pieces_kernel<T, W, true><<<grid, kNT, 0, s>>>(p, keys, vals, partials, tpr);
        else embed_pieces_kernel<T, W, false><<<grid, kNT, 0, s>>>(p, keys, vals, partials, tpr);
        count_launches(1);
    }
    const dim3 grid((unsigned)ceil_div(p.vocab, kRowsPerCta), slices);
    if (p.vec) embed_rows_kernel<T, O, W, true><<<grid, kNT, 0, s>>>(p, keys, vals, partials, tpr);
    else embed_rows_kernel<T, O, W, false><<<grid, kNT, 0, s>>>(p, keys, vals, partials, tpr);
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
    g.counts = take((size_t)(g.tiles + 1) * (size_t)(1 << g.digit_bits) * 4);
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
    const uint32_t *kin = nullptr, *vin = nullptr;
    if (p.tokens > 0) {
        for (int pass = 0; pass < g.passes; ++pass) {
            const int shift = pass * g.digit_bits;
            uint32_t *ko = keys[pass & 1], *vo = vals[pass & 1];
            sort_count_kernel<<<(unsigned)g.tiles, kNT, 0, s>>>(p, kin, shift, g.digit_bits, counts);
            if (g.tiles <= kFoldTiles) {
                sort_place_kernel<true><<<(unsigned)g.tiles, kNT, 0, s>>>(p, kin, vin, shift, g.digit_bits, counts,
                                                                         g.tiles, ko, vo);
                count_launches(2);
            } else {
                const int digits = 1 << g.digit_bits;
                sort_columns_kernel<<<(unsigned)ceil_div(digits, kNT), kNT, 0, s>>>(counts, g.tiles, digits);
                sort_place_kernel<false><<<(unsigned)g.tiles, kNT, 0, s>>>(p, kin, vin, shift, g.digit_bits, counts,
                                                                          g.tiles, ko, vo);
                count_launches(3);
            }
            if (cudaGetLastError() != cudaSuccess) return SC_ERR_CUDA;
            kin = ko;
            vin = vo;
        }
    }
    cudaError_t e = cudaErrorInvalidValue;
    if (dtype == SC_F32) e = sums_of<float, float>(p, kin, vin, partials, s);
    else if (dtype == SC_F16) e = wtype == SC_F32 ? sums_of<f16, float>(p, kin, vin, partials, s)
                                                  : sums_of<f16, f16>(p, kin, vin, partials, s);
    else if (dtype == SC_BF16) e = wtype == SC_F32 ? sums_of<bf16, float>(p, kin, vin, partials, s)
                                                   : sums_of<bf16, bf16>(p, kin, vin, partials, s);
    return e == cudaSuccess ? SC_OK : SC_ERR_CUDA;
}

}  // namespace scg
