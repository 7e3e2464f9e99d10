// The norm of a token's channels (with the residual sum in front of it) and its
// gradient: kernels, by element type in sc_norm_*.cu.
//
//   s = x + residual, rounded;  n = (s - m) r;  y = n weight + bias
//   dn = dy weight;  dx = r (dn - mean(dn) - n mean(dn n)) + dsum
//   dweight = sum over tokens of dy n;  dbias = sum over tokens of dy
// (rms: m = 0, and mean(dn) drops out.)
//
// A row lies in the registers of kLanes threads, N elements each, so each tensor is
// read and written once: bytes are all that the operator costs (a third of the
// issue slots at most).  The variance is of the centred row, a second sum over
// registers, not a difference of moments.  Rows of up to 32 vectors of 16 bytes take
// part of a warp or one, wider ones up to 1024 threads, which then meet in shared
// memory.  Rows beyond kRowMax elements are read again for each of their sums.
//
// The gradient's sums over tokens: a persistent CTA keeps its columns' sums in
// registers over all its rows, writes one row of partial sums, and a second kernel
// adds those in the order of the CTAs: the same bits on every run.
#pragma once
#include <algorithm>

#include "sc_seq.cuh"
#include "sc_seq_launch.h"

namespace scg {

namespace {

constexpr long long kRowMax = 8192;

template <class T> constexpr int kWidth = 16 / (int)sizeof(T);  // elements of a vector

__device__ __forceinline__ long long at(uint32_t row, uint32_t length, long long sb, long long st) {
    const uint32_t b = row / length;
    return (long long)b * sb + (long long)(row - b * length) * st;
}

// Element j of vector i of a lane: aligned rows by vectors, others by elements.
template <class T, bool kVec, int kLanes>
__device__ __forceinline__ int column(int i, int j, int lane) {
    return kVec ? (i * kLanes + lane) * kWidth<T> + j : (i * kWidth<T> + j) * kLanes + lane;
}

template <class T, bool kVec, int kLanes, int NV>
struct Row {
    static constexpr int W = kWidth<T>;
    Vec<T, W> v[NV];
    __device__ __forceinline__ void load(const T* p, int lane, int channels) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if constexpr (kVec) {
                const int c = column<T, kVec, kLanes>(i, 0, lane);
                if (c < channels) v[i].load(p + c);
                else v[i].zero();
            } else {
                T e[W];
#pragma unroll
                for (int j = 0; j < W; ++j) {
                    const int c = column<T, kVec, kLanes>(i, j, lane);
                    e[j] = c < channels ? __ldg(p + c) : from_f32<T>(0.0f);
                }
                memcpy(v[i].w, e, 16);
            }
        }
    }
    __device__ __forceinline__ float get(int i, int j) const { return v[i].get(j); }
    __device__ __forceinline__ static void store(T* p, int lane, int channels, const float (&f)[NV * W]) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if constexpr (kVec) {
                const int c = column<T, kVec, kLanes>(i, 0, lane);
                if (c < channels) {
                    Vec<T, W> o;
                    o.set(&f[i * W]);
                    o.store(p + c);
                }
            } else {
#pragma unroll
                for (int j = 0; j < W; ++j) {
                    const int c = column<T, kVec, kLanes>(i, j, lane);
                    if (c < channels) p[c] = from_f32<T>(f[i * W + j]);
                }
            }
        }
    }
};

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
            float s = 0.0f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) s += slot[k * kWarps + w];
            v[k] = s;
        }
    }
}

template <int kLanes> constexpr int kThreads = kLanes < 256 ? 256 : kLanes;

// ---------------------------------------------------------------- forward
template <class T, bool kVec, int kLanes, int NV>
__global__ void __launch_bounds__(kThreads<kLanes>) norm_kernel(NormParams p) {
    constexpr int W = kWidth<T>, N = NV * W, kGroups = kThreads<kLanes> / kLanes;
    __shared__ float s_sum[kGroups][2][kLanes > 32 ? kLanes / 32 : 1];
    const int group = threadIdx.x / kLanes, lane = threadIdx.x % kLanes, channels = (int)p.channels;
    const long long r0 = (long long)blockIdx.x * kGroups + group;
    const bool live = r0 < p.rows;
    if (kLanes >= 32 && !live) return;  // part of a warp stays for the shuffles
    const uint32_t r = live ? (uint32_t)r0 : 0u;
    const int some = live ? channels : 0;
    using R = Row<T, kVec, kLanes, NV>;
    R x;
    x.load(static_cast<const T*>(p.x) + at(r, p.length, p.x_batch, p.x_token), lane, some);
    float f[N];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < W; ++j) f[i * W + j] = x.get(i, j);
    if (p.residual) {
        R e;
        e.load(static_cast<const T*>(p.residual) + at(r, p.length, p.residual_batch, p.residual_token), lane, some);
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < W; ++j) f[i * W + j] = to_f32(from_f32<T>(f[i * W + j] + e.get(i, j)));
        R::store(static_cast<T*>(p.sum) + at(r, p.length, p.sum_batch, p.sum_token), lane, some, f);
    }
    const float per = 1.0f / (float)channels;
    float mean = 0.0f;
    if (!p.rms) {
        float s[1] = {0.0f};
#pragma unroll
        for (int i = 0; i < N; ++i) s[0] += f[i];
        row_sum<kLanes, 1>(s, s_sum[group][0], lane, group);
        mean = s[0] * per;
    }
    float q[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < W; ++j) {
            float& c = f[i * W + j];
            c = column<T, kVec, kLanes>(i, j, lane) < channels ? c - mean : 0.0f;
            q[0] = fmaf(c, c, q[0]);
        }
    row_sum<kLanes, 1>(q, s_sum[group][1], lane, group);
    const float rstd = 1.0f / sqrtf(fmaf(q[0], per, p.eps));
    if (p.saved && lane == 0 && live) reinterpret_cast<float2*>(p.saved)[r] = make_float2(mean, rstd);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if (kVec && column<T, kVec, kLanes>(i, 0, lane) >= channels) continue;
#pragma unroll
        for (int j = 0; j < W; ++j) {
            const int c = column<T, kVec, kLanes>(i, j, lane);
            float& o = f[i * W + j];
            if (!kVec && c >= channels) continue;
            o *= rstd;
            const float w = p.weight ? parameter<T>(p.weight, p.params_f32, c) : 1.0f;
            o = p.bias ? fmaf(o, w, parameter<T>(p.bias, p.params_f32, c)) : o * w;
        }
    }
    R::store(static_cast<T*>(p.y) + at(r, p.length, p.y_batch, p.y_token), lane, some, f);
}

// --------------------------------------------------------------- gradient
// CTAs that an SM holds: 65536 registers by 128 a thread (64 of 1024 threads).
template <int kLanes> constexpr int kResident = kThreads<kLanes> == 256 ? 2 : 1;

template <class T, bool kVec, int kLanes, int NV>
__global__ void __launch_bounds__(kThreads<kLanes>, kResident<kLanes>) norm_grad_kernel(NormParams p) {
    constexpr int W = kWidth<T>, N = NV * W, NT = kThreads<kLanes>, kGroups = NT / kLanes;
    __shared__ float s_sum[kGroups][2][2 * (kLanes > 32 ? kLanes / 32 : 1)];
    __shared__ float s_col[kGroups > 1 ? NT * N : 1];
    const int group = threadIdx.x / kLanes, lane = threadIdx.x % kLanes, channels = (int)p.channels;
    using R = Row<T, kVec, kLanes, NV>;
    float w[N], dw[N], db[N];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < W; ++j) {
            const int c = column<T, kVec, kLanes>(i, j, lane);
            w[i * W + j] = c >= channels ? 0.0f : p.weight ? parameter<T>(p.weight, p.params_f32, c) : 1.0f;
            dw[i * W + j] = db[i * W + j] = 0.0f;
        }
    const float per = 1.0f / (float)channels;
    const long long step = (long long)gridDim.x * kGroups;
    // a warp's groups go round together, for the shuffles
    const long long first = (long long)blockIdx.x * kGroups + (kLanes >= 32 ? group : threadIdx.x / 32 * (32 / kLanes));
    const int mine = kLanes >= 32 ? 0 : group % (32 / (kLanes < 32 ? kLanes : 32));
    R x, dy, ds;
    float2 stat;
    auto fetch = [&](long long base) {
        const long long row = base + mine;
        const bool live = row < p.rows;
        const uint32_t r = live ? (uint32_t)row : 0u;
        const int some = live ? channels : 0;
        x.load(static_cast<const T*>(p.x) + at(r, p.length, p.x_batch, p.x_token), lane, some);
        dy.load(static_cast<const T*>(p.dy) + at(r, p.length, p.dy_batch, p.dy_token), lane, some);
        if (p.dsum) ds.load(static_cast<const T*>(p.dsum) + at(r, p.length, p.dsum_batch, p.dsum_token), lane, some);
        stat = __ldg(reinterpret_cast<const float2*>(p.saved) + r);
    };
    int turn = 0;
    if (first < p.rows) fetch(first);
    for (long long base = first; base < p.rows; base += step) {
        const R x0 = x, dy0 = dy, ds0 = ds;
        const float mean = stat.x, rstd = stat.y;
        if (base + step < p.rows) fetch(base + step);  // under way during this row's sums
        float s[2] = {0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < W; ++j) {
                const int k = i * W + j;
                const float g = dy0.get(i, j), n = (x0.get(i, j) - mean) * rstd, dn = g * w[k];
                s[0] += dn;
                // w = 0 behind the row's end, where n is not 0
                s[1] = fmaf(dn, n, s[1]);
                db[k] += g;
                dw[k] = fmaf(g, n, dw[k]);
            }
        row_sum<kLanes, 2>(s, s_sum[group][turn], lane, group);
        turn ^= 1;
        const float a = p.rms ? 0.0f : s[0] * per, b = s[1] * per;
        float o[N];
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < W; ++j) {
                const int k = i * W + j;
                const float n = (x0.get(i, j) - mean) * rstd;
                o[k] = fmaf(-n, b, dy0.get(i, j) * w[k] - a) * rstd;
                if (p.dsum) o[k] += ds0.get(i, j);
            }
        if (base + mine < p.rows)
            R::store(static_cast<T*>(p.dx) + (base + mine) * channels, lane, channels, o);
    }
    if (!p.partials) return;
    // one row of partial sums a CTA: over its groups, in their order
    auto put = [&](int which, const float (&v)[N]) {
        float* to = p.partials + ((long long)blockIdx.x * 2 + which) * channels;
        if constexpr (kGroups == 1) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int j = 0; j < W; ++j) {
                    const int c = column<T, kVec, kLanes>(i, j, lane);
                    if (c < channels) to[c] = v[i * W + j];
                }
        } else {
            __syncthreads();
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int j = 0; j < W; ++j) s_col[group * (kLanes * N) + column<T, kVec, kLanes>(i, j, lane)] = v[i * W + j];
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
    __shared__ float slot[2][kWideNT / 32];
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
    const float rstd = 1.0f / sqrtf(fmaf(q[0], per, p.eps));
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
    __shared__ float slot[2 * kWideNT / 32];
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
constexpr int kColumnNT = 256;
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
template <class T, bool kVec, int kLanes, int NV>
cudaError_t go(const NormParams& p, bool grad, cudaStream_t s) {
    constexpr int NT = kThreads<kLanes>, kGroups = NT / kLanes;
    if (grad) norm_grad_kernel<T, kVec, kLanes, NV><<<(unsigned)p.parts, NT, 0, s>>>(p);
    else norm_kernel<T, kVec, kLanes, NV><<<(unsigned)((p.rows + (long long)kGroups - 1) / kGroups), NT, 0, s>>>(p);
    return cudaGetLastError();
}

template <class T, bool kVec>
cudaError_t by_width(const NormParams& p, bool grad, cudaStream_t s) {
    const long long n = (p.channels + kWidth<T> - 1) / kWidth<T>;
    if (n <= 8) return go<T, kVec, 8, 1>(p, grad, s);
    if (n <= 16) return go<T, kVec, 16, 1>(p, grad, s);
    if (n <= 32) return go<T, kVec, 32, 1>(p, grad, s);
    if (n <= 64) return go<T, kVec, 32, 2>(p, grad, s);
    if (n <= 128) return go<T, kVec, 64, 2>(p, grad, s);
    if (n <= 256) return go<T, kVec, 128, 2>(p, grad, s);
    if (n <= 512) return go<T, kVec, 256, 2>(p, grad, s);
    if (n <= 1024) return go<T, kVec, 512, 2>(p, grad, s);
    if constexpr (sizeof(T) == 4) return go<T, kVec, 1024, 2>(p, grad, s);
    return cudaErrorInvalidValue;
}

template <class T>
cudaError_t launch_norm_as(const NormParams& p, bool grad, cudaStream_t s) {
    if (p.channels <= kRowMax) {
        const cudaError_t e = p.vec ? by_width<T, true>(p, grad, s) : by_width<T, false>(p, grad, s);
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
    const dim3 grid((unsigned)((p.channels + kColumnNT - 1) / kColumnNT), (unsigned)p.parts);
    norm_columns_kernel<T><<<grid, kColumnNT, 0, s>>>(p);
    count_launches(1);
    return cudaGetLastError();
}

}  // namespace

// By element type, one translation unit each.
cudaError_t launch_norm_f32(const NormParams& p, bool grad, cudaStream_t s);
cudaError_t launch_norm_f16(const NormParams& p, bool grad, cudaStream_t s);
cudaError_t launch_norm_bf16(const NormParams& p, bool grad, cudaStream_t s);

}  // namespace scg
