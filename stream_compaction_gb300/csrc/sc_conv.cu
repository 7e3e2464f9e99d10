// The short causal convolution of a sequence model, one filter of `width` taps
// per channel, with an optional SiLU; its gradient; and the form for one token.
//
//   pre[t] = bias + sum_k w[k] * x[t-W+1+k]        y = pre * sigmoid(pre)
//   dpre   = dy * sig * (1 + pre * (1 - sig))
//   dx[t]  = sum_k w[k] * dpre[t+W-1-k]
//   dw[k]  = sum_t dpre[t] * x[t-W+1+k]            dbias = sum_t dpre[t]
// each sum over positions of one segment only.  A few operations per element:
// the floor is the bytes (x in, y out; x, dy in, dx out).
//
// A thread takes a few neighbouring channels (16 bytes of x; fewer for the
// gradient, whose registers hold four values per tap) and walks a run of
// tokens with the last inputs in registers, so x is read once but for the
// width - 1 tokens before the run.  Runs are as long as leaves the machine
// enough warps.  A tap j tokens back takes part while j <= t - (start of t's
// segment): a uniform predicate, and no masked value is ever multiplied.  The
// gradient recomputes pre, runs width - 1 tokens past its end for dx, and
// leaves its sums over tokens as one partial row per run, which a second
// kernel adds in order.
#include <algorithm>

#include "sc_seq.cuh"
#include "sc_seq_launch.h"

namespace scg {

namespace {

constexpr int kNT = 128;

// N channels from c on (kVec: aligned and whole), zeros beyond.
template <class T, int N, bool kVec>
__device__ __forceinline__ void load_ch(const T* p, long long left, float (&v)[N]) {
    if constexpr (kVec) {
        Vec<T, N> q;
        q.load(p);
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = q.get(i);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = i < left ? to_f32(__ldg(p + i)) : 0.0f;
    }
}
template <class T, int N, bool kVec>
__device__ __forceinline__ void store_ch(T* p, long long left, const float (&v)[N]) {
    if constexpr (kVec) {
        Vec<T, N> q;
        q.set(v);
        q.store(p);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i < left) p[i] = from_f32<T>(v[i]);
    }
}

// Start of the segment that holds token t, or anything at or below t - reach
// when it lies further back (heads == nullptr: the row has no segment starts).
__device__ __forceinline__ long long segment_start(const uint8_t* heads, long long t, int reach) {
    if (heads)
        for (long long q = t; q > t - reach && q >= 0; --q)
            if (heads[q]) return q;
    return -(1ll << 40);
}

// Input at position t of a row, t < 0: the state's (zeros without one).
template <class T, int N, bool kVec>
__device__ __forceinline__ void load_x(const ConvParams& p, const T* row, long long b, long long c, long long t,
                                       long long left, float (&v)[N]) {
    if (t >= 0) {
        load_ch<T, N, kVec>(row + t * p.x_token, left, v);
    } else if (p.state && t >= 1 - p.width) {
        load_ch<T, N, kVec>(static_cast<const T*>(p.state) + (b * (p.width - 1) + t + p.width - 1) * p.channels + c, left,
                            v);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = 0.0f;
    }
}

// Weights of N channels: w[k] meets the input WD - 1 - k tokens back (taps
// further back than width - 1: not used).
template <class T, int WD, int N>
__device__ __forceinline__ void load_weights(const ConvParams& p, long long c, long long left, float (&w)[WD][N],
                                             float (&bias)[N]) {
    const T* src = static_cast<const T*>(p.weight);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        bias[i] = p.bias && i < left ? to_f32(static_cast<const T*>(p.bias)[c + i]) : 0.0f;
#pragma unroll
        for (int k = 0; k < WD; ++k) {
            const int tap = k - (WD - p.width);
            w[k][i] = tap >= 0 && i < left ? to_f32(src[(c + i) * p.width + tap]) : 0.0f;
        }
    }
}

// pre at a token: `win` the WD - 1 inputs before it, `lim` how many of them count.
template <int WD, int N>
__device__ __forceinline__ void convolve(const float (&w)[WD][N], const float (&bias)[N], const float (&win)[WD - 1][N],
                                         const float (&x)[N], int lim, float (&pre)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) pre[i] = fmaf(w[WD - 1][i], x[i], bias[i]);
#pragma unroll
    for (int j = 1; j < WD; ++j)
        if (j <= lim)
#pragma unroll
            for (int i = 0; i < N; ++i) pre[i] = fmaf(w[WD - 1 - j][i], win[WD - 1 - j][i], pre[i]);
}

template <int WD, int N>
__device__ __forceinline__ void slide(float (&win)[WD - 1][N], const float (&x)[N]) {
#pragma unroll
    for (int k = 0; k + 1 < WD - 1; ++k)
#pragma unroll
        for (int i = 0; i < N; ++i) win[k][i] = win[k + 1][i];
#pragma unroll
    for (int i = 0; i < N; ++i) win[WD - 2][i] = x[i];
}

// A CTA's place in the flat grid: channel block, run of tokens, row.
struct Place {
    long long c, run, b;
    __device__ __forceinline__ Place(unsigned cblocks, unsigned runs, int n) {
        const unsigned q = blockIdx.x / cblocks;
        c = ((long long)(blockIdx.x % cblocks) * kNT + threadIdx.x) * n;
        run = q % runs;
        b = q / runs;
    }
};

// Thread: channels c .. c + N - 1, one run of tokens of one row.
template <class T, int WD, int N, bool kVec>
__global__ void __launch_bounds__(kNT) conv_kernel(ConvParams p, int run, unsigned cblocks, unsigned runs) {
    const Place at(cblocks, runs, N);
    const long long c = at.c, b = at.b;
    const long long left = p.channels - c;
    if (left <= 0) return;
    const long long t0 = at.run * run, t1 = min(t0 + run, p.length);
    const T* row = static_cast<const T*>(p.x) + b * p.x_batch + c;
    T* out = static_cast<T*>(p.y) + b * p.y_batch + c;
    const uint8_t* heads = p.heads ? p.heads + b * p.length : nullptr;
    float w[WD][N], bias[N], win[WD - 1][N];
    load_weights<T, WD, N>(p, c, left, w, bias);
#pragma unroll
    for (int k = 0; k < WD - 1; ++k) load_x<T, N, kVec>(p, row, b, c, t0 - (WD - 1) + k, left, win[k]);
    long long start = segment_start(heads, t0, WD);
    constexpr int U = 4;
    for (long long t = t0; t < t1; t += U) {
        float x[U][N];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (t + u < t1) load_ch<T, N, kVec>(row + (t + u) * p.x_token, left, x[u]);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (t + u < t1) {
                if (heads && heads[t + u]) start = t + u;
                const int lim = (int)min((long long)p.width - 1, t + u - start);
                float pre[N];
                convolve<WD, N>(w, bias, win, x[u], lim, pre);
                if (p.silu)
#pragma unroll
                    for (int i = 0; i < N; ++i) pre[i] *= sigmoid(pre[i]);
                store_ch<T, N, kVec>(out + (t + u) * p.y_token, left, pre);
                slide<WD, N>(win, x[u]);
            }
        }
    }
    if (p.final_state && t1 == p.length) {
        T* fs = static_cast<T*>(p.final_state) + b * (p.width - 1) * p.channels + c;
#pragma unroll
        for (int j = 1; j < WD; ++j) {  // the input j tokens before the end
            if (j < p.width) {
                float v[N];
                const bool in = p.length - j >= start;
#pragma unroll
                for (int i = 0; i < N; ++i) v[i] = in ? win[WD - 1 - j][i] : 0.0f;
                store_ch<T, N, kVec>(fs + (long long)(p.width - 1 - j) * p.channels, left, v);
            }
        }
    }
}

// Gradient over the same runs.  pend[k]: dx of the position WD - 1 - k tokens
// back, as far as it is summed.  partials[b * runs + run][width + 1][channels].
template <class T, int WD, int N, bool kVec>
__global__ void __launch_bounds__(kNT) conv_grad_kernel(ConvParams p, int run, unsigned cblocks, unsigned runs) {
    const Place at(cblocks, runs, N);
    const long long c = at.c, b = at.b;
    const long long left = p.channels - c;
    if (left <= 0) return;
    const long long t0 = at.run * run, t1 = min(t0 + run, p.length);
    const long long end = min(t1 + p.width - 1, p.length);  // the tokens whose dpre reaches this run
    const T* row = static_cast<const T*>(p.x) + b * p.x_batch + c;
    const T* dyr = static_cast<const T*>(p.dy) + b * p.dy_batch + c;
    T* dxr = p.dx ? static_cast<T*>(p.dx) + b * p.dx_batch + c : nullptr;
    const uint8_t* heads = p.heads ? p.heads + b * p.length : nullptr;
    float w[WD][N], bias[N], win[WD - 1][N], pend[WD][N], dw[WD][N], db[N];
    load_weights<T, WD, N>(p, c, left, w, bias);
#pragma unroll
    for (int k = 0; k < WD - 1; ++k) load_x<T, N, kVec>(p, row, b, c, t0 - (WD - 1) + k, left, win[k]);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        db[i] = 0.0f;
#pragma unroll
        for (int k = 0; k < WD; ++k) pend[k][i] = dw[k][i] = 0.0f;
    }
    long long start = segment_start(heads, t0, WD);
    // a position's dx is complete WD - 1 tokens later: the loop runs on past
    // `end` with no more terms until the run's last one has been stored
    constexpr int U = 4;
    for (long long t = t0; t < t1 + WD - 1; t += U) {
        float x[U][N], dy[U][N];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (t + u < end) {
                load_ch<T, N, kVec>(row + (t + u) * p.x_token, left, x[u]);
                load_ch<T, N, kVec>(dyr + (t + u) * p.dy_token, left, dy[u]);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const long long s = t + u;
            if (s < t1 + WD - 1) {
#pragma unroll
                for (int i = 0; i < N; ++i) {
#pragma unroll
                    for (int k = 0; k + 1 < WD; ++k) pend[k][i] = pend[k + 1][i];
                    pend[WD - 1][i] = 0.0f;
                }
                if (s < end) {
                    if (heads && heads[s]) start = s;
                    const int lim = (int)min((long long)p.width - 1, s - start);
                    float g[N];
                    if (p.silu) {
                        convolve<WD, N>(w, bias, win, x[u], lim, g);
#pragma unroll
                        for (int i = 0; i < N; ++i) {
                            const float sg = sigmoid(g[i]);
                            g[i] = dy[u][i] * sg * fmaf(g[i], 1.0f - sg, 1.0f);
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < N; ++i) g[i] = dy[u][i];
                    }
#pragma unroll
                    for (int i = 0; i < N; ++i) pend[WD - 1][i] = w[WD - 1][i] * g[i];
#pragma unroll
                    for (int j = 1; j < WD; ++j)
                        if (j <= lim)
#pragma unroll
                            for (int i = 0; i < N; ++i)
                                pend[WD - 1 - j][i] = fmaf(w[WD - 1 - j][i], g[i], pend[WD - 1 - j][i]);
                    if (s < t1) {
#pragma unroll
                        for (int i = 0; i < N; ++i) {
                            db[i] += g[i];
                            dw[WD - 1][i] = fmaf(g[i], x[u][i], dw[WD - 1][i]);
                        }
#pragma unroll
                        for (int j = 1; j < WD; ++j)
                            if (j <= lim)
#pragma unroll
                                for (int i = 0; i < N; ++i)
                                    dw[WD - 1 - j][i] = fmaf(g[i], win[WD - 1 - j][i], dw[WD - 1 - j][i]);
                    }
                    slide<WD, N>(win, x[u]);
                }
                const long long q = s - (WD - 1);  // complete
                if (q >= t0 && dxr) store_ch<T, N, kVec>(dxr + q * p.dx_token, left, pend[0]);
                if (q < 0 && t0 == 0 && q >= 1 - p.width && p.dstate)
                    store_ch<T, N, kVec>(static_cast<T*>(p.dstate) +
                                             (b * (p.width - 1) + q + p.width - 1) * p.channels + c,
                                         left, pend[0]);
            }
        }
    }
    if (p.partials) {
        float* part = p.partials + ((b * runs + at.run) * (p.width + 1)) * p.channels + c;
#pragma unroll
        for (int k = 0; k <= WD; ++k) {
            const int tap = k == WD ? p.width : k - (WD - p.width);
            if (tap >= 0)
#pragma unroll
                for (int i = 0; i < N; ++i)
                    if (i < left) part[(long long)tap * p.channels + i] = k == WD ? db[i] : dw[k == WD ? 0 : k][i];
        }
    }
}

// dweight and dbias: the partial rows added in order.
__global__ void __launch_bounds__(kNT) conv_sum_kernel(ConvParams p, long long rows) {
    const long long n = (p.width + 1) * p.channels, i = (long long)blockIdx.x * kNT + threadIdx.x;
    if (i >= n) return;
    const float* src = p.partials + i;
    float sum = 0.0f;
    long long r = 0;
    for (; r + 8 <= rows; r += 8) {
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = __ldg(src + (r + j) * n);
        sum += ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
    }
    for (; r < rows; ++r) sum += __ldg(src + r * n);
    const long long tap = i / p.channels, c = i % p.channels;
    if (tap < p.width) {
        if (p.dweight) p.dweight[c * p.width + tap] = sum;
    } else if (p.dbias) {
        p.dbias[c] = sum;
    }
}

// One token of one row: its window is the slot's state and x.
template <class T, int N, bool kVec>
__global__ void __launch_bounds__(kNT) conv_step_kernel(ConvParams p, unsigned cblocks) {
    const Place at(cblocks, 1, N);
    const long long c = at.c, b = at.b;
    const long long left = p.channels - c;
    if (left <= 0) return;
    const long long slot = p.slots ? (long long)__ldg(p.slots + b) : b;
    T* out = static_cast<T*>(p.y) + b * p.y_batch + c;
    float pre[N];
    if (slot < 0 || slot >= p.pool_rows) {
#pragma unroll
        for (int i = 0; i < N; ++i) pre[i] = 0.0f;
        store_ch<T, N, kVec>(out, left, pre);
        return;
    }
    const T* wt = static_cast<const T*>(p.weight) + c * p.width;
    T* st = static_cast<T*>(p.pool) + slot * (p.width - 1) * p.channels + c;
#pragma unroll
    for (int i = 0; i < N; ++i) pre[i] = p.bias && i < left ? to_f32(static_cast<const T*>(p.bias)[c + i]) : 0.0f;
    float x[N];
    load_ch<T, N, kVec>(static_cast<const T*>(p.x) + b * p.x_batch + c, left, x);
    // every thread reads the rows of its own channels before it writes them
    for (int k = 0; k < p.width - 1; ++k) {
        float v[N];
        if constexpr (kVec) {
            Vec<T, N> q;
            q.load_rw(st + (long long)k * p.channels);
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] = q.get(i);
            if (k > 0) q.store(st + (long long)(k - 1) * p.channels);
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                v[i] = 0.0f;
                if (i < left) {
                    const T e = st[(long long)k * p.channels + i];
                    v[i] = to_f32(e);
                    if (k > 0) st[(long long)(k - 1) * p.channels + i] = e;
                }
            }
        }
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i < left) pre[i] = fmaf(to_f32(wt[(long long)i * p.width + k]), v[i], pre[i]);
    }
    if (p.width > 1) store_ch<T, N, kVec>(st + (long long)(p.width - 2) * p.channels, left, x);
#pragma unroll
    for (int i = 0; i < N; ++i)
        if (i < left) {
            pre[i] = fmaf(to_f32(wt[(long long)i * p.width + p.width - 1]), x[i], pre[i]);
            if (p.silu) pre[i] *= sigmoid(pre[i]);
        }
    store_ch<T, N, kVec>(out, left, pre);
}

long long ceil_div(long long a, long long b) { return (a + b - 1) / b; }

// Tokens per thread: the longest run up to `most` that leaves eight warps per
// SM, at least `least`.
int run_length(long long batch, long long length, long long channels, int n, int least, int most) {
    const long long warps = ceil_div(channels, 32ll * n) * std::max(batch, 1ll), want = 8ll * 152;
    int run = most;
    while (run > least && warps * ceil_div(length, run) < want) run /= 2;
    return run;
}

// Channels per thread: 16 bytes forward, 4 backward (2 beyond 4 taps).
template <class T> constexpr int kFwdCh = 16 / (int)sizeof(T);
constexpr int grad_channels(int width) { return width <= 4 ? 4 : 2; }
constexpr int kGradLeast = 8, kGradMost = 128;

template <class T, int WD>
cudaError_t conv_of(const ConvParams& p, cudaStream_t s) {
    constexpr int N = kFwdCh<T>;
    const int run = run_length(p.batch, p.length, p.channels, N, 8, 32);
    const unsigned cblocks = (unsigned)ceil_div(p.channels, (long long)kNT * N), runs = (unsigned)ceil_div(p.length, run);
    const unsigned grid = cblocks * runs * (unsigned)p.batch;
    if (p.vec) conv_kernel<T, WD, N, true><<<grid, kNT, 0, s>>>(p, run, cblocks, runs);
    else conv_kernel<T, WD, N, false><<<grid, kNT, 0, s>>>(p, run, cblocks, runs);
    return cudaGetLastError();
}

template <class T, int WD>
cudaError_t conv_grad_of(const ConvParams& p, cudaStream_t s) {
    constexpr int N = grad_channels(WD);
    const int run = run_length(p.batch, p.length, p.channels, N, kGradLeast, kGradMost);
    const unsigned cblocks = (unsigned)ceil_div(p.channels, (long long)kNT * N), runs = (unsigned)ceil_div(p.length, run);
    const unsigned grid = cblocks * runs * (unsigned)p.batch;
    if (p.vec) conv_grad_kernel<T, WD, N, true><<<grid, kNT, 0, s>>>(p, run, cblocks, runs);
    else conv_grad_kernel<T, WD, N, false><<<grid, kNT, 0, s>>>(p, run, cblocks, runs);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !p.partials) return e;
    conv_sum_kernel<<<(unsigned)ceil_div((p.width + 1) * p.channels, kNT), kNT, 0, s>>>(
        p, p.batch * ceil_div(p.length, run));
    return cudaGetLastError();
}

template <class T>
cudaError_t conv_step_of(const ConvParams& p, cudaStream_t s) {
    constexpr int N = kFwdCh<T>;
    const unsigned cblocks = (unsigned)ceil_div(p.channels, (long long)kNT * N), grid = cblocks * (unsigned)p.batch;
    if (p.vec) conv_step_kernel<T, N, true><<<grid, kNT, 0, s>>>(p, cblocks);
    else conv_step_kernel<T, N, false><<<grid, kNT, 0, s>>>(p, cblocks);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_conv(int dtype, const ConvParams& p, cudaStream_t s) {
    count_launches(1);
    const bool wide = p.width > 4;
    switch (dtype) {
    case SC_F32: return wide ? conv_of<float, 8>(p, s) : conv_of<float, 4>(p, s);
    case SC_F16: return wide ? conv_of<f16, 8>(p, s) : conv_of<f16, 4>(p, s);
    case SC_BF16: return wide ? conv_of<bf16, 8>(p, s) : conv_of<bf16, 4>(p, s);
    default: return cudaErrorInvalidValue;
    }
}

size_t conv_grad_scratch(long long batch, long long length, long long channels, int width) {
    const int run = run_length(batch, length, channels, grad_channels(width), kGradLeast, kGradMost);
    return (size_t)batch * (size_t)ceil_div(length, run) * (size_t)(width + 1) * (size_t)channels * 4;
}

cudaError_t launch_conv_grad(int dtype, const ConvParams& p, cudaStream_t s) {
    count_launches(p.partials ? 2 : 1);
    const bool wide = p.width > 4;
    switch (dtype) {
    case SC_F32: return wide ? conv_grad_of<float, 8>(p, s) : conv_grad_of<float, 4>(p, s);
    case SC_F16: return wide ? conv_grad_of<f16, 8>(p, s) : conv_grad_of<f16, 4>(p, s);
    case SC_BF16: return wide ? conv_grad_of<bf16, 8>(p, s) : conv_grad_of<bf16, 4>(p, s);
    default: return cudaErrorInvalidValue;
    }
}

cudaError_t launch_conv_step(int dtype, const ConvParams& p, cudaStream_t s) {
    count_launches(1);
    switch (dtype) {
    case SC_F32: return conv_step_of<float>(p, s);
    case SC_F16: return conv_step_of<f16>(p, s);
    case SC_BF16: return conv_step_of<bf16>(p, s);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace scg
