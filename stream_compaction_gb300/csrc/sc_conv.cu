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
// A thread takes four neighbouring channels and walks a run of tokens with the
// last inputs in registers, so x is read once but for the width - 1 tokens
// before the run.  The raw elements of the next kAhead tokens are on their way
// while kAhead are worked on: with the machine's threads that keeps enough
// bytes under way for the memory's latency.  Runs are as long as leaves the
// machine enough warps.  A tap j tokens back takes part while j < width and, in
// packed rows, j <= t - (start of t's segment): uniform conditions, and no masked
// value is ever multiplied.  The gradient recomputes pre, runs width - 1 tokens
// past its end for dx, and leaves its sums over tokens as one partial row per
// run, which a second kernel adds in order.
//
// 8 x 4096 tokens, 4096 channels, width 4, SiLU, bfloat16: forward 97 us (5.5 TB/s, 81 %
// of a copy's rate), gradient 206 (3.9 TB/s), its sums 7; float32 forward 184 (5.8
// TB/s).  No unit is full in the gradient: it issues in 56 % of its slots with 10 warps
// an SM (144 registers allow 12), and DRAM is a third busy: too few warps to hide one
// another's waits.  The forward kernel issues in 60 % with 20 warps.  With two channels
// a thread and no loads ahead: 818 us for the three, 310 so.
#include <algorithm>

#include "sc_seq.cuh"
#include "sc_seq_launch.h"

namespace scg {

namespace {

constexpr int kNT = 128;
constexpr int kCh = 4;     // channels per thread, in two pairs
constexpr int kAhead = 4;  // tokens

// Four channels from c on, as they lie in memory; zeros beyond `left` (kVec:
// aligned, and all there).
template <class T, bool kVec>
struct Four;
template <class T>
struct Four<T, true> {
    Vec<T, 4> v;
    __device__ __forceinline__ void load(const T* p, long long) { v.load(p); }
    __device__ __forceinline__ void zero() { v.zero(); }
    __device__ __forceinline__ f2 pair(int i) const { return v.pair(i); }
    __device__ __forceinline__ static void store(T* p, long long, const f2 (&f)[2]) {
        Vec<T, 4> q;
        q.set_pairs(f);
        q.store(p);
    }
};
template <class T>
struct Four<T, false> {
    T v[4];
    __device__ __forceinline__ void load(const T* p, long long left) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = i < left ? __ldg(p + i) : from_f32<T>(0.0f);
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = from_f32<T>(0.0f);
    }
    __device__ __forceinline__ f2 pair(int i) const { return pack2(to_f32(v[2 * i]), to_f32(v[2 * i + 1])); }
    __device__ __forceinline__ static void store(T* p, long long left, const f2 (&f)[2]) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < left) p[i] = from_f32<T>(i & 1 ? hi2(f[i / 2]) : lo2(f[i / 2]));
    }
};

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

// Start of the segment that holds token t, or anything at or below t - reach
// when it lies further back.
__device__ __forceinline__ long long segment_start(const uint8_t* heads, long long t, int reach) {
    for (long long q = t; q > t - reach && q >= 0; --q)
        if (heads[q]) return q;
    return -(1ll << 40);
}

// The filter of four channels and its last inputs.  w[k] meets the input
// WD - 1 - k tokens back; taps further back than width - 1 are not used.
template <class T, int WD, bool kVec>
struct Filter {
    f2 w[WD][2], bias[2], win[WD - 1][2];
    __device__ __forceinline__ Filter(const ConvParams& p, const T* row, long long b, long long c, long long t0,
                                      long long left) {
        const T* src = static_cast<const T*>(p.weight) + c * p.width;
        float v[WD + 1][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[WD][i] = p.bias && i < left ? to_f32(static_cast<const T*>(p.bias)[c + i]) : 0.0f;
#pragma unroll
            for (int k = 0; k < WD; ++k) {
                const int tap = k - (WD - p.width);
                v[k][i] = tap >= 0 && i < left ? to_f32(src[i * p.width + tap]) : 0.0f;
            }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            bias[i] = pack2(v[WD][2 * i], v[WD][2 * i + 1]);
#pragma unroll
            for (int k = 0; k < WD; ++k) w[k][i] = pack2(v[k][2 * i], v[k][2 * i + 1]);
        }
#pragma unroll
        for (int k = 0; k < WD - 1; ++k) {  // the inputs before t0: x, the state, or zeros
            const long long t = t0 - (WD - 1) + k;
            Four<T, kVec> q;
            q.zero();
            if (t >= 0) q.load(row + t * p.x_token, left);
            else if (p.state && t >= 1 - p.width)
                q.load(static_cast<const T*>(p.state) + (b * (p.width - 1) + t + p.width - 1) * p.channels + c, left);
            win[k][0] = q.pair(0);
            win[k][1] = q.pair(1);
        }
    }
    // pre at a token with input x, of which `lim` inputs before it count
    __device__ __forceinline__ void apply(const f2 (&x)[2], int lim, f2 (&pre)[2]) const {
#pragma unroll
        for (int i = 0; i < 2; ++i) pre[i] = fma2(w[WD - 1][i], x[i], bias[i]);
#pragma unroll
        for (int j = 1; j < WD; ++j)
            if (j <= lim)
#pragma unroll
                for (int i = 0; i < 2; ++i) pre[i] = fma2(w[WD - 1 - j][i], win[WD - 1 - j][i], pre[i]);
    }
    __device__ __forceinline__ void slide(const f2 (&x)[2]) {
#pragma unroll
        for (int k = 0; k + 1 < WD - 1; ++k)
#pragma unroll
            for (int i = 0; i < 2; ++i) win[k][i] = win[k + 1][i];
#pragma unroll
        for (int i = 0; i < 2; ++i) win[WD - 2][i] = x[i];
    }
};

// CTAs an SM that the forward kernel's registers leave room for, where rows are
// aligned and not packed and the taps at most four.  16 bits: 8 (64 registers; the
// bfloat16 training case 312 us with its gradient, 320 with 4).  float32, whose elements
// ahead take twice the registers: 5 (94); 8 x 4096 x 4096, forward: 184 us with 5, 188
// with 4, 192 with 6, 238 with 8, which spills.
template <class T> constexpr int kFastCtas = sizeof(T) == 2 ? 8 : 5;

// Thread: channels c .. c + 3, one run of tokens of one row.
template <class T, int WD, bool kVec, bool kHeads>
__global__ void __launch_bounds__(kNT, WD == 4 && kVec && !kHeads ? kFastCtas<T> : 4)
    conv_kernel(ConvParams p, int run, unsigned cblocks, unsigned runs) {
    const Place at(cblocks, runs, kCh);
    const long long c = at.c, b = at.b, left = p.channels - c;
    if (left <= 0) return;
    const long long t0 = at.run * run, t1 = min(t0 + run, p.length);
    const T* row = static_cast<const T*>(p.x) + b * p.x_batch + c;
    T* out = static_cast<T*>(p.y) + b * p.y_batch + c + t0 * p.y_token;
    const uint8_t* heads = kHeads ? p.heads + b * p.length : nullptr;
    Four<T, kVec> next[kAhead];
    auto fetch = [&](long long t) {  // past the run: its last token, unused
#pragma unroll
        for (int u = 0; u < kAhead; ++u) next[u].load(row + min(t + u, t1 - 1) * p.x_token, left);
    };
    fetch(t0);
    Filter<T, WD, kVec> f(p, row, b, c, t0, left);
    long long start = kHeads ? segment_start(heads, t0, WD) : 0;
    int lim = p.width - 1;
    auto token = [&](const Four<T, kVec>& q, long long t) {
        f2 x[2] = {q.pair(0), q.pair(1)}, pre[2];
        if (kHeads) {
            if (heads[t]) start = t;
            lim = (int)min((long long)p.width - 1, t - start);
        }
        f.apply(x, lim, pre);
        if (p.silu) {
            pre[0] = mul2(pre[0], sigmoid_2<T>(pre[0]));
            pre[1] = mul2(pre[1], sigmoid_2<T>(pre[1]));
        }
        Four<T, kVec>::store(out, left, pre);
        out += p.y_token;
        f.slide(x);
    };
    for (long long t = t0; t < t1; t += kAhead) {
        Four<T, kVec> now[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) now[u] = next[u];
        if (t + kAhead < t1) fetch(t + kAhead);
        if (t + kAhead <= t1) {
#pragma unroll
            for (int u = 0; u < kAhead; ++u) token(now[u], t + u);
        } else {
#pragma unroll
            for (int u = 0; u < kAhead; ++u)
                if (t + u < t1) token(now[u], t + u);
        }
    }
    if (p.final_state && t1 == p.length) {
        T* fs = static_cast<T*>(p.final_state) + b * (p.width - 1) * p.channels + c;
#pragma unroll
        for (int j = 1; j < WD; ++j) {  // the input j tokens before the end
            if (j < p.width) {
                const bool in = !kHeads || p.length - j >= start;
                const f2 v[2] = {in ? f.win[WD - 1 - j][0] : 0ull, in ? f.win[WD - 1 - j][1] : 0ull};
                Four<T, kVec>::store(fs + (long long)(p.width - 1 - j) * p.channels, left, v);
            }
        }
    }
}

// Gradient over the same runs.  pend[k]: dx of the position WD - 1 - k tokens
// back, as far as it is summed.  partials[b * runs + run][width + 1][channels].
template <class T, int WD, bool kVec, bool kHeads>
__global__ void __launch_bounds__(kNT) conv_grad_kernel(ConvParams p, int run, unsigned cblocks, unsigned runs) {
    const Place at(cblocks, runs, kCh);
    const long long c = at.c, b = at.b, left = p.channels - c;
    if (left <= 0) return;
    const long long t0 = at.run * run, t1 = min(t0 + run, p.length);
    const long long end = min(t1 + p.width - 1, p.length);  // the tokens whose dpre reaches this run
    const T* row = static_cast<const T*>(p.x) + b * p.x_batch + c;
    const T* dyr = static_cast<const T*>(p.dy) + b * p.dy_batch + c;
    T* dxr = p.dx ? static_cast<T*>(p.dx) + b * p.dx_batch + c : nullptr;
    const uint8_t* heads = kHeads ? p.heads + b * p.length : nullptr;
    Four<T, kVec> nx[kAhead], ng[kAhead];
    auto fetch = [&](long long t) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const long long q = min(t + u, end - 1);
            nx[u].load(row + q * p.x_token, left);
            ng[u].load(dyr + q * p.dy_token, left);
        }
    };
    fetch(t0);
    Filter<T, WD, kVec> f(p, row, b, c, t0, left);
    f2 pend[WD][2], dw[WD][2], db[2] = {0ull, 0ull};
#pragma unroll
    for (int k = 0; k < WD; ++k)
#pragma unroll
        for (int i = 0; i < 2; ++i) pend[k][i] = dw[k][i] = 0ull;
    long long start = kHeads ? segment_start(heads, t0, WD) : 0;
    int lim = p.width - 1;
    // token s: its terms (kOwn: of the sums over the run's tokens too), and dx of
    // the position WD - 1 tokens back, which has got all of its own
    auto shift = [&]() {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
            for (int k = 0; k + 1 < WD; ++k) pend[k][i] = pend[k + 1][i];
            pend[WD - 1][i] = 0ull;
        }
    };
    auto terms = [&](const Four<T, kVec>& qx, const Four<T, kVec>& qg, long long s, bool own) {
        const f2 x[2] = {qx.pair(0), qx.pair(1)};
        f2 g[2] = {qg.pair(0), qg.pair(1)};
        if (kHeads) {
            if (heads[s]) start = s;
            lim = (int)min((long long)p.width - 1, s - start);
        }
        if (p.silu) {
            f2 pre[2];
            f.apply(x, lim, pre);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const f2 sg = sigmoid_2<T>(pre[i]);
                g[i] = mul2(mul2(g[i], sg), fma2(pre[i], fma2(sg, both(-1.0f), both(1.0f)), both(1.0f)));
            }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) pend[WD - 1][i] = mul2(f.w[WD - 1][i], g[i]);
#pragma unroll
        for (int j = 1; j < WD; ++j)
            if (j <= lim)
#pragma unroll
                for (int i = 0; i < 2; ++i) pend[WD - 1 - j][i] = fma2(f.w[WD - 1 - j][i], g[i], pend[WD - 1 - j][i]);
        if (own) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                db[i] = add2(db[i], g[i]);
                dw[WD - 1][i] = fma2(g[i], x[i], dw[WD - 1][i]);
            }
#pragma unroll
            for (int j = 1; j < WD; ++j)
                if (j <= lim)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        dw[WD - 1 - j][i] = fma2(g[i], f.win[WD - 1 - j][i], dw[WD - 1 - j][i]);
        }
        f.slide(x);
    };
    auto finish = [&](long long q) {
        if (q >= t0) {
            if (dxr) Four<T, kVec>::store(dxr + q * p.dx_token, left, pend[0]);
        } else if (q < 0 && t0 == 0 && q >= 1 - p.width && p.dstate) {
            Four<T, kVec>::store(static_cast<T*>(p.dstate) + (b * (p.width - 1) + q + p.width - 1) * p.channels + c, left,
                                 pend[0]);
        }
    };
    // the loop runs on past `end`, with no more terms, until the run's last dx is complete
    for (long long t = t0; t < t1 + WD - 1; t += kAhead) {
        Four<T, kVec> x[kAhead], g[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            x[u] = nx[u];
            g[u] = ng[u];
        }
        if (t + kAhead < end) fetch(t + kAhead);
        if (t - (WD - 1) >= t0 && t + kAhead <= t1 && dxr) {  // whole steps inside the run
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                shift();
                terms(x[u], g[u], t + u, true);
                Four<T, kVec>::store(dxr + (t + u - (WD - 1)) * p.dx_token, left, pend[0]);
            }
        } else {
#pragma unroll 1
            for (int u = 0; u < kAhead; ++u) {
                const long long s = t + u;
                if (s >= t1 + WD - 1) break;
                shift();
                // (x[u] with a running index would have to lie in memory)
                const Four<T, kVec> xu = u == 0 ? x[0] : u == 1 ? x[1] : u == 2 ? x[2] : x[3];
                const Four<T, kVec> gu = u == 0 ? g[0] : u == 1 ? g[1] : u == 2 ? g[2] : g[3];
                if (s < end) terms(xu, gu, s, s < t1);
                finish(s - (WD - 1));
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
                for (int i = 0; i < 4; ++i) {
                    const f2 v = k == WD ? db[i / 2] : dw[k == WD ? 0 : k][i / 2];
                    if (i < left) part[(long long)tap * p.channels + i] = i & 1 ? hi2(v) : lo2(v);
                }
        }
    }
}

// dweight and dbias: the partial rows added in order, by kSumParts threads a
// column, each a stretch of the rows.
constexpr int kSumCols = 32, kSumParts = 8;
__global__ void __launch_bounds__(kSumCols * kSumParts) conv_sum_kernel(ConvParams p, long long rows) {
    __shared__ float s_sum[kSumParts][kSumCols];
    const long long n = (p.width + 1) * p.channels, i = (long long)blockIdx.x * kSumCols + threadIdx.x % kSumCols;
    const int part = threadIdx.x / kSumCols;
    const long long per = (rows + kSumParts - 1) / kSumParts, end = min((part + 1) * per, rows);
    float sum = 0.0f;
    if (i < n) {
        const float* src = p.partials + i;
        long long r = part * per;
        for (; r + 8 <= end; r += 8) {
            float v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = __ldg(src + (r + j) * n);
            sum += ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
        }
        for (; r < end; ++r) sum += __ldg(src + r * n);
    }
    s_sum[part][threadIdx.x % kSumCols] = sum;
    __syncthreads();
    if (part != 0 || i >= n) return;
#pragma unroll
    for (int q = 1; q < kSumParts; ++q) sum += s_sum[q][threadIdx.x];
    const long long tap = i / p.channels, c = i % p.channels;
    if (tap < p.width) {
        if (p.dweight) p.dweight[c * p.width + tap] = sum;
    } else if (p.dbias) {
        p.dbias[c] = sum;
    }
}

// One token of one row: its window is the slot's state and x.  Every load is
// under way before the first product.
template <class T, int WD, bool kVec>
__global__ void __launch_bounds__(kNT) conv_step_kernel(ConvParams p, unsigned cblocks) {
    const Place at(cblocks, 1, kCh);
    const long long c = at.c, b = at.b, left = p.channels - c;
    if (left <= 0) return;
    const long long slot = p.slots ? (long long)__ldg(p.slots + b) : b;
    T* out = static_cast<T*>(p.y) + b * p.y_batch + c;
    if (slot < 0 || slot >= p.pool_rows) {
        const f2 none[2] = {0ull, 0ull};
        Four<T, kVec>::store(out, left, none);
        return;
    }
    T* st = static_cast<T*>(p.pool) + slot * (p.width - 1) * p.channels + c;
    const int pad = WD - p.width;  // rows of the window that there are not
    Four<T, kVec> win[WD];
#pragma unroll
    for (int k = 0; k < WD - 1; ++k) {
        win[k].zero();
        if (k >= pad) {
            const T* from = st + (long long)(k - pad) * p.channels;
            if constexpr (kVec) {
                win[k].v.load_rw(from);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (i < left) win[k].v[i] = from[i];
            }
        }
    }
    win[WD - 1].load(static_cast<const T*>(p.x) + b * p.x_batch + c, left);
    const T* src = static_cast<const T*>(p.weight) + c * p.width;
    float w[4][WD], bias[4];
    if (kVec && p.width == WD) {  // the four filters lie together
        Vec<T, 4 * WD> q;
        q.load(src);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int k = 0; k < WD; ++k) w[i][k] = q.get(i * WD + k);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int k = 0; k < WD; ++k) w[i][k] = k >= pad && i < left ? to_f32(src[i * p.width + k - pad]) : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) bias[i] = p.bias && i < left ? to_f32(static_cast<const T*>(p.bias)[c + i]) : 0.0f;
    f2 pre[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        pre[i] = pack2(bias[2 * i], bias[2 * i + 1]);
#pragma unroll
        for (int k = 0; k < WD; ++k)
            if (k >= pad) pre[i] = fma2(pack2(w[2 * i][k], w[2 * i + 1][k]), win[k].pair(i), pre[i]);
        if (p.silu) pre[i] = mul2(pre[i], sigmoid_2<T>(pre[i]));
    }
    Four<T, kVec>::store(out, left, pre);
#pragma unroll
    for (int k = 0; k < WD - 1; ++k)
        if (k >= pad) {
            const f2 v[2] = {win[k + 1].pair(0), win[k + 1].pair(1)};
            Four<T, kVec>::store(st + (long long)(k - pad) * p.channels, left, v);
        }
}

long long ceil_div(long long a, long long b) { return (a + b - 1) / b; }

// Tokens per thread: the longest run up to `most` that leaves eight warps per
// SM, at least `least`.
int run_length(long long batch, long long length, long long channels, int n, int least, int most) {
    const long long warps = ceil_div(channels, 32ll * n) * std::max(batch, 1ll), want = 8 * seq_sms();
    int run = most;
    while (run > least && warps * ceil_div(length, run) < want) run /= 2;
    return run;
}

// Tokens of a run: 8 x 4096 x 4096 bfloat16, forward and gradient, took 345 us
// with at most 32 and 64, 325 with 64 and 128, 320 with 64 and 256, 342 with 256
// and 256 (and 312 with the forward kernel held to 64 registers).
constexpr int kLeast = 8, kMost = 64;
constexpr int kGradLeast = 8, kGradMost = 256;

template <class T, int WD>
cudaError_t conv_of(const ConvParams& p, cudaStream_t s) {
    const int run = run_length(p.batch, p.length, p.channels, kCh, kLeast, kMost);
    const unsigned cblocks = (unsigned)ceil_div(p.channels, kNT * kCh), runs = (unsigned)ceil_div(p.length, run);
    const unsigned grid = cblocks * runs * (unsigned)p.batch;
    auto go = [&](auto kernel) { kernel<<<grid, kNT, 0, s>>>(p, run, cblocks, runs); };
    if (p.heads) p.vec ? go(conv_kernel<T, WD, true, true>) : go(conv_kernel<T, WD, false, true>);
    else p.vec ? go(conv_kernel<T, WD, true, false>) : go(conv_kernel<T, WD, false, false>);
    return cudaGetLastError();
}

template <class T, int WD>
cudaError_t conv_grad_of(const ConvParams& p, cudaStream_t s) {
    const int run = run_length(p.batch, p.length, p.channels, kCh, kGradLeast, kGradMost);
    const unsigned cblocks = (unsigned)ceil_div(p.channels, kNT * kCh), runs = (unsigned)ceil_div(p.length, run);
    const unsigned grid = cblocks * runs * (unsigned)p.batch;
    auto go = [&](auto kernel) { kernel<<<grid, kNT, 0, s>>>(p, run, cblocks, runs); };
    if (p.heads) p.vec ? go(conv_grad_kernel<T, WD, true, true>) : go(conv_grad_kernel<T, WD, false, true>);
    else p.vec ? go(conv_grad_kernel<T, WD, true, false>) : go(conv_grad_kernel<T, WD, false, false>);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !p.partials) return e;
    conv_sum_kernel<<<(unsigned)ceil_div((p.width + 1) * p.channels, kSumCols), kSumCols * kSumParts, 0, s>>>(
        p, p.batch * ceil_div(p.length, run));
    return cudaGetLastError();
}

template <class T, int WD>
cudaError_t conv_step_of(const ConvParams& p, cudaStream_t s) {
    const unsigned cblocks = (unsigned)ceil_div(p.channels, kNT * kCh), grid = cblocks * (unsigned)p.batch;
    if (p.vec) conv_step_kernel<T, WD, true><<<grid, kNT, 0, s>>>(p, cblocks);
    else conv_step_kernel<T, WD, false><<<grid, kNT, 0, s>>>(p, cblocks);
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
    const int run = run_length(batch, length, channels, kCh, kGradLeast, kGradMost);
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
    const bool wide = p.width > 4;
    switch (dtype) {
    case SC_F32: return wide ? conv_step_of<float, 8>(p, s) : conv_step_of<float, 4>(p, s);
    case SC_F16: return wide ? conv_step_of<f16, 8>(p, s) : conv_step_of<f16, 4>(p, s);
    case SC_BF16: return wide ? conv_step_of<bf16, 8>(p, s) : conv_step_of<bf16, 4>(p, s);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace scg
