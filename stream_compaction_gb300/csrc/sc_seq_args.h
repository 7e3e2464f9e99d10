// What the C entry points of the sequence operators check their arguments with:
// extents, strides, alignment, and whether outputs share memory.
#pragma once
#include <algorithm>
#include <cstdint>
#include <cstring>
#include <cuda_runtime.h>

#include "../../include/sc_seq.h"
#include "sc_seq_launch.h"

namespace scg {

constexpr int64_t kMaxGrid = 2147483647;

inline int bytes_of(int dtype) { return dtype == SC_F32 ? 4 : dtype == SC_F16 || dtype == SC_BF16 ? 2 : 0; }
inline bool multiple(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
inline cudaStream_t cu(sc_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

// a * b * c * d, or -1 beyond 2^60 (all at least 0).
inline int64_t product(int64_t a, int64_t b, int64_t c = 1, int64_t d = 1) {
    const __int128 lim = (__int128)1 << 60;
    __int128 v = (__int128)a * b;
    if (v > lim) return -1;
    v *= c;
    if (v > lim) return -1;
    v *= d;
    return v > lim ? -1 : (int64_t)v;
}

// A batch x tokens x channels tensor with free strides.
struct Tensor {
    const void* p = nullptr;
    int64_t batch = 0, tokens = 0, channels = 0, sb = 0, st = 0;
    int eb = 1;
    int64_t span() const {  // elements from the first to behind the last
        if (!batch || !tokens || !channels) return 0;
        const __int128 n = (__int128)(batch - 1) * sb + (__int128)(tokens - 1) * st + channels;
        return n > ((__int128)1 << 60) ? -1 : (int64_t)n;
    }
    bool ok() const { return p && multiple(p, eb) && sb >= 0 && st >= 0 && span() >= 0; }
    // every element has its own address
    bool distinct() const {
        const bool many_b = batch > 1, many_t = tokens > 1;
        if (many_t && st < channels) return false;
        if (many_b && sb < channels) return false;
        if (!many_b || !many_t) return true;
        return sb >= (__int128)(tokens - 1) * st + channels || st >= (__int128)(batch - 1) * sb + channels;
    }
    bool vec(int elems) const {
        return multiple(p, std::min(16, elems * eb)) && (batch <= 1 || sb % elems == 0) && (tokens <= 1 || st % elems == 0);
    }
};
inline Tensor flat(const void* p, int64_t n, int eb) { return {p, 1, 1, n, 0, 0, eb}; }

// Whether two tensors share memory; column slices of one joint buffer do not.
inline bool share(const Tensor& a, const Tensor& b) {
    const int64_t na = a.span(), nb = b.span();
    if (!a.p || !b.p || na <= 0 || nb <= 0) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    if (!(x < y + (uintptr_t)nb * b.eb && y < x + (uintptr_t)na * a.eb)) return false;
    const int64_t stride = a.tokens > 1 ? a.st : a.sb;
    if (a.eb == b.eb && stride > 0 && a.tokens == b.tokens && a.batch == b.batch && (a.tokens <= 1 || a.st == b.st) &&
        (a.batch <= 1 || (a.sb == b.sb && a.sb % stride == 0)) && (x - y) % a.eb == 0) {
        const int64_t diff = ((int64_t)(x - y)) / a.eb;            // a's first element behind b's
        const int64_t col = ((diff % stride) + stride) % stride;   // its column in b's rows
        if (col >= b.channels && col + a.channels <= stride) return false;
    }
    return true;
}

// Whether every output has its memory to itself: none shares it with an input or
// with another output.  The ranges of addresses decide nearly always.
template <int kOut, int kIn>
bool apart(const Tensor (&out)[kOut], const Tensor (&in)[kIn]) {
    const Tensor* all[kOut + kIn];
    uintptr_t lo[kOut + kIn], hi[kOut + kIn];
    int n = 0, outs = 0;
    auto add = [&](const Tensor& t) {
        const int64_t span = t.p ? t.span() : 0;
        if (span <= 0) return;
        all[n] = &t;
        lo[n] = reinterpret_cast<uintptr_t>(t.p);
        hi[n] = lo[n] + (uintptr_t)span * t.eb;
        ++n;
    };
    for (const Tensor& t : out) add(t);
    outs = n;
    for (const Tensor& t : in) add(t);
    for (int i = 0; i < outs; ++i)
        for (int j = i + 1; j < n; ++j)
            if (lo[i] < hi[j] && lo[j] < hi[i] && share(*all[i], *all[j])) return false;
    return true;
}

inline bool vec_row(int64_t dim, int64_t ld, const void* p, int elems, int64_t rows) {
    return multiple(p, 16) && dim % elems == 0 && (rows <= 1 || ld % elems == 0);
}

inline sc_status zero(void* p, size_t bytes, cudaStream_t s) {
    if (!p || !bytes) return SC_OK;
    return status_of(cudaMemsetAsync(p, 0, bytes, s));
}
// dst = src, or zeros without one
inline sc_status copy_or_zero(void* dst, const void* src, size_t bytes, cudaStream_t s) {
    if (!dst || !bytes || dst == src) return SC_OK;
    if (!src) return zero(dst, bytes, s);
    return status_of(cudaMemcpyAsync(dst, src, bytes, cudaMemcpyDeviceToDevice, s));
}

}  // namespace scg
