// Shared pieces of the sequence operators (embedding, convolution, selective
// scan): element types, 16-byte vector access, two-lane float32 arithmetic and
// the activation functions.  All arithmetic is float32; an element is rounded
// to its type once, when it is stored.
#pragma once
#include <cstdint>
#include <cstring>
#include <type_traits>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

namespace scg {

using bf16 = __nv_bfloat16;
using f16 = __half;

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(bf16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(f16 v) { return __half2float(v); }
template <class T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ bf16 from_f32<bf16>(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ f16 from_f32<f16>(float v) { return __float2half_rn(v); }

// Two float32 values in one 64-bit register pair; each operation rounds both.
using f2 = unsigned long long;
__device__ __forceinline__ f2 pack2(float lo, float hi) {
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ float lo2(f2 v) {
    return __uint_as_float((uint32_t)v);
}
__device__ __forceinline__ float hi2(f2 v) {
    return __uint_as_float((uint32_t)(v >> 32));
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
    f2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
    f2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
    f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ float ex2(float v) {  // 2^v
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ f2 ex2_2(f2 v) { return pack2(ex2(lo2(v)), ex2(hi2(v))); }

// N consecutive elements of T, moved in accesses of up to 16 bytes.
template <class T, int N>
struct Vec {
    static constexpr int kBytes = (int)sizeof(T) * N;
    static_assert(kBytes % 4 == 0, "whole 32-bit words");
    static constexpr int kWords = kBytes / 4;
    uint32_t w[kWords];
    template <class U, bool kConst>
    __device__ __forceinline__ void load_as(const T* p) {
        constexpr int per = (int)sizeof(U) / 4;
#pragma unroll
        for (int i = 0; i < kWords / per; ++i) {
            const U* q = reinterpret_cast<const U*>(p) + i;
            U v;
            if constexpr (kConst) v = __ldg(q);
            else v = *q;
            const uint32_t* e = reinterpret_cast<const uint32_t*>(&v);
#pragma unroll
            for (int j = 0; j < per; ++j) w[i * per + j] = e[j];
        }
    }
    template <bool kConst>
    __device__ __forceinline__ void load_any(const T* p) {
        if constexpr (kBytes % 16 == 0) load_as<uint4, kConst>(p);
        else if constexpr (kBytes % 8 == 0) load_as<uint2, kConst>(p);
        else load_as<uint32_t, kConst>(p);
    }
    __device__ __forceinline__ void load(const T* p) { load_any<true>(p); }      // read-only for the kernel
    __device__ __forceinline__ void load_rw(const T* p) { load_any<false>(p); }  // memory it also writes
    __device__ __forceinline__ void store(T* p) const {
        if constexpr (kBytes % 16 == 0) {
#pragma unroll
            for (int i = 0; i < kWords / 4; ++i)
                reinterpret_cast<uint4*>(p)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
        } else if constexpr (kBytes % 8 == 0) {
#pragma unroll
            for (int i = 0; i < kWords / 2; ++i) reinterpret_cast<uint2*>(p)[i] = make_uint2(w[2 * i], w[2 * i + 1]);
        } else {
#pragma unroll
            for (int i = 0; i < kWords; ++i) reinterpret_cast<uint32_t*>(p)[i] = w[i];
        }
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = 0u;
    }
    // element i as float32 (i known at compile time)
    __device__ __forceinline__ float get(int i) const {
        if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
        else return to_f32(reinterpret_cast<const T*>(&w[i / 2])[i % 2]);
    }
    // elements 2 i and 2 i + 1 as a pair
    __device__ __forceinline__ f2 pair(int i) const {
        if constexpr (sizeof(T) == 4) {
            return pack2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
        } else if constexpr (std::is_same<T, bf16>::value) {  // a bfloat16 is the upper half of a float32
            return pack2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
        } else {
            return pack2(get(2 * i), get(2 * i + 1));
        }
    }
    __device__ __forceinline__ void set_pairs(const f2 (&v)[N / 2]) {
        float f[N];
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            f[2 * i] = lo2(v[i]);
            f[2 * i + 1] = hi2(v[i]);
        }
        set(f);
    }
    __device__ __forceinline__ void set(const float* v) {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < N; ++i) w[i] = __float_as_uint(v[i]);
        } else {
#pragma unroll
            for (int i = 0; i < N; i += 2) {
                T e[2] = {from_f32<T>(v[i]), from_f32<T>(v[i + 1])};
                uint32_t u;
                memcpy(&u, e, 4);
                w[i / 2] = u;
            }
        }
    }
};

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// 2^(d A2): one step's decay.  A recurrence multiplies hundreds of them, so a
// mean error counts, not only its spread: the instruction's results lie low, by
// 0.5e-8 to 2.7e-8 of the result on average for arguments between -0.25 and 0
// (measured, by octave; its spread is 3e-8).  The exponent is nudged up by about
// that (1.7e-8 of the result), in the multiply-add that forms it anyway.  The
// gradient by A over 4096 tokens against 64 bits: 1.4e-6 off without, 0.6e-6 with
// it (correctly rounded exponentials: 0.3e-6).  Decays that are multiplied so often
// are those near 1.  With it, mean errors by octave of |d A|: between -1.6e-8 and
// 1.2e-8 from 2^-12 to 2, 0.7e-8 to 4, 4.6e-8 to 8, 1.3e-7 to 16, where the rounding
// of A log2(e) takes over (spread 3e-8 to 5e-8, 0.9e-7, 1.7e-7, 3.5e-7) and little of
// a state is left.  d = 0 still gives exactly 1.  Where the decays of a whole run are
// taken at once (one exponential of the sum of d) there is nothing to add up, and no
// nudge.
constexpr float kNudge = 2.4e-8f;
__device__ __forceinline__ f2 decay_2(f2 d, f2 A2) { return ex2_2(fma2(d, A2, pack2(kNudge, kNudge))); }
__device__ __forceinline__ float decay(float d, float A2) { return ex2(fmaf(d, A2, kNudge)); }

// A, as the decays take it: times log2(e), and -infinity as the lowest finite value.  A
// step then multiplies a state by 0 all the same, and d = 0, which fills the kernels'
// tiles behind a row's end, keeps it: 0 times infinity would not.
__device__ __forceinline__ float rate(float A) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(A * kLog2e), "f"(-3.4028235e38f));
    return r;
}

__device__ __forceinline__ float rcp(float v) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ f2 rcp_2(f2 v) { return pack2(rcp(lo2(v)), rcp(hi2(v))); }
__device__ __forceinline__ f2 both(float v) { return pack2(v, v); }

// exp(-a) for a >= 0 (NaN: NaN), 0 beyond 87.3.  2^t takes t = -a log2(e) rounded
// to float32, an error of up to |t| 2^-25 in the exponent.  kFine takes it out:
// exp(-a) = 2^t exp(r), r = -a - t ln 2, with ln 2 in two parts (the argument
// reduction of Cody and Waite), exp(r) = 1 + r.
constexpr float kLn2Low = -1.9046542e-9f;  // ln 2 - kLn2
__device__ __forceinline__ float capped(float a) {  // beyond 104 nothing changes, and an infinity would give r = NaN
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(104.0f));
    return r;
}
template <bool kFine>
__device__ __forceinline__ float exp_minus(float a) {
    if constexpr (!kFine) {
        return ex2(a * -kLog2e);
    } else {
        a = capped(a);
        const float t = a * -kLog2e, e = ex2(t);
        return fmaf(e, fmaf(t, -kLn2Low, fmaf(t, -kLn2, -a)), e);
    }
}
template <bool kFine>
__device__ __forceinline__ f2 exp_minus_2(f2 a) {
    if constexpr (!kFine) {
        return ex2_2(mul2(a, both(-kLog2e)));
    } else {
        a = pack2(capped(lo2(a)), capped(hi2(a)));
        const f2 t = mul2(a, both(-kLog2e)), e = ex2_2(t);
        const f2 r = fma2(t, both(-kLn2Low), fma2(t, both(-kLn2), a ^ 0x8000000080000000ull));
        return fma2(e, r, e);
    }
}

// The activations for elements of T.  In 16 bits an element's own rounding hides
// the exponent's error ((4 + |v|) 2^-24 of exp(-|v|)); in float32 it would be the
// largest of all, so it is taken out, for two to four more instructions.
template <class T> constexpr bool kFine = sizeof(T) == 4;

// 1 / (1 + exp(-v)).  float32: exp(-|v|) / (1 + exp(-|v|)) below 0, within 9 x 2^-24
// of the result; 16 bits: exp(-v) = infinity gives 0.
template <class T>
__device__ __forceinline__ float sigmoid(float v) {
    if constexpr (!kFine<T>) return rcp(1.0f + ex2(v * -kLog2e));
    const float e = exp_minus<true>(fabsf(v)), r = rcp(1.0f + e);
    return v < 0.0f ? e * r : r;
}
template <class T>
__device__ __forceinline__ f2 sigmoid_2(f2 v) {
    if constexpr (!kFine<T>) return rcp_2(add2(both(1.0f), ex2_2(mul2(v, both(-kLog2e)))));
    const f2 e = exp_minus_2<true>(v & 0x7fffffff7fffffffull), r = rcp_2(add2(both(1.0f), e)), below = mul2(e, r);
    return pack2(lo2(v) < 0.0f ? lo2(below) : lo2(r), hi2(v) < 0.0f ? hi2(below) : hi2(r));
}

// log(1 + exp(v)) = max(v, 0) + log1p(e), e = exp(-|v|) in (0, 1], and
// log1p(e) = 2 artanh(s), s = e / (2 + e) <= 1/3; artanh(s) = s + s^3 P(s^2)
// with the cubic P fitted to (artanh(s) / s - 1) / s^2 at Chebyshev points of
// s^2 in [0, 1/9] (relative error of the sum below 2e-8).  No branch and no
// cancellation.  Relative error: within 11 x 2^-24 in float32, (9 + |v|) 2^-24 in 16
// bits (v < 0); 0 below -87.3.
constexpr float kP0 = 0.3333332f, kP1 = 0.20003836f, kP2 = 0.14116974f, kP3 = 0.13433797f;
template <class T>
__device__ __forceinline__ float softplus(float v) {
    const float e = exp_minus<kFine<T>>(fabsf(v));
    const float s = e * rcp(2.0f + e), q = s * s;
    const float p = fmaf(fmaf(fmaf(kP3, q, kP2), q, kP1), q, kP0);
    return fmaf(2.0f, fmaf(p * q, s, s), fmaxf(v, 0.0f));  // NaN: e is NaN
}
template <class T>
__device__ __forceinline__ f2 softplus_2(f2 v) {
    const f2 e = exp_minus_2<kFine<T>>(v & 0x7fffffff7fffffffull);
    const f2 s = mul2(e, rcp_2(add2(both(2.0f), e))), q = mul2(s, s);
    const f2 p = fma2(fma2(fma2(both(kP3), q, both(kP2)), q, both(kP1)), q, both(kP0));
    return fma2(both(2.0f), fma2(mul2(p, q), s, s), pack2(fmaxf(lo2(v), 0.0f), fmaxf(hi2(v), 0.0f)));
}

}  // namespace scg
