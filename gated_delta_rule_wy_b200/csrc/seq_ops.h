// seq_ops.h -- device helpers of the layers around the mixer (selective scan, convolution
// backward, head norm): runs of consecutive elements held as raw words, pairs of fp32 values,
// asynchronous copies, and the elementwise laws in fp32.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <float.h>
#include <stdint.h>

namespace gdr2 {
namespace seq {

// E consecutive elements of type T as 32-bit words (bf16 stays packed, two to a word).
template <typename T, int E> struct Raw {
    static constexpr int kWords = E * (int)sizeof(T) / 4;
    static_assert(E * sizeof(T) % 4 == 0, "a run is whole words");
    uint32_t w[kWords];

    __device__ __forceinline__ void zero()
    {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = 0u;
    }
    __device__ __forceinline__ float get(int i) const
    {
        if constexpr (sizeof(T) == 2) return __uint_as_float((i & 1) ? (w[i / 2] & 0xffff0000u) : (w[i / 2] << 16));
        else return __uint_as_float(w[i]);
    }
    // p: E elements, all valid and aligned to min(16, the run's bytes)
    __device__ __forceinline__ void load_vec(const T *p)
    {
        if constexpr (kWords % 4 == 0) {
#pragma unroll
            for (int i = 0; i < kWords / 4; ++i) {
                const uint4 a = __ldg(reinterpret_cast<const uint4 *>(p) + i);
                w[4 * i] = a.x; w[4 * i + 1] = a.y; w[4 * i + 2] = a.z; w[4 * i + 3] = a.w;
            }
        } else if constexpr (kWords == 2) {
            const uint2 a = __ldg(reinterpret_cast<const uint2 *>(p));
            w[0] = a.x; w[1] = a.y;
        } else {
            static_assert(kWords == 1, "runs are 1, 2 or a multiple of 4 words");
            w[0] = __ldg(reinterpret_cast<const uint32_t *>(p));
        }
    }
    // elements min(c + i, last) of a row, one by one: every load is in the row and none waits for a test
    __device__ __forceinline__ void load_clamped(const T *row, int c, int last)
    {
        if constexpr (sizeof(T) == 2) {
            const unsigned short *u = reinterpret_cast<const unsigned short *>(row);
#pragma unroll
            for (int i = 0; i < kWords; ++i) {
                const uint32_t lo = __ldg(u + min(c + 2 * i, last)), hi = __ldg(u + min(c + 2 * i + 1, last));
                w[i] = lo | (hi << 16);
            }
        } else {
#pragma unroll
            for (int i = 0; i < kWords; ++i) w[i] = __ldg(reinterpret_cast<const uint32_t *>(row) + min(c + i, last));
        }
    }
};

// bf16 pair, a in the low half
__device__ __forceinline__ uint32_t pack2(float a, float b)
{
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// E fp32 values to E elements of type T at p (rounded to nearest even)
template <typename T, int E> __device__ __forceinline__ void store_vec(T *p, const float (&v)[E])
{
    constexpr int kWords = E * (int)sizeof(T) / 4;
    uint32_t w[kWords];
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
        if constexpr (sizeof(T) == 2) w[i] = pack2(v[2 * i], v[2 * i + 1]);
        else w[i] = __float_as_uint(v[i]);
    }
    if constexpr (kWords % 4 == 0) {
#pragma unroll
        for (int i = 0; i < kWords / 4; ++i)
            reinterpret_cast<uint4 *>(p)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    } else if constexpr (kWords == 2) {
        *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
    } else {
        static_assert(kWords == 1, "runs are 1, 2 or a multiple of 4 words");
        *reinterpret_cast<uint32_t *>(p) = w[0];
    }
}
template <typename T> __device__ __forceinline__ void store_one(T *p, float v)
{
    if constexpr (sizeof(T) == 2) *p = __float2bfloat16_rn(v);
    else *p = v;
}
template <typename T, int E> __device__ __forceinline__ void store_each(T *p, const float (&v)[E], int valid)
{
#pragma unroll
    for (int i = 0; i < E; ++i)
        if (i < valid) store_one(p + i, v[i]);
}
// One element as raw bits, so that a load in flight is not waited for, and its value.
template <typename T> __device__ __forceinline__ uint32_t load_bits(const T *p)
{
    if constexpr (sizeof(T) == 2) return __ldg(reinterpret_cast<const unsigned short *>(p));
    else return __ldg(reinterpret_cast<const uint32_t *>(p));
}
template <typename T> __device__ __forceinline__ float bits_value(uint32_t b)
{
    return __uint_as_float(sizeof(T) == 2 ? b << 16 : b);
}

// Asynchronous copies to shared memory, BYTES (4, 8 or 16) each, and their groups.
template <int BYTES> __device__ __forceinline__ void copy_async(void *dst, const void *src)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"((unsigned)__cvta_generic_to_shared(dst)), "l"(src),
                 "n"(BYTES)
                 : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT> __device__ __forceinline__ void copies_wait()  // until at most LEFT groups are under way
{
    asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory");
}

constexpr float kLog2e = 1.4426950408889634f;

// 2^x on the special-function unit (relative error 2^-22; 0 below the normal range)
__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float rcp(float x)  // 1 / x, one unit in the last place; 0 for infinity
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// 2^(d a2) for a decay, a2 = A log2 e. The special-function unit's results lie 0.35 x 2^-24 below the value on
// average (measured over arguments in (-4, 0)), which a long memory would add up over its tokens; kDecayBias
// in the exponent takes that out. It leaves 2^0 = 1 as it is.
constexpr float kDecayBias = 3.0e-8f;
__device__ __forceinline__ float decay2(float d, float a2) { return ex2(fmaf(d, a2, kDecayBias)); }

// A for use by the kernels, and as the rate a2 of decay2. An A of minus infinity counts as the lowest finite value, so that
// a step of 0, as those that fill up a tile are, leaves the state (infinity times 0 is NaN) and any other clears it.
__device__ __forceinline__ float held(float a) { return a < -FLT_MAX ? -FLT_MAX : a; }
__device__ __forceinline__ float decay_rate(float a) { return held(a * kLog2e); }

// e^x for x <= 0 with the rounding of x log2 e, which grows with |x|, put back: the product's error is exact in a
// fused multiply-add, and the rest of log2 e's digits are a second constant. (Below x = -104, where the value is 0,
// it is left out: for an infinite x it is infinity minus infinity.)
__device__ __forceinline__ float exp_rest(float x)
{
    constexpr float kLog2eRest = 1.925963e-8f, kLn2 = 0.69314718f;
    const float y = x * kLog2e, rest = fmaf(x, kLog2eRest, fmaf(x, kLog2e, -y));
    const float e = ex2(y);
    return fmaf(e * kLn2, x < -104.f ? 0.f : rest, e);
}

// log(1 + e^v) = max(v, 0) + log(1 + e), e = e^-|v| in (0, 1], with log(1 + e) = 2 atanh(s),
// s = e / (2 + e) in (0, 1/3]: no cancellation for the small e of a trained layer's step
// sizes, where log(1 + e) from the logarithm loses them. atanh(s) / s is a minimax polynomial
// (Remez exchange) of degree 4 in s^2 on [0, 1/9], relative error 8e-9 with these fp32 coefficients.
__device__ __forceinline__ float softplus(float v)
{
    const float e = exp_rest(-fabsf(v));
    const float s = e * rcp(2.f + e), t = s * s;
    float p = fmaf(0.28178335f, t, 0.27960603f);
    p = fmaf(p, t, 0.40024910f);
    p = fmaf(p, t, 0.66666315f);
    p = fmaf(p, t, 2.f);
    return fmaf(s, p, fmaxf(v, 0.f));
}
// 1 / (1 + e^-v); below v = -88 the exponential overflows and the quotient is 0
__device__ __forceinline__ float sigmoid(float v) { return rcp(1.f + ex2(-v * kLog2e)); }
// the same without an exponential above 1: a step of any size below zero, infinite ones too, has a slope of 0, not
// the quotient of an infinity
__device__ __forceinline__ float softplus_slope(float v)
{
    const float e = exp_rest(-fabsf(v));
    return (v < 0.f ? e : 1.f) * rcp(1.f + e);
}

// Two fp32 values in one 64-bit register, and the instructions that work on both at once.
typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 pair(float lo, float hi)
{
    f32x2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void split(f32x2 v, float &lo, float &hi)
{
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b)
{
    f32x2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b)
{
    f32x2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c)
{
    f32x2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
// 2^(d a) h + o for two states: a value carried over a segment whose step sizes sum to d, and the segment's own part.
// The factor alone may pass fp32's range where the product does not (h zero or small before growth, large before
// decay): it is then applied in four parts, each held to 2^-126 .. 2^127. The limits change no result: four such
// factors take every nonzero h (2^-149 at least) to infinity, and every finite one to zero. NaN takes the first way.
__device__ __forceinline__ f32x2 carry2(float d, float a, float b, f32x2 h, f32x2 o)
{
    const float x = d * a, y = d * b;
    if (!(fmaxf(fabsf(x), fabsf(y)) > 125.f)) return fma2(pair(decay2(d, a), decay2(d, b)), h, o);
    auto quarter = [](float v) { return ex2(fminf(fmaxf(0.25f * v, -126.f), 127.f)); };
    const f32x2 q = pair(quarter(x), quarter(y));
#pragma unroll
    for (int i = 0; i < 4; ++i) h = mul2(q, h);
    return add2(h, o);
}
// 16 bytes of shared memory as two pairs
__device__ __forceinline__ void lds_pairs(const float *p, f32x2 &a, f32x2 &b)
{
    const ulonglong2 v = *reinterpret_cast<const ulonglong2 *>(p);
    a = v.x;
    b = v.y;
}

// The sequence that token t of a packed stream belongs to: the last s in [0, N) with
// cu[s] <= t (empty sequences share cu[s] with the next). Stays in [0, N) for any array.
__device__ __forceinline__ int find_sequence(const int *cu, int N, int t)
{
    int lo = 0, hi = N - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (__ldg(cu + mid) <= t) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

}  // namespace seq
}  // namespace gdr2
