// What the kernels of the head's rows share: the (maximum, sum) pairs of a
// softmax in base 2, sums with compensation, and what d needs of a row.
#pragma once

#include <cstdint>

namespace jetq {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// What d needs of a row, written by the backward pass's first kernel.
struct alignas(16) GradRow {
    int target; // -1: a row without a loss, the rest is zero
    float lse2; // lse in base 2
    float dloss;
    float dt;   // exp(z_t - lse) - 1, from a logit that this row's own sum gives
};

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void join_pair(float2 &a, const float2 b)
{
    const float m = fmaxf(a.x, b.x);
    if (m > -INFINITY)
        a = make_float2(m, a.y * ex2(a.x - m) + b.y * ex2(b.x - m));
    else
        a.y += b.y; // both empty (or NaN)
}

// s + b as s + c, exactly (Knuth's two-sum), c added to the compensation.
__device__ __forceinline__ void two_sum(float &s, float &c, float b)
{
    const float t = __fadd_rn(s, b), u = __fsub_rn(t, s);
    c = __fadd_rn(c, __fadd_rn(__fsub_rn(s, __fsub_rn(t, u)), __fsub_rn(b, u)));
    s = t;
}

// Eight products of BF16 pairs (exact in FP32) added to s + c.
__device__ __forceinline__ void dot8(float &s, float &c, const uint4 &a, const uint4 &b)
{
    const uint32_t p[4] = {a.x, a.y, a.z, a.w}, q[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        two_sum(s, c, __fmul_rn(__uint_as_float(p[e] << 16), __uint_as_float(q[e] << 16)));
        two_sum(s, c, __fmul_rn(__uint_as_float(p[e] & 0xffff0000u), __uint_as_float(q[e] & 0xffff0000u)));
    }
}

// The sum s + c; an infinite one has no rest.
__device__ __forceinline__ double whole_sum(float s, float c)
{
    return c == c ? (double)s + (double)c : (double)s;
}

} // namespace jetq
