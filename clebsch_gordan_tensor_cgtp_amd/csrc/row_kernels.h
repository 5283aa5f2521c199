// HIP source shared by the kernels that are compiled for a configuration: runs of a row's elements,
// lane exchanges, activations.  It comes after the configuration's constants:
//   T, R   element type in memory; type of statistics, weights and sums (float, or double)
//   ACT    0 identity 1 sigmoid 2 silu 3 tanh (0 where there is none)
#pragma once

namespace cgtp {

static const char kRowKernels[] = R"HIP(
#define DEV static __device__ __forceinline__

// ---------------------------------------------------------------- runs of elements
// Rows start at any element, so the vector types claim no more than the element's alignment.

template <int N, typename S, typename X> DEV void load_run(const S *p, X *x)
{
    if constexpr (N > 0) {
        constexpr int W = 16 / sizeof(S);
        constexpr int n = N >= W ? W : N >= 8 ? 8 : N >= 4 ? 4 : N >= 2 ? 2 : 1;
        typedef S V __attribute__((ext_vector_type(n), aligned(sizeof(S))));
        if constexpr (n == 1) {
            x[0] = (X)p[0];
        } else {
            const V r = *reinterpret_cast<const V *>(p);
#pragma unroll
            for (int i = 0; i < n; ++i) x[i] = (X)r[i];
        }
        load_run<N - n>(p + n, x + n);
    }
}

template <int N, typename S> DEV void store_run(S *p, const R *x)
{
    if constexpr (N > 0) {
        constexpr int W = 16 / sizeof(S);
        constexpr int n = N >= W ? W : N >= 8 ? 8 : N >= 4 ? 4 : N >= 2 ? 2 : 1;
        typedef S V __attribute__((ext_vector_type(n), aligned(sizeof(S))));
        if constexpr (n == 1) {
            p[0] = (S)x[0];
        } else {
            V r;
#pragma unroll
            for (int i = 0; i < n; ++i) r[i] = (S)x[i];
            *reinterpret_cast<V *>(p) = r;
        }
        store_run<N - n>(p + n, x + n);
    }
}

// ---------------------------------------------------------------- lane exchanges
// Exchanges of a butterfly: inside 16 lanes by DPP (quads, then mirrored halves and rows, whose
// values are equal by then), across them by the permlane swaps.  Every lane ends with the same bits.
// A swap's results are copied into plain variables first: bit-casting the elements of the builtin's
// vector made the front end read element 0 for both.

template <int CTRL> DEV float dpp(float v)
{
    return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 15, 15, false));
}
template <int CTRL> DEV double dpp(double v)
{
    const unsigned long long b = __builtin_bit_cast(unsigned long long, v);
    const unsigned lo = __builtin_amdgcn_mov_dpp((int)b, CTRL, 15, 15, false);
    const unsigned hi = __builtin_amdgcn_mov_dpp((int)(b >> 32), CTRL, 15, 15, false);
    return __builtin_bit_cast(double, (unsigned long long)hi << 32 | lo);
}
DEV float swap16(float v)
{
    const unsigned a = __builtin_bit_cast(unsigned, v);
    const auto r = __builtin_amdgcn_permlane16_swap(a, a, false, false);
    const unsigned r0 = r[0], r1 = r[1];
    return __builtin_bit_cast(float, r0) + __builtin_bit_cast(float, r1);
}
DEV float swap32(float v)
{
    const unsigned a = __builtin_bit_cast(unsigned, v);
    const auto r = __builtin_amdgcn_permlane32_swap(a, a, false, false);
    const unsigned r0 = r[0], r1 = r[1];
    return __builtin_bit_cast(float, r0) + __builtin_bit_cast(float, r1);
}
DEV double join64(unsigned lo, unsigned hi)
{
    return __builtin_bit_cast(double, (unsigned long long)hi << 32 | lo);
}
DEV double swap16(double v)
{
    const unsigned long long b = __builtin_bit_cast(unsigned long long, v);
    const auto lo = __builtin_amdgcn_permlane16_swap((unsigned)b, (unsigned)b, false, false);
    const auto hi = __builtin_amdgcn_permlane16_swap((unsigned)(b >> 32), (unsigned)(b >> 32), false, false);
    return join64(lo[0], hi[0]) + join64(lo[1], hi[1]);
}
DEV double swap32(double v)
{
    const unsigned long long b = __builtin_bit_cast(unsigned long long, v);
    const auto lo = __builtin_amdgcn_permlane32_swap((unsigned)b, (unsigned)b, false, false);
    const auto hi = __builtin_amdgcn_permlane32_swap((unsigned)(b >> 32), (unsigned)(b >> 32), false, false);
    return join64(lo[0], hi[0]) + join64(lo[1], hi[1]);
}

// ---------------------------------------------------------------- activations
// A text before this one may ask for the hardware's exponential and reciprocal in float too (FAST_EXP).
#ifndef FAST_EXP
#define FAST_EXP (sizeof(T) == 2)
#endif
// Rows of 16 bits take the hardware's exponential and reciprocal: their errors, |g| 2^-23 and 2^-23 of the
// result, are far below a rounding to 16 bits; the weight gradients, which are float, have them in every row's
// term, as large as a few of float's own roundings (the join's backward, 8,192 scalar rows
// of 4,096 in bf16 with a SiLU gate: 131 us with expf and a division, 116 us).
DEV float exp_of(float v) { return FAST_EXP ? __builtin_amdgcn_exp2f(v * 1.44269504f) : expf(v); }
DEV float inverse(float v) { return FAST_EXP ? __builtin_amdgcn_rcpf(v) : 1.0f / v; }
DEV double inverse(double v) { return 1.0 / v; }
DEV double exp_of(double v) { return exp(v); }
DEV float tanh_of(float v) { return tanhf(v); }
DEV double tanh_of(double v) { return tanh(v); }
DEV float root_inverse(float v) { return 1.0f / __builtin_sqrtf(v); }
DEV double root_inverse(double v) { return 1.0 / __builtin_sqrt(v); }

// tanh(g) from e = exp(-2 |g|) and r = 1 / (1 + e); below 1/4, where 1 - e would cancel, its series to g^9 (what
// follows is under 2^-26 of it there).  Doubles take the function itself.
DEV float tanh_from(float g, float e, float r)
{
    const float t = (1.0f - e) * r, g2 = g * g;
    const float small = g * (1.0f + g2 * (-1.0f / 3 + g2 * (2.0f / 15 + g2 * (-17.0f / 315 + g2 * (62.0f / 2835)))));
    return g2 < 0.0625f ? small : g < 0 ? -t : t;
}
DEV double tanh_from(double g, double, double) { return tanh(g); }

DEV R act_value(R g)
{
    if (ACT == 0) return g;
    if (ACT == 3) {
        if (!FAST_EXP || sizeof(T) == 2) return tanh_of(g);
        const R e = exp_of(g < 0 ? 2 * g : -2 * g);
        return tanh_from(g, e, inverse((R)1 + e));
    }
    const R s = inverse((R)1 + exp_of(-g));
    return ACT == 1 ? s : g * s;
}

// act'(g) and act(g).  The sigmoid and its complement are q = e / (1 + e) and 1 - q, e = exp(-|g|), and the slope
// their product; with 1 - s from s it would carry a rounding of 1 (17% of it at 15, all of it at 17).  tanh's
// slope is 4 e / (1 + e)^2 with e = exp(-2 |g|), not 1 - tanh^2.  SiLU's complement is a small term beside 1 there.
DEV R act_slope(R g, R &value)
{
    if (ACT == 0) {
        value = g;
        return (R)1;
    }
    if (ACT == 3) {
        const R e = exp_of(g < 0 ? 2 * g : -2 * g), r = inverse((R)1 + e);
        value = tanh_from(g, e, r);
        return 4 * (e * r * r);
    }
    if (ACT == 1) {
        const R e = exp_of(g < 0 ? g : -g), q = e * inverse((R)1 + e);
        value = g < 0 ? q : (R)1 - q;
        return q * ((R)1 - q);
    }
    const R s = inverse((R)1 + exp_of(-g));
    value = g * s;
    return s * ((R)1 + g * ((R)1 - s));
}
)HIP";

}  // namespace cgtp
