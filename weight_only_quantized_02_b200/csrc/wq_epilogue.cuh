// wq_epilogue.cuh -- the layer's epilogue, shared by every kernel that
// writes y:
//
//     y[m][n] = round(act(v + bias[n]) * mul[m][n] + residual[m][n]),
//
// v the accumulated (and, for INT8, scaled) sum of output (m, n), everything
// in fp32 and rounded once; or the fp32 value v itself (EpiArgs::out_f32, the
// vocabulary head's unrounded logits).
//
// Kernels are instantiated without an epilogue (EPI = false: wq_linear's
// code, unchanged) and with one, whose parts are chosen at run time by
// branches that are the same for every thread.  A part costs one 16-bit load
// per output (2 of the layer's bytes for every K bytes or K / 2 bytes of
// weights), so what bounds the layer still does; the loads' latency, at the
// end of a call, is what can be seen, and loading is therefore separate from
// storing: a thread with several outputs loads all their operands first.
//
// y may be the residual or mul buffer itself (the same element): every
// element is read and written by the same thread, and the operands are read
// past L1 (ld.cg), so a line cached before another SM's write is never used.
#pragma once

#include <cstdint>
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "wq.h"
#include "wq_internal.h"

namespace wq {

// A kernel's parameters, with an epilogue or without.  The stream-K, integer and
// role-split kernels' instances without one have nothing of it, parameters and stores
// included, so that they are compiled as if there were none: with it among the
// parameters, and stores shared by both forms, the integer GEMV of 5120 x 17408 took
// 21.6 us at four tokens instead of 19.9, the role-split GEMM of 17408 x 5120 33.9 at
// 64 instead of 32.3.  (The other two kernels' stores are shared and cost the same.)
template <class Params>
struct WithEpilogue : Params {
    EpiArgs epi;
};
template <class Params, bool EPI>
using EpiParams = std::conditional_t<EPI, WithEpilogue<Params>, Params>;

// The two tensor operands of one output, as loaded: converted only where they
// are used.  A thread with several outputs asks once whether an operand is there
// and loads them all (epi_load_batch).  Converted beside its load, or behind a
// branch for each, every load was waited for before the next began (role-split
// GEMM, 17408 x 5120, 128 tokens with a residual and GELU: 76 us, so 58).
struct EpiOps {
    uint16_t mul, res;
};

template <bool F16 = false>
__device__ __forceinline__ EpiOps epi_none() // of absent operands: 1 and 0
{
    return EpiOps{(uint16_t)(F16 ? 0x3C00u : 0x3F80u), 0};
}

template <bool F16>
__device__ __forceinline__ float act16_to_float(uint16_t b)
{
    if constexpr (F16)
        return __half2float(__ushort_as_half(b));
    else
        return __uint_as_float((uint32_t)b << 16);
}

template <bool F16>
__device__ __forceinline__ uint16_t float_to_act16(float v)
{
    if constexpr (F16)
        return __half_as_ushort(__float2half_rn(v));
    else
        return __bfloat16_as_ushort(__float2bfloat16_rn(v));
}

// erfc(a) for a >= 0: t exp(-a^2 + P(t)), t = 1 / (1 + a / 2) (the substitution of
// Press et al., Numerical Recipes, 6.2), P a Chebyshev fit of ln(erfc(a) exp(a^2) / t)
// over 0 < t <= 1 in powers of t.  Relative error, by evaluation in fp32 against
// binary64 for a up to 9: 4.1e-7 near 0, then that of the exponential's argument,
// together at most (2 + 1.4 a^2) 2^-22 with the fast exponential's.  Straight code,
// for several values side by side (prompt GEMM, INT8 5120 x 17408, 333 tokens: 59 us
// against 66 with erfcf).
__device__ __forceinline__ float epi_erfc(float a)
{
    const float t = __fdividef(1.f, fmaf(0.5f, a, 1.f));
    float p = 0.170868918f;
    p = fmaf(p, t, -0.822135866f);
    p = fmaf(p, t, 1.48848701f);
    p = fmaf(p, t, -1.13517654f);
    p = fmaf(p, t, 0.278852999f);
    p = fmaf(p, t, -0.186283216f);
    p = fmaf(p, t, 0.0967833176f);
    p = fmaf(p, t, 0.374092042f);
    p = fmaf(p, t, 1.00002372f);
    p = fmaf(p, t, -1.26551223f);
    return t * __expf(fmaf(-a, a, p));
}

// The activation of CNT values.  The erf form is written with erfc, which keeps
// its relative accuracy where 1 + erf cancels; the tanh form is v * logistic(2 u),
// which does not cancel either.  The logistic function is written with exp(-|u|), so
// that the quotient's denominator stays between 1 and 2 (a fast division by exp(-u)
// gives 0 from 2^126 on, where SiLU is still a normal number: -4e-37 at -88), and uses
// the fast exponential and reciprocal (a few 2^-22 of its value, and one more per
// unit of |u|), against an output of 8 or 11 significant bits.
template <int CNT>
__device__ __forceinline__ void epi_activations(float (&v)[CNT], int act)
{
    if (act == WQ_ACT_NONE)
        return;
    if (act == WQ_ACT_RELU) {
#pragma unroll
        for (int j = 0; j < CNT; ++j)
            v[j] = v[j] < 0.f ? 0.f : v[j];
    } else if (act == WQ_ACT_GELU) {
#pragma unroll
        for (int j = 0; j < CNT; ++j) {
            const float e = epi_erfc(0.70710678f * fabsf(v[j]));
            v[j] = 0.5f * v[j] * (v[j] > 0.f ? 2.f - e : e);
        }
    } else {
#pragma unroll
        for (int j = 0; j < CNT; ++j) {
            float u = v[j]; // WQ_ACT_SILU: v * logistic(v)
            if (act == WQ_ACT_GELU_TANH)
                u = 1.5957691f * fmaf(0.044715f * u, u * u, u); // 2 sqrt(2/pi) (v + 0.044715 v^3)
            const float t = __expf(-fabsf(u));
            float r;
            asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + t));
            v[j] = (u < 0.f ? v[j] * t : v[j]) * r;
        }
    }
}

// One value, out of line: the formulas inlined at every output of the unrolled
// stores would multiply the kernels' code.
static __device__ __noinline__ float epi_activation(float v, int act)
{
    float x[1] = {v};
    epi_activations(x, act);
    return x[0];
}

// The operands of output (m, n); absent ones are the identity.
template <bool EPI, bool F16 = false>
__device__ __forceinline__ EpiOps epi_load(const EpiArgs &e, int m, int n)
{
    EpiOps o = epi_none<F16>();
    if constexpr (EPI) {
        if (e.mul)
            o.mul = __ldcg(e.mul + (long long)m * e.ld_mul + n);
        if (e.res)
            o.res = __ldcg(e.res + (long long)m * e.ld_res + n);
    }
    return o;
}

// The operands of several outputs, in flight together: at(j, m, n) names output j,
// and is false where there is none.
template <bool EPI, bool F16 = false, int CNT, class At>
__device__ __forceinline__ void epi_load_batch(const EpiArgs &e, EpiOps (&o)[CNT], At at)
{
#pragma unroll
    for (int j = 0; j < CNT; ++j)
        o[j] = epi_none<F16>();
    if constexpr (EPI) {
        if (e.mul)
#pragma unroll
            for (int j = 0; j < CNT; ++j) {
                int m, n;
                if (at(j, m, n))
                    o[j].mul = __ldcg(e.mul + (long long)m * e.ld_mul + n);
            }
        if (e.res)
#pragma unroll
            for (int j = 0; j < CNT; ++j) {
                int m, n;
                if (at(j, m, n))
                    o[j].res = __ldcg(e.res + (long long)m * e.ld_res + n);
            }
    }
}

// Of outputs (m0 + j, n), the first jn of which exist.
template <bool EPI, bool F16 = false, int CNT>
__device__ __forceinline__ void epi_load_tokens(const EpiArgs &e, EpiOps (&o)[CNT], int m0, int jn, int n)
{
    epi_load_batch<EPI, F16>(e, o, [&](int j, int &m, int &nn) {
        m = m0 + j;
        nn = n;
        return j < jn;
    });
}

template <bool EPI, bool F16 = false>
__device__ __forceinline__ float epi_bias(const EpiArgs &e, int n)
{
    if constexpr (EPI)
        if (e.bias)
            return act16_to_float<F16>(__ldcg(e.bias + n));
    return 0.f;
}

// act(v + bias) * mul + residual.  The sum v + bias and the product's fused
// add round in fp32, 2^-24 relative each, far below the output's rounding.
template <bool F16>
__device__ __forceinline__ float epi_value(const EpiArgs &e, float v, float bias, const EpiOps &o)
{
    v += bias;
    if (e.act != WQ_ACT_NONE)
        v = epi_activation(v, e.act);
    return fmaf(v, act16_to_float<F16>(o.mul), act16_to_float<F16>(o.res));
}

// Writes output (m, n) with accumulated value v.
template <bool EPI, bool F16 = false>
__device__ __forceinline__ void epi_store(const EpiArgs &e, uint16_t *y, int N, int m, int n, float v, float bias,
                                          const EpiOps &o)
{
    const size_t at = (size_t)m * N + n;
    if constexpr (EPI) {
        if (e.out_f32) {
            reinterpret_cast<float *>(y)[at] = v;
            return;
        }
        v = epi_value<F16>(e, v, bias, o);
    }
    y[at] = float_to_act16<F16>(v);
}

// The integer paths' form: v in binary64, rounded once where there is no
// epilogue, to fp32 first where there is one.
template <bool EPI>
__device__ __forceinline__ void epi_store64(const EpiArgs &e, uint16_t *y, int N, int m, int n, double v, float bias,
                                            const EpiOps &o)
{
    if constexpr (EPI)
        epi_store<true>(e, y, N, m, n, (float)v, bias, o);
    else
        y[(size_t)m * N + n] = __bfloat16_as_ushort(__double2bfloat16(v));
}

} // namespace wq
