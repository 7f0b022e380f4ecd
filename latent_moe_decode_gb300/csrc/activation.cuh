// The activations of the BF16 products and their derivatives.
//
//   none  z            relu  max(z, 0)            silu  z s(z),  s(v) = 1 / (1 + exp(-v))
//   gelu  z P(z), P the normal distribution function     gelu_tanh  z s(v), v = sqrt(8 / pi) (z + 0.044715 z^3)
// (0.5 z (1 + tanh(v / 2)) = z s(v): the form that keeps its relative precision where tanh nears -1.)
#pragma once

#include "common.cuh"

namespace moe {
namespace act_impl {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kTanhScale = 1.5957691216057308f;   // sqrt(8 / pi)
constexpr float kTanhCubic = 0.044715f;
constexpr float kInvSqrt2Pi = 0.3989422804014327f;

__device__ __forceinline__ float rcp(float v) {  // within one unit in the last place
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float exp2_fast(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// Two FP32 values in a pair of registers, and the instructions that take two at once.
typedef uint64_t Pair;
__device__ __forceinline__ Pair pair(float a, float b) {
  Pair r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ Pair both(float v) { return pair(v, v); }
__device__ __forceinline__ void split(Pair v, float* a, float* b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(*a), "=f"(*b) : "l"(v)); }
__device__ __forceinline__ Pair add2(Pair a, Pair b) {
  Pair r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ Pair mul2(Pair a, Pair b) {
  Pair r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) {
  Pair r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ Pair rcp2(Pair v) {
  float a, b;
  split(v, &a, &b);
  return pair(rcp(a), rcp(b));
}
template <bool FAST>
__device__ __forceinline__ Pair exp_or_exp2(Pair v) {  // FAST: 2^v, else e^v
  float a, b;
  split(v, &a, &b);
  return FAST ? pair(exp2_fast(a), exp2_fast(b)) : pair(expf(a), expf(b));
}

// The epilogues of tiles with a short K wait for these, two warps a scheduler on a chain of TMEM load, special
// functions, polynomial and store (one reciprocal and one exponential a value, of which an SM computes 16 a cycle,
// would take 4096 x 7168 x 512 12.5 us): so two values an instruction where there is one for it.
// 4096 x 7168 x 512 with bias, us: BF16 silu 38, gelu 43 (with one value an instruction 3 to 4 % more), FP32
// results' silu 54, gelu 71 (15 to 25 % more; with a rounded division and normcdff 98 and 151, when the bias cost 8 more).
// FAST is for results that go to BF16: the special-function unit's 2^x. Else expf.

// z times 1 / (1 + exp(-v)) (0 where that is below 2^-126). FAST: within some 2^-20 of the value to
// |v| = 12 (the exponent's argument is rounded).
template <bool FAST>
__device__ __forceinline__ void times_sigmoid(Pair v, float* z0, float* z1) {
  const Pair e = exp_or_exp2<FAST>(mul2(v, both(FAST ? -kLog2e : -1.f)));
  split(mul2(pair(*z0, *z1), rcp2(add2(e, both(1.f)))), z0, z1);
}

__device__ __forceinline__ Pair tanh_argument(Pair z) {
  return mul2(mul2(both(kTanhScale), z), fma2(mul2(both(kTanhCubic), z), z, both(1.f)));
}

// exp(a^2 / 2) P(-a) of a >= 0, P the normal distribution function: t times a polynomial in t =
// 1 / (1 + 0.305 a), fitted for this file by Remez' exchange to the least largest relative error on
// a = 0 to 15: 1.25e-7 with the coefficients in FP32.
__device__ __forceinline__ Pair scaled_tail(Pair a) {
  const Pair t = rcp2(fma2(both(0.305f), a, both(1.f)));
  Pair p = fma2(t, both(0.0364274166f), both(-0.151896889f));
  p = fma2(t, p, both(0.183906286f));
  p = fma2(t, p, both(-0.0363741916f));
  p = fma2(t, p, both(0.120207309f));
  p = fma2(t, p, both(0.103657576f));
  p = fma2(t, p, both(0.12243049f));
  p = fma2(t, p, both(0.121641998f));
  return mul2(t, p);
}

// P(z) and, of it, exp(-z^2 / 2). FAST: within some 2^-18, with the rounding of z^2 / 2 up to 40. Else
// what that rounding left out is brought in to the first order: within 1e-6, rms 2e-7. Beyond 15 P
// is 0 or 1 in FP32.
template <bool FAST>
__device__ __forceinline__ Pair normal_cdf(float z0, float z1, Pair* density) {
  Pair a = pair(fabsf(z0), fabsf(z1)), e;
  if (FAST) {
    e = exp_or_exp2<true>(mul2(mul2(a, both(-0.5f * kLog2e)), a));
  } else {
    a = pair(fminf(fabsf(z0), 15.f), fminf(fabsf(z1), 15.f));
    const Pair m = mul2(a, both(-0.5f)), h = mul2(m, a);
    e = exp_or_exp2<false>(h);
    e = fma2(e, fma2(m, a, mul2(h, both(-1.f))), e);
  }
  *density = e;
  float l0, l1, u0, u1;  // P(-|z|), P(|z|)
  const Pair low = mul2(scaled_tail(a), e);
  split(low, &l0, &l1);
  split(fma2(low, both(-1.f), both(1.f)), &u0, &u1);
  return pair(z0 < 0.f ? l0 : u0, z1 < 0.f ? l1 : u1);
}

// max(z, 0); a NaN stays one.
__device__ __forceinline__ float relu(float z) {
  float r;
  asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(r) : "f"(z));
  return r;
}

// act(z) of N values, an even number (the choice outside the loop: it is the same for all of them).
template <bool FAST, int N>
__device__ __forceinline__ void apply(int act, float (&z)[N]) {
  switch (act) {
    case BF16_ACT_RELU:
#pragma unroll
      for (int i = 0; i < N; ++i) z[i] = relu(z[i]);
      break;
    case BF16_ACT_SILU:
#pragma unroll
      for (int i = 0; i < N; i += 2) times_sigmoid<FAST>(pair(z[i], z[i + 1]), &z[i], &z[i + 1]);
      break;
    case BF16_ACT_GELU:
#pragma unroll
      for (int i = 0; i < N; i += 2) {
        Pair d;
        split(mul2(pair(z[i], z[i + 1]), normal_cdf<FAST>(z[i], z[i + 1], &d)), &z[i], &z[i + 1]);
      }
      break;
    case BF16_ACT_GELU_TANH:
#pragma unroll
      for (int i = 0; i < N; i += 2) times_sigmoid<FAST>(tanh_argument(pair(z[i], z[i + 1])), &z[i], &z[i + 1]);
      break;
    default: break;
  }
}

// act(z) and its derivative, of two values. Where a sigmoid has reached 0 or 1 the term with its own
// slope is 0 however large z is (so that z of +-infinity has the limit's derivative).
__device__ __forceinline__ void with_slope(int act, const float (&z)[2], float (&value)[2], float (&slope)[2]) {
  const Pair zs = pair(z[0], z[1]);
  switch (act) {
    case BF16_ACT_SILU:
    case BF16_ACT_GELU_TANH: {
      const bool silu = act == BF16_ACT_SILU;
      float s[2];
      split(rcp2(add2(exp_or_exp2<true>(mul2(silu ? zs : tanh_argument(zs), both(-kLog2e))), both(1.f))), &s[0], &s[1]);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float t = s[i] * (1.f - s[i]), d = silu ? 1.f : kTanhScale * fmaf(3.f * kTanhCubic * z[i], z[i], 1.f);
        value[i] = z[i] * s[i];
        slope[i] = t == 0.f ? s[i] : fmaf(z[i] * t, d, s[i]);
      }
      break;
    }
    case BF16_ACT_GELU: {
      Pair density;
      float d[2], p[2];
      split(normal_cdf<true>(z[0], z[1], &density), &p[0], &p[1]);
      split(mul2(density, both(kInvSqrt2Pi)), &d[0], &d[1]);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        value[i] = z[i] * p[i];
        slope[i] = d[i] == 0.f ? p[i] : fmaf(z[i], d[i], p[i]);
      }
      break;
    }
    default:
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        value[i] = act == BF16_ACT_RELU ? relu(z[i]) : z[i];
        slope[i] = act == BF16_ACT_NONE || z[i] > 0.f ? 1.f : 0.f;  // (relu of a NaN: 0)
      }
      break;
  }
}

}  // namespace act_impl
}  // namespace moe
