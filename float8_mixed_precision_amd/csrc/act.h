// Activations of the linear epilogue and their derivatives, in fp32 with the
// hardware exponential and reciprocal (1 ulp each):
//
//   none, relu(z) = max(z, 0), relu2(z) = max(z, 0)^2
//   silu(z) = z s(z),  gelu_tanh(z) = z s(2 sqrt(2/pi) (z + 0.044715 z^3)),
//       s(v) = 1 / (1 + e^-v)
//   gelu(z) = z P(z), P the normal distribution function
//
// in four forms of code:
//  ACT_ID    none
//  ACT_RELUS relu and relu2
//  ACT_SIG   silu and gelu_tanh: v = z (c1 + c3 z^2) with c1 and c3 from the call
//  ACT_ERF   gelu: P(-t) = e^(-t^2/2) m(u), t = |z|, u = 1 / (1 + 0.3 t), m a
//            polynomial of degree 6: the scaled tail e^(t^2/2) P(-t) is smooth in u
//            on [0, 14], and its minimax polynomial (fitted in 64 bits to its
//            values) is off by 1.9e-6 relatively at every t, so the left tail
//            keeps its digits.  e^(-t^2/2) serves the derivative P + z p too.
//
// Errors, over every finite bf16 z, v the exponent's argument (z^2 / 2 for gelu): act
// relative (3 |v| + 8) 2^-24, gelu 2^-18 more; slopes absolute 2^-21, gelu 2^-19.  All
// far below half a bf16 step, 2^-8.
//
// z is bounded where a product of an infinity and a zero would lose the limit: act(+inf)
// = +inf, act(-inf) = 0 (none: -inf), slopes 1 and (within 2^-106) 0; act of a NaN is
// NaN.  (Below -128 silu and gelu_tanh, below -64 gelu, are 0 in fp32.)
#pragma once

#include "fp8l_internal.h"

namespace fp8l {
namespace {

constexpr int ACT_ID = 0, ACT_RELUS = 1, ACT_SIG = 2, ACT_ERF = 3, ACT_FORMS = 4;

constexpr int act_form(int act) {
  return act == FP8L_ACT_GELU ? ACT_ERF
         : act == FP8L_ACT_GELU_TANH || act == FP8L_ACT_SILU ? ACT_SIG
         : act == FP8L_ACT_NONE ? ACT_ID : ACT_RELUS;
}

// What the forms need of the activation, worked out on the host.
struct ActConsts {
  int act;
  uint32_t peak;               // |z| in bf16 where |act| is largest for z < 0, twice
  float c1, c3;                // ACT_SIG: e^-v = 2^(z (c1 + c3 z^2))
  float d1, d3;                // ACT_SIG: dv/dz = d1 + d3 z^2
};

inline ActConsts act_consts(int act) {
  constexpr float L = 1.44269504088896341f, K = 1.59576912160573071f;   // log2 e, 2 sqrt(2/pi)
  ActConsts c = {};
  c.act = act;
  // gelu -0.7518, gelu_tanh -0.7525, silu -1.2785 (the others are 0 for z < 0)
  c.peak = act == FP8L_ACT_SILU ? 0x3FA43FA4u : act == FP8L_ACT_GELU_TANH ? 0x3F413F41u
                                                                          : 0x3F403F40u;
  if (act == FP8L_ACT_SILU) {
    c.c1 = -L;
    c.d1 = 1.f;
  } else if (act == FP8L_ACT_GELU_TANH) {
    c.c1 = -L * K;
    c.c3 = -L * K * 0.044715f;
    c.d1 = K;
    c.d3 = 3.f * K * 0.044715f;
  }
  return c;
}

// maximum and minimum that keep a NaN
__device__ __forceinline__ float max_nan(float a, float b) {
  return __builtin_elementwise_maximum(a, b);
}
__device__ __forceinline__ float min_nan(float a, float b) {
  return __builtin_elementwise_minimum(a, b);
}

// P(-t) for t >= 0, and e = e^(-t^2/2)
__device__ __forceinline__ float normal_tail(float t, float &e) {
  const float u = __builtin_amdgcn_rcpf(__builtin_fmaf(t, 0.3f, 1.0f));
  float m = -0.0845932811498642f;
  m = __builtin_fmaf(m, u, 0.2405729740858078f);
  m = __builtin_fmaf(m, u, -0.04864469915628433f);
  m = __builtin_fmaf(m, u, 0.16476468741893768f);
  m = __builtin_fmaf(m, u, 0.10670444369316101f);
  m = __builtin_fmaf(m, u, 0.12127471715211868f);
  m = __builtin_fmaf(m, u, -7.979083602549508e-05f);
  e = __builtin_amdgcn_exp2f((t * -0.72134752044448170f) * t);
  return e * m;
}

template <int FORM>
__device__ __forceinline__ float act_value(const ActConsts &c, float z) {
  if (FORM == ACT_SIG) {
    const float x = max_nan(z, -128.f);
    const float b = min_nan(x, 128.f);            // (c3 = 0 times an infinite square)
    const float v = b * __builtin_fmaf(c.c3, b * b, c.c1);
    return x * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(v));
  }
  if (FORM == ACT_ERF) {
    const float t = min_nan(__builtin_fabsf(z), 64.f);
    float e;
    const float n = normal_tail(t, e);
    return __builtin_fmaf(-t, n, max_nan(z, 0.f));
  }
  if (FORM == ACT_ID) return z;
  const float m = max_nan(z, 0.f);
  return m * (c.act == FP8L_ACT_RELU ? 1.f : m);
}

template <int FORM>
__device__ __forceinline__ float act_slope(const ActConsts &c, float z) {
  if (FORM == ACT_SIG) {
    // s + z v' s (1 - s), 1 - s = e^-v s without a cancellation
    const float x = min_nan(max_nan(z, -128.f), 128.f);
    const float q = x * x;
    const float e = __builtin_amdgcn_exp2f(min_nan(x * __builtin_fmaf(c.c3, q, c.c1), 126.f));
    const float s = __builtin_amdgcn_rcpf(1.0f + e);
    const float w = x * __builtin_fmaf(c.d3, q, c.d1);
    return __builtin_fmaf(s, w * (e * s), s);
  }
  if (FORM == ACT_ERF) {
    const float t = min_nan(__builtin_fabsf(z), 64.f);
    float e;
    const float n = normal_tail(t, e);
    const float cdf = z >= 0.f ? 1.0f - n : n;
    return __builtin_fmaf(__builtin_copysignf(t, z), e * 0.39894228040143268f, cdf);
  }
  if (FORM == ACT_ID) return 1.f;
  return z <= 0.f ? 0.f : c.act == FP8L_ACT_RELU ? 1.f : 2.f * z;
}

// A sum with a rounding of its own: the compiler would fuse a product in front of it
// where it sees one, in some kernels and not in others.
__device__ __forceinline__ float add32(float a, float b) {
#pragma clang fp contract(off)
  return a + b;
}

// Four values of a linear's output from z: y = act(z) + r as bf16 pairs, and the
// bf16 z.  act applies to the rounded z; without one z is rounded once, with r.
template <int FORM>
__device__ __forceinline__ uint2 act_out4(const ActConsts &c, const float (&f)[4], bool has_r,
                                          uint2 r, uint2 &z) {
  z = make_uint2(bf16x2_bits(f[0], f[1]), bf16x2_bits(f[2], f[3]));
  float v[4] = {f[0], f[1], f[2], f[3]};
  if (FORM != ACT_ID) {
    const float b[4] = {bf16_to_f32(z.x & 0xFFFFu), __uint_as_float(z.x & 0xFFFF0000u),
                        bf16_to_f32(z.y & 0xFFFFu), __uint_as_float(z.y & 0xFFFF0000u)};
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = act_value<FORM>(c, b[e]);
  }
  if (has_r) {
    v[0] = add32(v[0], bf16_to_f32(r.x & 0xFFFFu));
    v[1] = add32(v[1], __uint_as_float(r.x & 0xFFFF0000u));
    v[2] = add32(v[2], bf16_to_f32(r.y & 0xFFFFu));
    v[3] = add32(v[3], __uint_as_float(r.y & 0xFFFF0000u));
  }
  return make_uint2(bf16x2_bits(v[0], v[1]), bf16x2_bits(v[2], v[3]));
}

// The largest |act(z)| of many bf16 z without evaluating act at each: act grows for z
// >= 0, and for z < 0 |act| grows up to one peak (the derivative's zero) and falls
// beyond it, so one of four z decides: the largest, the negative ones nearest the peak
// on either side, and a NaN of negative sign.  (fp32 errors of act do not matter:
// around the peak all z have one bf16 value, and elsewhere neighbours differ by 2^-9
// relatively or more.)  Found on bit patterns, two z a register, in 3 instructions an
// element where evaluating takes 11 to 18:
//   top     signed maximum: the largest z >= 0, or a NaN of positive sign
//   below   unsigned minimum of d = (z ^ sign) - peak: z <= peak nearest to it
//   above   unsigned maximum of d: peak < z < 0 nearest to it (d wraps around)
//   neg     unsigned maximum of z: a NaN of negative sign sorts above all others
// A z of +0 changes none of them.
struct ActKeys {
  uint32_t top, below, above, neg;
};
__device__ __forceinline__ void act_keys_add(ActKeys &k, uint32_t z, uint32_t peak) {
  typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
  typedef short i16x2 __attribute__((ext_vector_type(2)));
#define FP8L_U2(v) __builtin_bit_cast(u16x2, v)
#define FP8L_I2(v) __builtin_bit_cast(i16x2, v)
  const u16x2 d = FP8L_U2(z ^ 0x80008000u) - FP8L_U2(peak);
  k.top = __builtin_bit_cast(uint32_t, __builtin_elementwise_max(FP8L_I2(k.top), FP8L_I2(z)));
  k.below = __builtin_bit_cast(uint32_t, __builtin_elementwise_min(FP8L_U2(k.below), d));
  k.above = __builtin_bit_cast(uint32_t, __builtin_elementwise_max(FP8L_U2(k.above), d));
  k.neg = __builtin_bit_cast(uint32_t, __builtin_elementwise_max(FP8L_U2(k.neg), FP8L_U2(z)));
#undef FP8L_U2
#undef FP8L_I2
}
// The u16 bits of the largest |bf16(act(z))| of a wave's keys, in every lane.
template <int FORM>
__device__ __forceinline__ uint32_t act_keys_amax(const ActConsts &c, const ActKeys &k) {
  const uint32_t peak = c.peak & 0xFFFFu;
  auto of = [&](uint32_t z16) {
    return bf16x2_bits(act_value<FORM>(c, __uint_as_float(z16 << 16)), 0.f) & 0x7FFFu;
  };
  const uint32_t top = wave_max(hmax16(k.top ^ 0x80008000u)) ^ 0x8000u;
  const uint32_t below = 0xFFFFu - wave_max(hmax16(~k.below));
  const uint32_t above = wave_max(hmax16(k.above));
  const uint32_t neg = wave_max(hmax16(k.neg));
  uint32_t m = of(top);
  if (below < 0x8000u - peak) m = max(m, of((below + peak) | 0x8000u));
  if (above >= 0x10000u - peak) m = max(m, of(((above + peak) & 0x7FFFu) | 0x8000u));
  if (neg > 0xFF80u) m = max(m, of(neg));
  return m;
}

// The form of an activation (not ACT_ID) chosen at run time, in kernels that memory
// bounds.
__device__ __forceinline__ float act_value_any(const ActConsts &c, int form, float z) {
  return form == ACT_SIG ? act_value<ACT_SIG>(c, z)
         : form == ACT_ERF ? act_value<ACT_ERF>(c, z) : act_value<ACT_RELUS>(c, z);
}

__device__ __forceinline__ float act_slope_any(const ActConsts &c, int form, float z) {
  return form == ACT_SIG ? act_slope<ACT_SIG>(c, z)
         : form == ACT_ERF ? act_slope<ACT_ERF>(c, z) : act_slope<ACT_RELUS>(c, z);
}

}  // namespace
}  // namespace fp8l
