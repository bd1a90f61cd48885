// Shared by the layer operators (fused linear layer, its backward, mixture of experts): activations
// and their derivatives in fp32, the epilogue's arguments, and the decode of a single weight.
#pragma once

#include <cuda_fp16.h>

#include <cmath>

#include "tern_internal.cuh"

namespace tern {

// What follows z = W x of a linear layer: y = act(z + bias) (+ residual), or with `gated` (n = 2f)
// y = act(z[0:f]) * z[f:2f] (+ residual). Everything in fp32, one rounding to fp16 at the end.
struct Epilogue {
  int act;                   // tern_act
  int gated;
  const uint16_t* bias;      // [n] or null
  const uint16_t* residual;  // [m][n_out] or null
  uint16_t* preact;          // [m][n] or null: z + bias, rounded to fp16
};

__device__ __forceinline__ float h2f(uint16_t h) { return __half2float(__ushort_as_half(h)); }
__device__ __forceinline__ uint16_t f2h(float f) { return __half_as_ushort(__float2half_rn(f)); }

// gelu is z Phi(z). For a = |z|, Phi(-a) = e^(-a^2 / 2) h(a), and h(a) = e^(a^2 / 2) Phi(-a) is smooth in t = 1 / (1 +
// 0.3 a): a polynomial t P(t) of degree 8, fitted here by reweighted least squares of the relative error on [0, 16], is
// within 2.2e-7 of it (5.3e-7 evaluated in fp32), so the negative tail keeps its relative precision too. The same
// exponential gives Phi'. (With the library's erfc and exponential dz of 2048 x 12288 took 139 us, 53 so.)
// Its tanh form is z sigmoid(u), u = sqrt(8 / pi) (z + 0.044715 z^3), since (1 + tanh(u / 2)) / 2 = sigmoid(u).
__device__ __forceinline__ float gelu_tanh_u(float z) { return 1.5957691216057308f * (z + 0.044715f * z * z * z); }

// Phi(z); *e is e^(-z^2 / 2).
__device__ __forceinline__ float normal_cdf(float z, float* e) {
  const float t = __fdividef(1.f, fmaf(0.3f, fabsf(z), 1.f));
  float p = 0.034704924f;
  p = fmaf(p, t, -0.15318732f);
  p = fmaf(p, t, 0.19948818f);
  p = fmaf(p, t, -0.04742666f);
  p = fmaf(p, t, 0.12529191f);
  p = fmaf(p, t, 0.10088924f);
  p = fmaf(p, t, 0.12060054f);
  p = fmaf(p, t, 0.11963908f);
  *e = __expf(-0.5f * z * z);
  const float q = p * t * *e;
  return z < 0.f ? q : 1.f - q;
}

// Out of line: inlined many times over it would cost the epilogues their registers.
static __device__ __noinline__ float gelu(float z) {
  float e;
  return z * normal_cdf(z, &e);
}

__device__ __forceinline__ float act_fwd(int act, float z) {
  switch (act) {
    case TERN_ACT_RELU: return z < 0.f ? 0.f : z;  // NaN stays NaN
    case TERN_ACT_RELU2: return z < 0.f ? 0.f : z * z;
    case TERN_ACT_SILU:
    case TERN_ACT_GELU_TANH: return __fdividef(z, 1.f + __expf(act == TERN_ACT_SILU ? -z : -gelu_tanh_u(z)));
    case TERN_ACT_GELU: return gelu(z);
    default: return z;
  }
}

// act(z) and act'(z) together. The fast exponential and division are off by a few units of 2^-24 times
// (1 + |u|), far below the rounding to fp16 that follows.
__device__ __forceinline__ void act_both(int act, float z, float* f, float* df) {
  if (act == TERN_ACT_SILU || act == TERN_ACT_GELU_TANH) {
    const float u = act == TERN_ACT_SILU ? z : gelu_tanh_u(z);
    // sigmoid s = 1 / (1 + e^-u) and its complement e^-u s (not 1 - s: the tails keep their relative precision);
    // Past e^88 the quotient is 0 (its divisor lies between 2^126 and 2^128, where this division gives that): both products
    // with a finite z vanish, as they do in fp32 anyhow, and -inf gives NaN as in the formulas.
    const float e = __expf(fminf(-u, 88.f)), s = __fdividef(1.f, 1.f + e), c = e * s;
    const float du = act == TERN_ACT_SILU ? 1.f : 1.5957691216057308f * (1.f + 0.134145f * z * z);
    *f = z * s;
    *df = s + z * s * c * du;
  } else if (act == TERN_ACT_GELU) {
    float e;
    const float c = normal_cdf(z, &e);
    *f = z * c;
    *df = fmaf(0.39894228040143268f * z, e, c);
  } else {
    *f = act_fwd(act, z);
    // relu's is 0 at 0; NaN stays NaN
    *df = act == TERN_ACT_NONE ? 1.f : z > 0.f ? (act == TERN_ACT_RELU ? 1.f : 2.f * z) : (z <= 0.f ? 0.f : z);
  }
}

// f called with the activation as a compile-time constant.
template <int V> struct ActC { static constexpr int value = V; };
template <class F>
__device__ __forceinline__ void with_act(int act, F f) {
  switch (act) {
    case TERN_ACT_RELU: f(ActC<TERN_ACT_RELU>{}); break;
    case TERN_ACT_RELU2: f(ActC<TERN_ACT_RELU2>{}); break;
    case TERN_ACT_SILU: f(ActC<TERN_ACT_SILU>{}); break;
    case TERN_ACT_GELU: f(ActC<TERN_ACT_GELU>{}); break;
    case TERN_ACT_GELU_TANH: f(ActC<TERN_ACT_GELU_TANH>{}); break;
    default: f(ActC<TERN_ACT_NONE>{});
  }
}

// t of weight k of a packed row (any layout); an invalid code gives an unspecified t.
__device__ __forceinline__ float decode_t(int layout, const uint8_t* row, int64_t k) {
  if (layout == TERN_Q2_0_G128) {
    const int f = (row[k >> 2] >> (2 * (int)(k & 3))) & 3;
    return (float)((f & 1) - (f & 2));
  }
  if (layout == TERN_Q1_0_G128) return ((row[k >> 3] >> (int)(k & 7)) & 1) ? 1.f : -1.f;
  int v = row[k / 5];
  for (int i = (int)(k % 5); i > 0; i--) v /= 3;
  return (float)(v % 3) - 1.f;
}

}  // namespace tern
