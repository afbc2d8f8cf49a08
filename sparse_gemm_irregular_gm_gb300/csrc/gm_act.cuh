// gm_act.cuh -- activations of the layers and their slopes. FINE: for results of 32 bits, by CUDA's functions; else with ex2
// and rcp: the share by which an activation multiplies z to about 2^-22 absolutely, and to 2^-15 of itself while it is over
// 2^-126 (z over -13 for gelu, -10 for gelu_tanh, -87 for silu): an eighth of a step of f16 at most. Slopes to 2^-21 absolutely.
#pragma once

#include <cuda_runtime.h>

#include "gm_layers.h"
#include "gm_umma.cuh"

namespace gm {

__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// exp(-z^2 / 2)
template <bool FINE>
__device__ __forceinline__ float bell(float z) {
  if constexpr (FINE) return expf(-0.5f * z * z);
  else return ex2(z * z * -0.72134752044f);
}

// Share of a standard normal below z: (1 + erf(z / sqrt 2)) / 2; b: bell(z), which it shares with the slope. In short: for
// z <= 0 it is b times a polynomial in t = 1 / (1 + 0.34 |z|), fitted here to erfcx(|z| / sqrt 2) / 2 up to |z| = 14 by
// reweighted least squares: off by 1.5e-7 at most, and by 1.5e-5 of itself, a 64th of a step of f16 and less of one of
// bf16, which keeps this tail down to z = -13. (A form good to 1.5e-7 alone was off by 0.4 % at -6 and 2 % at -10.)
template <bool FINE>
__device__ __forceinline__ float normal_below(float z, float b) {
  if constexpr (FINE) {
    return 0.5f * erfcf(z * -0.70710678f);
  } else {
    const float t = rcp(fmaf(fabsf(z), 0.34f, 1.f));
    float p = fmaf(t, 0.0439592674f, -0.196740165f);
    p = fmaf(t, p, 0.257386237f);
    p = fmaf(t, p, -0.0246442128f);
    p = fmaf(t, p, 0.153612018f);
    p = fmaf(t, p, 0.130469978f);
    p = fmaf(t, p, 0.135956869f);
    const float tail = t * p * b;
    return z < 0.f ? tail : 1.f - tail;
  }
}
template <bool FINE>
__device__ __forceinline__ float normal_below(float z) {
  return normal_below<FINE>(z, FINE ? 0.f : bell<FINE>(z));
}

// 1 / (1 + exp(-x))
template <bool FINE>
__device__ __forceinline__ float logistic(float x) {
  if constexpr (FINE) return 1.f / (1.f + expf(-x));
  else return rcp(1.f + ex2(x * -1.44269504089f));
}

// (1 + tanh(u)) / 2 = logistic(2 u), u = sqrt(2 / pi) (z + 0.044715 z^3)
constexpr float kTanhA = 1.5957691216f, kTanhB = 0.044715f;
__device__ __forceinline__ float gelu_tanh_arg(float z) { return z * fmaf(z * z, kTanhA * kTanhB, kTanhA); }

// z, or the end of [-most, most] that it lies beyond; NaN stays.
__device__ __forceinline__ float within(float z, float most) {
  float y;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(z), "f"(most));
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(y), "f"(-most));
  return y;
}

// act'(z). It is 0 or 1 in fp32 well before the ends that z is brought within, where the terms of an infinite z (a finite one
// kept in f16 may be) would give NaN.
template <bool FINE>
__device__ __forceinline__ float slope(float z, int act) {
  if (act == GM_ACT_RELU) return z > 0.f ? 1.f : 0.f;
  if (act == GM_ACT_GELU) {
    z = within(z, 30.f);
    const float b = bell<FINE>(z);
    return fmaf(z * 0.3989422804f, b, normal_below<FINE>(z, b));
  }
  if (act == GM_ACT_GELU_TANH) {
    z = within(z, 30.f);
    const float s = logistic<FINE>(gelu_tanh_arg(z));
    return fmaf(z * s * (1.f - s), fmaf(z * z, 3.f * kTanhA * kTanhB, kTanhA), s);
  }
  if (act == GM_ACT_SILU) {
    z = within(z, 128.f);
    const float s = logistic<FINE>(z);
    return s * fmaf(z, 1.f - s, 1.f);
  }
  return 1.f;
}

}  // namespace gm
