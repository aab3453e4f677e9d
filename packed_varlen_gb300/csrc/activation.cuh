// Activations of the linear layers' epilogues, in fp32.
//
// Each is written so that no digits cancel: the logistic and the error function
// are taken of the side that is small, so a large negative argument gives
// a small result of full relative accuracy, down to bf16's subnormal numbers.  exp2 and
// the reciprocal are the approximate ones; with them the logistic is off by 2^-20 of
// itself (beside what its argument's rounding makes of it), far below the
// result's bf16 step.
#pragma once

#include <math.h>
#include <stdint.h>

#include "packedattn.h"
#include "tc_ptx.cuh"

namespace pa {

// v / (1 + 2^t) for t = u + 16.  2^t overflows, and its reciprocal is flushed to zero, where
// the result may still be 2^-120; with both terms of the divisor 2^-16 of what they are,
// everything stays within fp32's range as long as the result is a bf16 number.
__device__ __forceinline__ float over_one_plus_exp2(float v, float u) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;\n" : "=f"(r) : "f"(0x1p-16f + tc::ex2(u)));
  return v * (r * 0x1p-16f);
}

template <int kAct>
__device__ __forceinline__ float activation(float v) {
  if (kAct == PA_ACT_RELU) return v < 0.f ? 0.f : v;   // (a NaN stays)
  if (kAct == PA_ACT_SILU) return over_one_plus_exp2(v, fmaf(v, -1.4426950408889634f, -16.f));
  if (kAct == PA_ACT_GELU) return 0.5f * v * erfcf(v * -0.70710678118654752f);
  if (kAct == PA_ACT_GELU_TANH) {
    // (1 + tanh u) / 2 = 1 / (1 + e^-2u), u = sqrt(2 / pi) (v + 0.044715 v^3)
    constexpr float c = -2.f * 0.79788456080286536f * 1.4426950408889634f;
    return over_one_plus_exp2(v, fmaf(c * v, fmaf(0.044715f * v, v, 1.f), -16.f));
  }
  return v;
}

// The activation `act` of n values in place: one branch for all.
template <int n>
__device__ __forceinline__ void activate(float (&f)[n], int act) {
  auto all = [&](auto of) {
#pragma unroll
    for (int e = 0; e < n; ++e) f[e] = of(f[e]);
  };
  switch (act) {
    case PA_ACT_RELU: all([](float v) { return activation<PA_ACT_RELU>(v); }); break;
    case PA_ACT_SILU: all([](float v) { return activation<PA_ACT_SILU>(v); }); break;
    case PA_ACT_GELU: all([](float v) { return activation<PA_ACT_GELU>(v); }); break;
    case PA_ACT_GELU_TANH: all([](float v) { return activation<PA_ACT_GELU_TANH>(v); }); break;
    default: break;
  }
}

}  // namespace pa
