// Activations of the linear layers' epilogues, in fp32.
//
// Each is written so that no digits cancel: the logistic and the error function
// are taken of the side that is small, so a large negative argument gives
// a small result of full relative accuracy.  exp2 and the reciprocal are the
// approximate ones (2^-22 relative each), far below the result's bf16 step.
#pragma once

#include <math.h>
#include <stdint.h>

#include "packedattn.h"
#include "tc_ptx.cuh"

namespace pa {

// v / (1 + 2^t): v times the logistic function of -t ln 2.
__device__ __forceinline__ float over_one_plus_exp2(float v, float t) {
  return __fdividef(v, 1.f + tc::ex2(t));
}

template <int kAct>
__device__ __forceinline__ float activation(float v) {
  if (kAct == PA_ACT_RELU) return v < 0.f ? 0.f : v;   // (a NaN stays)
  if (kAct == PA_ACT_SILU) return over_one_plus_exp2(v, v * -1.4426950408889634f);
  if (kAct == PA_ACT_GELU) return 0.5f * v * erfcf(v * -0.70710678118654752f);
  if (kAct == PA_ACT_GELU_TANH) {
    // (1 + tanh u) / 2 = 1 / (1 + e^-2u), u = sqrt(2 / pi) (v + 0.044715 v^3)
    constexpr float c = -2.f * 0.79788456080286536f * 1.4426950408889634f;
    return over_one_plus_exp2(v, c * v * fmaf(0.044715f * v, v, 1.f));
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
