// gated_util.h -- the gates of the gated linear recurrence (gfx950): what a
// token makes of its two gate inputs, in fp32.
#pragma once

#include "device_util.h"

namespace ssm {

__device__ __forceinline__ float sigmoid_f(float v) { return fast_rcp(1.0f + fast_exp2(-v * kLog2e)); }

struct Gates {
  float rho, iota;   // sigma of the two gates
  float a;           // exp(A rho)
  float m, inv_m;    // sqrt(1 - a^2) and its reciprocal, both 0 where nothing is left of 1 - a^2
};

// 1 - a^2 = -2 a sinh(y), y = log a: as a difference it would lose the bits
// that a long memory is made of (a = 0.999: 2^-9 of them).  The series ends
// with y^7; from |y| = 0.5 on (next term 1e-8 there) the difference is exact
// enough.
__device__ __forceinline__ Gates gates_of(float r, float i, float A) {
  Gates g;
  g.rho = sigmoid_f(r);
  g.iota = sigmoid_f(i);
  const float y = A * g.rho;
  g.a = fast_exp2(y * kLog2e);
  const float y2 = y * y;
  const float s = fmaf(y2, fmaf(y2, fmaf(y2, 1.0f / 5040.0f, 1.0f / 120.0f), 1.0f / 6.0f), 1.0f);
  const float m2 = y > -0.5f ? -2.0f * g.a * y * s : fmaf(-g.a, g.a, 1.0f);
  g.inv_m = m2 > 1e-37f ? __builtin_amdgcn_rsqf(m2) : 0.0f;   // (A > 0: nothing)
  g.m = m2 > 1e-37f ? m2 * g.inv_m : 0.0f;
  return g;
}

}  // namespace ssm
