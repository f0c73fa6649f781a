// gated_util.h -- the gates of the gated linear recurrence (gfx950): what a
// token makes of its two gate inputs, in fp32.
#pragma once

#include "device_util.h"

namespace ssm {

// A channel's parameters as the gates use them.
struct Channel {
  float A, A_log2e, A_kept;   // A_kept: A, or 0 where A > 0
  float r_off, i_off;         // the biases times -log2 e
};
__device__ __forceinline__ Channel channel_of(float A, float r_bias, float i_bias) {
  return {A, A * kLog2e, A < 0.0f ? A : 0.0f, -r_bias * kLog2e, -i_bias * kLog2e};
}

// sigma(v + bias), off = -bias log2 e
__device__ __forceinline__ float sigmoid_off(float v, float off) { return fast_rcp(1.0f + fast_exp2(fmaf(v, -kLog2e, off))); }

struct Gates {
  float rho, iota;   // sigma of the two gates
  float a;           // exp(A rho)
  float m2;          // 1 - a^2, 0 where A >= 0
};

// 1 - a^2 = -2 a sinh(y), y = log a: as a difference it would lose the bits
// that a long memory is made of (a = 0.999: 9 of them).  The series ends with
// y^5, whose next term is 5e-8 of it at |y| = 0.25; from there on the difference
// is as exact (its two roundings, 6e-8 of 1, against 0.39 and more).
__device__ __forceinline__ Gates gates_of(float r, float i, const Channel &c) {
  Gates g;
  g.rho = sigmoid_off(r, c.r_off);
  g.iota = sigmoid_off(i, c.i_off);
  g.a = fast_exp2(c.A_log2e * g.rho);
  const float y = c.A_kept * g.rho, y2 = y * y;
  const float s = fmaf(y2, fmaf(y2, -1.0f / 60.0f, -1.0f / 3.0f), -2.0f);
  g.m2 = y > -0.25f ? g.a * y * s : fmaf(-g.a, g.a, 1.0f);
  return g;
}

}  // namespace ssm
