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

// exp(-(v + bias)), off = -bias log2 e, of which sigma(v + bias) = 1 / (1 + w).  The
// exponent is rounded once to a float, so sigma is off by (3 |v| + 5) 2^-24 of it at
// the most; the sum v + bias in fp32 alone would be off as much as |v| 2^-24 makes.
__device__ __forceinline__ float gate_exp(float v, float off) { return fast_exp2(fmaf(v, -kLog2e, off)); }
// 1 - sigma = w sigma: as a difference it would be off by sigma's last bit, and at
// v = 12, where it is 6e-6, keep six bits.  (Clamped in the product's own
// instruction; inf 0 of a gate whose sigma is 0 becomes 0.)
__device__ __forceinline__ float shut(float w, float sigma) { return fminf(fmaxf(w * sigma, 0.0f), 1.0f); }

// sigma and 1 - sigma in a register: the smaller one, with a minus where it is
// sigma itself.
__device__ __forceinline__ float fold_gate(float w, float sigma) { return w < 1.0f ? w * sigma : -sigma; }
__device__ __forceinline__ void unfold_gate(float v, float &sigma, float &shut) {
  const float less = fabsf(v), more = 1.0f - less;
  const bool is = __float_as_int(v) < 0;
  sigma = is ? less : more;
  shut = is ? more : less;
}

struct Gates {
  float w_r, w_i;    // exp(-v) of the two gates
  float rho, iota;   // sigma of them
  float a;           // exp(A rho)
  float m2;          // 1 - a^2, 0 where A >= 0
};

// 1 - a^2 = -2 a sinh(y), y = log a: as a difference it would lose the bits
// that a long memory is made of (a = 0.999: 9 of them).  The series ends with
// y^5, whose next term is 5e-8 of it at |y| = 0.25; from there on the difference
// is as exact (its two roundings, 6e-8 of 1, against 0.39 and more).
__device__ __forceinline__ Gates gates_of(float r, float i, const Channel &c) {
  Gates g;
  g.w_r = gate_exp(r, c.r_off);
  g.w_i = gate_exp(i, c.i_off);
  g.rho = fast_rcp(1.0f + g.w_r);
  g.iota = fast_rcp(1.0f + g.w_i);
  g.a = fast_exp2(c.A_log2e * g.rho);
  const float y = c.A_kept * g.rho, y2 = y * y;
  const float s = fmaf(y2, fmaf(y2, -1.0f / 60.0f, -1.0f / 3.0f), -2.0f);
  g.m2 = y > -0.25f ? g.a * y * s : fmaf(-g.a, g.a, 1.0f);
  return g;
}

}  // namespace ssm
