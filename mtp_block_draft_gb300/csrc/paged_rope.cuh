// Rotary angles of the cache's writers.
//
// Angles. Position p turns pair i by p f_i turns, f_i = theta^(-2i/hd) / 2 pi < 1. The host
// forms f_i in double and passes f_i 2^64 as an integer; p times that, modulo 2^64, is the angle's
// fraction of a turn in fixed point, which loses nothing more at far positions and needs none of
// the GPU's slow double arithmetic. What is left is f_i's own error: its power is off by
// (ln(theta) 2i/hd + 4) 2^-53 of itself at most, in turns less than 2^-53, so p 2^-53 at
// position p. The fraction goes to the sine as a 24-bit value and a first-order correction for the rest.
#pragma once

#include "paged.cuh"

namespace {

struct Turns {
  unsigned long long f[DMTP_OPS_MAX_HEAD_DIM / 2];
};

__device__ __forceinline__ float2 cos_sin_turns(unsigned long long frac) {
  const int hi = (int)(frac >> 32);                       // signed: [-1/2, 1/2) turns
  const float xh = __int2float_rn(hi);
  const long long rest = (long long)(frac - ((unsigned long long)(long long)xh << 32));
  const float d = __ll2float_rn(rest) * 3.4061215800304e-19f;  // 2 pi 2^-64
  float s, c;
  sincospif(xh * 4.656612873077393e-10f, &s, &c);          // 2 * 2^-32 half turns
  return make_float2(fmaf(-s, d, c), fmaf(c, d, s));
}

}  // namespace
