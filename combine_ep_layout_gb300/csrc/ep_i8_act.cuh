// ep_i8_act.cuh -- the gate's activation of the int8 products.
#pragma once

#include "ep_gb300_i8.h"

namespace epg {

// v sigmoid(s): silu with s = v; the tanh form of gelu is the same with
// s = 2 sqrt(2 / pi) (v + 0.044715 v^3), as (1 + tanh(u)) / 2 is sigmoid(2 u).  The exponential
// is off by 2^-22 and by the rounding of its argument, |s| 2^-23, which sigmoid's slope takes
// to under 4 2^-24 of |v|.
__device__ __forceinline__ float i8_activate(int act, float v) {
  const float s = act == EP_ACT_SILU ? v : v * fmaf(0.07135481282553f * v, v, 1.5957691216057308f);
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(-1.4426950408889634f * s));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
  return v * r;
}

}  // namespace epg
