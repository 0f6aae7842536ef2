// Rows held by teams of lanes: exponentials relative to a row's maximum, and reductions over the lanes of a team
// (internal).
#pragma once

#include "common.h"

namespace fkm {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// exp(x - shift).  The product with log2(e) rounds to |x - shift| 2^-24 of the
// result, which is lost in a 16-bit gradient; for fp32 logits the product's
// rounding and log2(e)'s own are put back to first order.
template <class T>
__device__ __forceinline__ float exp_diff(float x, float shift) {
  const float t = x - shift;
  if constexpr (T::SZ == 4) {
    constexpr float kLog2eLow = 1.925963033500757e-8f;
    const float c = t < -150.f ? -150.f : t;  // exp is 0 there; NaN stays
    const float y = c * kLog2e;
    const float r = fmaf(c, kLog2eLow, fmaf(c, kLog2e, -y));
    const float e = __builtin_amdgcn_exp2f(y);
    return fmaf(e, r * kLn2, e);
  } else {
    return __builtin_amdgcn_exp2f(t * kLog2e);
  }
}

// The value of the lane paired with this one: neighbours, pairs, then mirrored
// halves of 8 and 16 lanes (within which every lane already holds the same).
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  const int i = __float_as_int(v);
  return __int_as_float(__builtin_amdgcn_update_dpp(i, i, CTRL, 0xF, 0xF, true));
}
// op over the LPR lanes of a team (a power of two, aligned), in every lane.
// All lanes of the wave take part.
template <int LPR, class Op>
__device__ __forceinline__ float team_op(float v, Op op) {
  if constexpr (LPR >= 2) v = op(v, dpp<0xB1>(v));    // quad_perm 1,0,3,2
  if constexpr (LPR >= 4) v = op(v, dpp<0x4E>(v));    // quad_perm 2,3,0,1
  if constexpr (LPR >= 8) v = op(v, dpp<0x141>(v));   // row_half_mirror
  if constexpr (LPR >= 16) v = op(v, dpp<0x140>(v));  // row_mirror
  if constexpr (LPR >= 32) {
    const auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = op(__uint_as_float(p[0]), __uint_as_float(p[1]));
  }
  if constexpr (LPR >= 64) {
    const auto p = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = op(__uint_as_float(p[0]), __uint_as_float(p[1]));
  }
  return v;
}
// Maximum of E values, two at a time (fmaxf would first canonicalise each value
// unpacked from a word: one instruction more per value).  A NaN may win or lose:
// the row's exponentials are NaN either way.
template <int E>
__device__ __forceinline__ float max_of(const float (&x)[E]) {
  static_assert(E % 2 == 0, "pairs");
  float m = x[0];
  asm("v_max_f32 %0, %1, %2" : "=v"(m) : "v"(x[0]), "v"(x[1]));
#pragma unroll
  for (int e = 2; e < E; e += 2) asm("v_max3_f32 %0, %1, %2, %3" : "=v"(m) : "v"(m), "v"(x[e]), "v"(x[e + 1]));
  return m;
}
template <int LPR>
__device__ __forceinline__ float team_max(float v) {
  return team_op<LPR>(v, [](float a, float b) { return fmaxf(a, b); });
}
template <int LPR>
__device__ __forceinline__ float team_sum(float v) {
  return team_op<LPR>(v, [](float a, float b) { return a + b; });
}

}  // namespace fkm
