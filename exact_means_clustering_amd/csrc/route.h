// Routing of rows to choices: what its kernels share (internal; formulas in flashkm_train.h).
#pragma once

#include "kernels.h"
#include "teams.h"
#include "vecio.h"

namespace fkm {

// One call's arguments, as the kernels take them.
template <class T>
struct RouteArgs {
  const typename T::raw* logits;
  int64_t n;
  int K;
  const float* bias;
  int G, keep, best, S;
  int softmax, renorm;
  float scale;
  const uint8_t* valid;
  int32_t* ids;
  float* weights;
  float* chosen;
  // whether c's order is not the logits' own: c is computed, and its order near a border is decided in 64 bits
  __host__ __device__ bool arith() const { return bias || (G > 1 && best == 2 && K > G); }
};

// What waits in LDS between lanes of one wave: its accesses keep their order.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

__device__ __forceinline__ bool is_nan_bits(float x) { return (__float_as_uint(x) & 0x7FFFFFFFu) > 0x7F800000u; }

// exp(t) for t <= 88 (no overflow, so that no step has inf * 0).
__device__ __forceinline__ float exp_to(float t) { return exp_diff<F32>(t < 88.f ? t : 88.f, 0.f); }

// The shift of a row's shares, from its largest chosen logit.
__device__ __forceinline__ float share_shift(float high, bool softmax) {
  if (high == -INFINITY) return 0.f;
  return softmax ? high : fminf(high, 0.f);
}
// A chosen logit's score over exp(shift): its share of the row's sum, before the division.
__device__ __forceinline__ float share_term(float z, float shift, bool softmax) {
  const float e = exp_diff<F32>(z, shift);
  if (softmax) return e;
  // exp(z - shift) / (1 + exp(z)), or where that could overflow 1 / (1 + exp(-z)) (the shift is 0 then)
  return z > 0.f ? 1.f / (1.f + exp_to(-z)) : e / (1.f + exp_to(z));
}

// The largest two of the values of all lanes of a wave, m1 >= m2, in every lane.
__device__ __forceinline__ void wave_top2(double& m1, double& m2) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) {
    const double a = __shfl_xor(m1, o), b = __shfl_xor(m2, o);
    const double low = m1 < a ? m1 : a;
    m1 = m1 < a ? a : m1;
    m2 = m2 < b ? b : m2;
    m2 = m2 < low ? low : m2;
  }
}

// One row by one wave, scores in 64 bits.  Selection after selection, the next choice in the order of (score, index) is
// looked for over the whole row, whose scores are computed again each time: no storage, any K.
template <class T>
__device__ __forceinline__ void route_row_exact(const RouteArgs<T>& a, int64_t row) {
  const int lane = lane_id();
  const typename T::raw* x = a.logits + row * a.K;
  const bool valid = !a.valid || a.valid[row];
  const bool arith = a.arith();
  float z = -INFINITY;  // of selection `lane`
  int id = -1;
  float total = 0.f;    // softmax: the sum of exp(logit - top)
  float top = -INFINITY;
  bool bad = false;
  if (valid) {
    for (int64_t k = lane; k < a.K; k += 64) {
      const float f = T::to_f32(x[k]);
      bad |= is_nan_bits(f) || (a.bias && is_nan_bits(a.bias[k]));
      top = fmaxf(top, f);
    }
    top = team_max<64>(top);
    bad = __ballot(bad) != 0 || (a.softmax && top == INFINITY);
  }
  if (valid && !bad && top > -INFINITY) {
    double sum = 0.0;
    if (a.softmax && (arith || !a.renorm)) {
      for (int64_t k = lane; k < a.K; k += 64) sum += exp((double)T::to_f32(x[k]) - (double)top);
      sum = wave_sum_f64(sum);
      total = (float)sum;
    }
    auto key = [&](int64_t k) {
      const double f = (double)T::to_f32(x[k]);
      if (!arith || f == -INFINITY) return f;
      double s = a.softmax ? exp(f - (double)top) / sum : 1.0 / (1.0 + exp(-f));
      if (a.bias) s += (double)a.bias[k];
      return s;
    };
    const int gs = a.K / a.G;
    uint64_t kept = ~0ull;
    if (a.G > 1) {
      double worth = -INFINITY;  // of group `lane`
      for (int g = 0; g < a.G; ++g) {
        double m1 = -INFINITY, m2 = -INFINITY;
        for (int64_t k = (int64_t)g * gs + lane; k < (int64_t)(g + 1) * gs; k += 64) {
          const double c = key(k);
          const double low = c < m1 ? c : m1;
          m1 = c < m1 ? m1 : c;
          m2 = m2 < low ? low : m2;
        }
        wave_top2(m1, m2);
        if (lane == g) worth = a.best == 2 && m2 > -INFINITY ? m1 + m2 : m1;
      }
      int better = 0;
      for (int g = 0; g < a.G; ++g) {
        const double w = __shfl(worth, g);
        better += w > worth || (w == worth && g < lane);
      }
      kept = __ballot(lane < a.G && better < a.keep && worth > -INFINITY);
    }
    double pc = INFINITY;  // the selection before
    int64_t pk = -1;
    for (int j = 0; j < a.S; ++j) {
      double bc = -INFINITY;
      int64_t bk = INT64_MAX;
      for (int64_t k = lane; k < a.K; k += 64) {
        if (!(kept >> (a.G > 1 ? k / gs : 0) & 1)) continue;
        const double c = key(k);
        if ((c < pc || (c == pc && k > pk)) && c > bc) bc = c, bk = k;
      }
#pragma unroll
      for (int o = 32; o >= 1; o >>= 1) {
        const double c = __shfl_xor(bc, o);
        const int64_t k = __shfl_xor((long long)bk, o);
        if (c > bc || (c == bc && k < bk)) bc = c, bk = k;
      }
      if (bk == INT64_MAX) break;  // uniform: every lane holds the same
      if (lane == j) id = (int)bk;
      pc = bc, pk = bk;
    }
    if (id >= 0) z = T::to_f32(x[id]);
  }
  float w;
  if (a.renorm) {
    const float shift = share_shift(team_max<64>(z), a.softmax);
    const float t = id >= 0 ? share_term(z, shift, a.softmax) : 0.f;
    const float sum = team_sum<64>(t);
    w = id >= 0 ? a.scale * (t / sum) : 0.f;
  } else {
    w = id < 0 ? 0.f : a.softmax ? a.scale * (exp_diff<F32>(z, top) / total) : a.scale * (1.f / (1.f + exp_to(-z)));
  }
  if (bad) w = z = __uint_as_float(0x7FC00000u);
  if (lane < a.S) {
    const int64_t at = row * a.S + lane;
    a.ids[at] = id;
    a.weights[at] = w;
    a.chosen[at] = z;
  }
}

}  // namespace fkm
