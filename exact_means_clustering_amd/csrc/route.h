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
// A chosen logit's score over exp(shift): its share of the row's sum, before the division.  A sigmoid is
// exp(z) / (1 + exp(z)), for z > 0 (where the shift is 0) 1 / (1 + exp(-z)).
__device__ __forceinline__ float share_term(float z, float shift, bool softmax) {
  const float e = exp_diff<F32>(z > 0.f && !softmax ? 0.f : z, shift);
  return softmax ? e : e * __builtin_amdgcn_rcpf(1.f + exp_diff<F32>(-fabsf(z), 0.f));
}

// A double as the halves that lane exchanges move.
template <int CTRL>
__device__ __forceinline__ double dpp64(double v) {
  const int lo = __double2loint(v), hi = __double2hiint(v);
  return __hiloint2double(__builtin_amdgcn_update_dpp(hi, hi, CTRL, 0xF, 0xF, true),
                          __builtin_amdgcn_update_dpp(lo, lo, CTRL, 0xF, 0xF, true));
}
// The values of the two lanes that are 16 (or FAR: 32) apart, in both of them.
template <bool FAR>
__device__ __forceinline__ void swap32(uint32_t v, uint32_t& a, uint32_t& b) {
  const auto p = FAR ? __builtin_amdgcn_permlane32_swap(v, v, false, false)
                     : __builtin_amdgcn_permlane16_swap(v, v, false, false);
  a = p[0], b = p[1];
}
template <bool FAR>
__device__ __forceinline__ void swap64(double v, double& a, double& b) {
  asm("s_nop 1" : "+v"(v));  // (two wait states between a write by inline code and the swap that reads it)
  uint32_t la, lb, ha, hb;
  swap32<FAR>((uint32_t)__double2loint(v), la, lb);
  swap32<FAR>((uint32_t)__double2hiint(v), ha, hb);
  a = __hiloint2double((int)ha, (int)la), b = __hiloint2double((int)hb, (int)lb);
}
// The value of lane i (the same i in all lanes).
__device__ __forceinline__ float lane_value(float v, int i) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), i));
}
__device__ __forceinline__ double lane_value(double v, int i) {
  return __hiloint2double(__builtin_amdgcn_readlane(__double2hiint(v), i),
                          __builtin_amdgcn_readlane(__double2loint(v), i));
}
// Reductions over the 64 lanes of a wave, in every lane.
template <class Op>
__device__ __forceinline__ double wave_op(double v, Op op) {
  v = op(v, dpp64<0xB1>(v));
  v = op(v, dpp64<0x4E>(v));
  v = op(v, dpp64<0x141>(v));
  v = op(v, dpp64<0x140>(v));
  double a, b;
  swap64<false>(v, a, b);
  v = op(a, b);
  swap64<true>(v, a, b);
  return op(a, b);
}
__device__ __forceinline__ double wave_max(double v) {
  return wave_op(v, [](double a, double b) { return __builtin_fmax(a, b); });
}
__device__ __forceinline__ uint32_t wave_min(uint32_t v) {
  auto d = [](uint32_t a, uint32_t b) { return a < b ? a : b; };
  v = d(v, (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, 0xB1, 0xF, 0xF, true));
  v = d(v, (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, 0x4E, 0xF, 0xF, true));
  v = d(v, (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, 0x141, 0xF, 0xF, true));
  v = d(v, (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, 0x140, 0xF, 0xF, true));
  uint32_t a, b;
  swap32<false>(v, a, b);
  v = d(a, b);
  swap32<true>(v, a, b);
  return d(a, b);
}

// A value into the largest two, m1 >= m2.
__device__ __forceinline__ void take2(double& m1, double& m2, double c) {
  m2 = __builtin_fmax(m2, __builtin_fmin(m1, c));
  m1 = __builtin_fmax(m1, c);
}
// The largest two of the values of all lanes of a wave, in every lane.
__device__ __forceinline__ void wave_top2(double& m1, double& m2) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) {
    const double a = __shfl_xor(m1, o), b = __shfl_xor(m2, o);
    take2(m1, m2, a);
    m2 = m2 < b ? b : m2;  // (b <= a)
  }
}

// The next choice of a wave's scores in the order of (score, index): pc and pk the one before, of which each lane has
// looked for the next (bc, bk; -inf and ~0 if it has none).  False if there is none.
__device__ __forceinline__ bool next_choice(double bc, uint32_t bk, double& pc, int64_t& pk) {
  pc = wave_max(bc);
  const uint32_t k = wave_min(bc == pc ? bk : ~0u);
  pk = k;
  return k != ~0u;  // uniform: every lane holds the same
}
// Which groups stay, from the worth of group `lane`.
__device__ __forceinline__ uint64_t groups_kept(double worth, int G, int keep) {
  const int lane = lane_id();
  int better = 0;
  for (int g = 0; g < G; ++g) {
    const double w = lane_value(worth, g);
    better += w > worth || (w == worth && g < lane);
  }
  return __ballot(lane < G && better < keep && worth > -INFINITY);
}
__device__ __forceinline__ double worth_of(double m1, double m2, int best) {
  return best == 2 && m2 > -INFINITY ? m1 + m2 : m1;
}

// The selections of one row with scores, by one wave in 64 bits: the choice of selection `lane`, or -1.  The K scores
// stay in the wave's LDS (c).  The row is valid and has no NaN (nor +inf under softmax).  Few calls come here: the code is
// kept small (one exponential, one quotient), since it is seldom in the instruction cache (about 8 us with 256 choices).
template <class T>
__device__ __forceinline__ int decide_row(const RouteArgs<T>& a, int64_t row, const float* bias, double* c) {
  const int lane = lane_id();
  const uint32_t K = a.K, gs = K / a.G;
  const typename T::raw* x = a.logits + row * a.K;
  float top = -INFINITY;
#pragma unroll 4
  for (uint32_t k = lane; k < K; k += 64) {
    const float f = T::to_f32(x[k]);
    top = fmaxf(top, f);
    c[k] = (double)f;
  }
  top = team_max<64>(top);
  double sum = 0.0;
#pragma unroll 1
  for (uint32_t k = lane; k < K; k += 64) {
    const double f = c[k], e = exp(a.softmax ? f - (double)top : -f);
    sum += e;
    c[k] = f == -INFINITY ? f : e;
  }
  sum = wave_op(sum, [](double a, double b) { return a + b; });
#pragma unroll 1
  for (uint32_t k = lane; k < K; k += 64) {
    const double e = c[k], s = (a.softmax ? e : 1.0) / (a.softmax ? sum : 1.0 + e);
    c[k] = e == -INFINITY ? e : s + (double)bias[k];
  }
  wave_sync();
  uint64_t kept = ~0ull;
  if (a.G > 1) {
    double m1 = -INFINITY, m2 = -INFINITY;
    if (lane < a.G) {
      uint32_t k = lane % gs;  // (lanes start at different places: banks)
#pragma unroll 4
      for (uint32_t i = 0; i < gs; ++i) {
        take2(m1, m2, c[lane * gs + k]);
        k = k + 1 < gs ? k + 1 : 0;
      }
    }
    kept = groups_kept(worth_of(m1, m2, a.best), a.G, a.keep);
  }
  int id = -1;
  double pc = INFINITY, bc = -INFINITY;
  int64_t pk = -1;
  uint32_t bk = ~0u;
  bool look = true;  // every lane for its first choice, then the lane whose choice was taken for its next one
#pragma unroll 1
  for (int j = 0; j < a.S; ++j) {
    if (look) {
      bc = -INFINITY, bk = ~0u;
#pragma unroll 4
      for (uint32_t k = lane; k < K; k += 64) {
        const double f = c[k];
        if ((kept >> (a.G > 1 ? k / gs : 0) & 1) && (f < pc || (f == pc && k > pk)) && f > bc) bc = f, bk = k;
      }
    }
    if (!next_choice(bc, bk, pc, pk)) break;
    look = bk == pk;
    if (lane == j) id = (int)pk;
  }
  return id;
}

// One row of any length by one wave, scores in 64 bits.  A lane keeps the kLaneBest best of its choices in registers, in
// order; the best of the lanes' first is the row's next selection, and a lane that has given all of them looks for more
// (they come in turn, so seldom).
constexpr int kLaneBest = 8;
template <class T>
__device__ __forceinline__ void route_row_exact(const RouteArgs<T>& a, int64_t row) {
  const int lane = lane_id();
  const uint32_t K = a.K;
  const typename T::raw* x = a.logits + row * a.K;
  const bool valid = !a.valid || a.valid[row];
  const bool arith = a.arith();
  float z = -INFINITY;  // of selection `lane`
  int id = -1;
  float total = 0.f;    // softmax: the sum of exp(logit - top)
  float top = -INFINITY;
  bool bad = false;
  if (valid) {
#pragma unroll 4
    for (uint32_t k = lane; k < K; k += 64) {
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
#pragma unroll 2
      for (uint32_t k = lane; k < K; k += 64) sum += exp((double)T::to_f32(x[k]) - (double)top);
      sum = wave_op(sum, [](double a, double b) { return a + b; });
      total = (float)sum;
    }
    auto key = [&](uint32_t k) {
      const double f = (double)T::to_f32(x[k]);
      if (!arith || f == -INFINITY) return f;
      const double e = exp(a.softmax ? f - (double)top : -f);
      const double s = (a.softmax ? e : 1.0) / (a.softmax ? sum : 1.0 + e);
      return a.bias ? s + (double)a.bias[k] : s;
    };
    const uint32_t gs = K / a.G;
    uint64_t kept = ~0ull;
    if (a.G > 1) {
      double worth = -INFINITY;  // of group `lane`
      for (int g = 0; g < a.G; ++g) {
        double m1 = -INFINITY, m2 = -INFINITY;
        for (uint32_t k = g * gs + lane; k < (g + 1) * gs; k += 64) take2(m1, m2, key(k));
        wave_top2(m1, m2);
        if (lane == g) worth = worth_of(m1, m2, a.best);
      }
      kept = groups_kept(worth, a.G, a.keep);
    }
    double pc = INFINITY, best[kLaneBest];  // the selection before, and the lane's best
    int64_t pk = -1;
    uint32_t at[kLaneBest];
    int given = 0;
    bool look = true, more = false;  // more: choices behind the lane's best
    for (int j = 0; j < a.S; ++j) {
      if (look) {
#pragma unroll
        for (int i = 0; i < kLaneBest; ++i) best[i] = -INFINITY, at[i] = ~0u;
        for (uint32_t k = lane; k < K; k += 64) {
          if (!(kept >> (a.G > 1 ? k / gs : 0) & 1)) continue;
          const double f = key(k);
          if (!(f > best[kLaneBest - 1]) || !(f < pc || (f == pc && k > pk))) continue;
#pragma unroll
          for (int i = kLaneBest - 1; i >= 0; --i) {  // (of equal scores the one in front came first)
            const bool down = i > 0 && f > best[i > 0 ? i - 1 : 0], here = !down && f > best[i];
            best[i] = down ? best[i > 0 ? i - 1 : 0] : here ? f : best[i];
            at[i] = down ? at[i > 0 ? i - 1 : 0] : here ? k : at[i];
          }
        }
        given = 0, more = best[kLaneBest - 1] > -INFINITY;
      }
      if (!next_choice(best[0], at[0], pc, pk)) break;
      look = false;
      if (at[0] == pk) {
#pragma unroll
        for (int i = 0; i + 1 < kLaneBest; ++i) best[i] = best[i + 1], at[i] = at[i + 1];
        best[kLaneBest - 1] = -INFINITY, at[kLaneBest - 1] = ~0u;
        look = ++given == kLaneBest && more;
      }
      if (lane == j) id = (int)pk;
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
