// Routing of rows whose K choices a team of lanes holds in registers (internal).
//
// A key is the 64-bit pattern (score, index), made so that the order of the patterns, read as doubles, is the order of
// the selection: the score's own 32 bits on top, and below them the index, inverted for scores that are not negative, so
// that of equal scores the lower index is the larger key.  The patterns are finite doubles whatever the scores (a NaN's
// row is found before), so v_max_f64 and v_min_f64, full-rate here, are a compare-exchange of two instructions that
// carries the index along and is exact.  A lane sorts its keys eight (or L) at a time, keeps the largest L, and the
// lists of a team's lanes are joined by bitonic merges: after log2(LPR) steps every lane holds the row's L largest keys in
// order.
//
// Where c's order is the logits' own, a key's score is the logit.  Else it is c in 32 bits, and a bound of its error says
// what rounding could have changed.  Where two neighbours of the selection are closer than their errors, or one choice
// that is not selected is as close to the last one, the row's candidates are put in order by their c in 64 bits, one a
// lane (unless the two have the same logit and bias: their order is the index's).  What is still open after that (more
// such choices, groups whose worths are closer than their errors, and probabilities that their common divisor in 32 bits
// leaves undecided), a few rows in ten thousand on random scores, is decided by the whole wave, all in 64 bits.
//
// Bound by vector instructions, not by the bytes: 630 of them for a lane's 32 values in rows of 1,024 bf16 of which two are
// taken (softmax, keys, sort, merges).  262,144 such rows are 80,500 of them a SIMD, of four cycles each: 134 us at 2.4 GHz,
// which is what they take (4.0 TB/s of logits; fp32, half the rows, 89 us and 6.0 TB/s).  So a row goes straight into
// registers, 16 bytes a lane and load, and a lane holds 32 values: the more it sorts alone, the fewer merges across lanes.
// Measured besides: 32,768 x 128 bf16, eight a row, 6.6 us; 65,536 x 256 fp32 plain 15, with sigmoids and a bias 30, and in
// 8 groups 43 (a row decided as a whole holds its wave up for 7 us: where most rows are left open, as in a router that
// starts at zero, up to 370).
#pragma once

#include "route.h"

namespace fkm {

__device__ __forceinline__ double key_of(float score, uint32_t col) {
  const uint32_t hi = __float_as_uint(score + 0.f);  // (-0 is 0)
  const uint32_t lo = ~(col ^ (uint32_t)((int32_t)hi >> 31));
  return __hiloint2double((int)hi, (int)lo);
}
__device__ __forceinline__ float key_score(double k) { return __int_as_float(__double2hiint(k)); }
__device__ __forceinline__ uint32_t key_col(double k) {
  return ~((uint32_t)__double2loint(k) ^ (uint32_t)(__double2hiint(k) >> 31));
}

// The larger and the smaller key.  (As instructions: the compiler would first quiet a NaN in each key that comes from
// integers, one v_max_f64 more for each, and no key is one.)
__device__ __forceinline__ double key_max(double a, double b) {
  double m;
  asm("v_max_f64 %0, %1, %2" : "=v"(m) : "v"(a), "v"(b));
  return m;
}
__device__ __forceinline__ double key_min(double a, double b) {
  double m;
  asm("v_min_f64 %0, %1, %2" : "=v"(m) : "v"(a), "v"(b));
  return m;
}
// a >= b afterwards
__device__ __forceinline__ void exchange(double& a, double& b) {
  const double h = key_max(a, b), l = key_min(a, b);
  a = h, b = l;
}
// Odd-even merge sort, descending.
template <int L>
__device__ __forceinline__ void sort_keys(double (&a)[L]) {
#pragma unroll
  for (int p = 1; p < L; p *= 2)
#pragma unroll
    for (int k = p; k >= 1; k /= 2)
#pragma unroll
      for (int j = k % p; j + k < L; j += 2 * k)
#pragma unroll
        for (int i = 0; i < k; ++i)
          if (i + j + k < L && (i + j) / (2 * p) == (i + j + k) / (2 * p)) exchange(a[i + j], a[i + j + k]);
}
// The L largest of two descending lists, descending.
template <int L>
__device__ __forceinline__ void merge_keys(double (&a)[L], const double (&b)[L]) {
#pragma unroll
  for (int i = 0; i < L; ++i) a[i] = key_max(a[i], b[L - 1 - i]);
#pragma unroll
  for (int h = L / 2; h >= 1; h /= 2)
#pragma unroll
    for (int i = 0; i < L; ++i)
      if (!(i & h)) exchange(a[i], a[i + h]);
}
template <int L, int CTRL>
__device__ __forceinline__ void merge_dpp(double (&a)[L]) {
  double b[L];
#pragma unroll
  for (int i = 0; i < L; ++i) b[i] = dpp64<CTRL>(a[i]);
  merge_keys<L>(a, b);
}
template <int L, bool FAR>
__device__ __forceinline__ void merge_swap(double (&a)[L]) {  // lanes 16 (or 32) apart
  double b[L];
#pragma unroll
  for (int i = 0; i < L; ++i) swap64<FAR>(a[i], a[i], b[i]);
  merge_keys<L>(a, b);
}
// The L largest keys of a team's lists, in every lane.
template <int L, int LPR>
__device__ __forceinline__ void join_lists(double (&a)[L]) {
  if constexpr (LPR >= 2) merge_dpp<L, 0xB1>(a);
  if constexpr (LPR >= 4) merge_dpp<L, 0x4E>(a);
  if constexpr (LPR >= 8) merge_dpp<L, 0x141>(a);
  if constexpr (LPR >= 16) merge_dpp<L, 0x140>(a);
  if constexpr (LPR >= 32) merge_swap<L, false>(a);
  if constexpr (LPR >= 64) merge_swap<L, true>(a);
}

// The part of a row (K choices, LPR * E at most) that a team's lanes hold: load j of lane g takes V columns from
// (j LPR + g) V on, 16 bytes; -inf where there are none.  Rows that are no multiple of 16 bytes or start anywhere (loose)
// are loaded at element alignment, their last few elements one by one.
template <class T, int E, int LPR>
struct Slice {
  static constexpr int V = 16 / T::SZ, NV = E / V;
  Pack<T, V> p[NV];
  static __device__ __forceinline__ int first(int j, int g) { return j * LPR * V + g * V; }
  // (ONCE: nothing of the row is read again)
  template <bool ONCE>
  __device__ __forceinline__ void load(const typename T::raw* row, int K, int g, bool loose, bool live) {
    if (!loose) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        p[j].fill_neg_inf();
        if (live && first(j, g) < K) {
          if constexpr (ONCE) p[j].load_nt(row + first(j, g));
          else p[j].load(row + first(j, g));
        }
      }
    } else {
      // one load of the row, j = tail of one lane, has fewer than V elements
      const int tail = K / (LPR * V), left = K % V;
      Pack<T, V> last;
      last.fill_neg_inf();
      const bool mine = live && left && first(tail, g) + left == K;
      if (mine) last.load_head(row + (K - left), left);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        p[j].fill_neg_inf();
        if (live && first(j, g) + V <= K) p[j].load_loose(row + first(j, g));
        if (mine && j == tail) p[j] = last;
      }
    }
  }
  __device__ __forceinline__ void values(float (&x)[E]) const {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float f[V];
      p[j].unpack(f);
#pragma unroll
      for (int v = 0; v < V; ++v) x[j * V + v] = f[v];
    }
  }
  // whether an element is NaN
  __device__ __forceinline__ bool has_nan() const {
    if constexpr (T::SZ == 2) {
      typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
      u16x2 m = 0;
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, p[j].w[i] & 0x7FFF7FFFu));
      const uint32_t inf = neg_inf_bits<T>() & 0x7FFFu;
      return m[0] > inf || m[1] > inf;
    } else {
      bool nan = false;
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) nan |= __uint_as_float(p[j].w[i]) != __uint_as_float(p[j].w[i]);
      return nan;
    }
  }
};

// The list's L largest joined with those of a lane's E values, the first of which has index `col`.
template <class T, int E, int LPR, int L>
__device__ __forceinline__ void add_keys(double (&top)[L], const float (&x)[E], int col, bool fresh) {
  using Sl = Slice<T, E, LPR>;
  static_assert(E % L == 0, "whole lists");
#pragma unroll
  for (int e0 = 0; e0 < E; e0 += L) {
    double k[L];
#pragma unroll
    for (int i = 0; i < L; ++i) k[i] = key_of(x[e0 + i], col + Sl::first((e0 + i) / Sl::V, 0) + (e0 + i) % Sl::V);
    sort_keys<L>(k);
    if (fresh && e0 == 0) {
#pragma unroll
      for (int i = 0; i < L; ++i) top[i] = k[i];
    } else {
      merge_keys<L>(top, k);
    }
  }
}

// Sum of a lane's values, pair by pair.
template <int E>
__device__ __forceinline__ float pair_sum(const float (&x)[E]) {
  float s[E];
#pragma unroll
  for (int e = 0; e < E; ++e) s[e] = x[e];
#pragma unroll
  for (int h = E / 2; h >= 1; h /= 2)
#pragma unroll
    for (int e = 0; e < h; ++e) s[e] += s[e + h];
  return s[0];
}

// exp(x - shift) to (2 |x - shift| + 3) u, and the sigmoid of x (0 for -inf).
__device__ __forceinline__ float quick_exp(float x, float shift) { return exp_diff<BF16>(x, shift); }
__device__ __forceinline__ float quick_sigmoid(float x) {
  return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-kLog2e * x));
}

constexpr float kU = 0x1p-24f;
// Bounds of the error of c in 32 bits: for a probability p = exp(t) / sum, (2 |t| + 3) u for the exponential (the
// difference's rounding and its scaling), 18 u for the sum of such (5 levels in a lane, 6 across, and its terms' own, of
// which |t| exp(t) is at most 0.37) and 3 u for the quotient; for a sigmoid s, 0.8 u for the exponential (s (1 - s) |t| is
// at most 0.23), u for 1 + e and u for the reciprocal; for c itself u |c|.  (2^-120: what is flushed below the normal
// range.)  score_error is without the last, for every choice of a row: (2 |t| + 28) exp(t) is at most 28.
__device__ __forceinline__ float score_error(bool softmax, float inv) { return softmax ? 28.f * inv : 3.f; }
__device__ __forceinline__ float pair_error(bool softmax, float high, float inv, float z, float c) {
  const float t = z - high;
  return kU * ((softmax ? quick_exp(z, high) * inv * (28.f - 2.f * t) : 3.f) + fabsf(c)) + 0x1p-120f;
}

// One wave's LDS, in floats, for rows of K choices taken SL at a time, S selections each.
struct RouteLds {
  int worth, z, e, exact, info, flag, extra, total;
  static __host__ __device__ RouteLds of(int SL, int K, int G, int S, bool scored) {
    RouteLds o{};
    // groups first: a row's scores (or the largest two of four, and a place a group), its groups' worths, and whether
    // they stay
    const int fours = 2 * SL * (K / 4 + G), ones = SL * ((K + 3) & ~3);
    o.worth = G > 1 ? (fours > ones ? fours : ones) : 0;
    const int groups = o.worth + (G > 1 ? 2 * SL * G : 0);
    // then, in the same place, the selections: keys, logits, shares before the division
    o.z = 2 * SL * S, o.e = o.z + SL * S;
    int at = o.e + SL * S;
    if (at < groups) at = groups;
    at = (at + 1) & ~1;
    o.exact = at, at += scored ? 2 * K : 0;  // one row's scores in 64 bits
    o.extra = at, at += scored ? 2 * SL : 0;  // the key of a choice that may belong to the selection
    o.info = at, at += 2 * SL;               // a row's largest logit, 1 / sum of exponentials
    o.flag = at, at += SL;                   // kOpen, kLast, kCopies
    o.total = (at + 3) & ~3;
    return o;
  }
};
// A row whose candidates are put in order in 64 bits, one that is so as a whole, and one whose extra candidate has copies
// (of the same logit and bias) behind it.
constexpr int kOpen = 2, kLast = 1, kCopies = 4;

// What a kernel is made for: rows of K <= LPR * E choices whose order is the logits' own; the same of any K, taken
// LPR * E at a time; and rows of K <= LPR * E with scores, a bias or groups.
enum RouteMode { kPlain, kWide, kScored };

template <class T, int E, int LPR, int L, RouteMode MODE>
__global__ __launch_bounds__(256, L == 32 ? 2 : MODE == kScored && (E == 32 || L == 16) ? 3 : 4) void route_rows_kernel(
    RouteArgs<T> a, bool loose, RouteLds o, uint32_t magic, uint32_t group_magic) {
  using Sl = Slice<T, E, LPR>;
  constexpr int V = Sl::V, NV = Sl::NV, SL = 64 / LPR;
  extern __shared__ __align__(16) float lds_all[];
  const int lane = lane_id(), slot = lane / LPR;
  int g = lane % LPR;
  float* lds = lds_all + (threadIdx.x >> 6) * o.total;
  double* sel = reinterpret_cast<double*>(lds);
  float *zs = lds + o.z, *es = lds + o.e, *info = lds + o.info;
  int* flag = reinterpret_cast<int*>(lds + o.flag);
  const bool arith = MODE == kScored && a.arith();
  const bool sums = a.softmax && (arith || !a.renorm);
  const int S = a.S;
  const int64_t waves = (int64_t)gridDim.x * (blockDim.x >> 6);
  const int64_t tiles = (a.n + SL - 1) / SL;
  const uint64_t team = LPR == 64 ? ~0ull : ((1ull << (LPR & 63)) - 1) << (slot * LPR);

  Sl next;
  bool next_live = false;
  auto fetch = [&](int64_t t) {
    const int64_t row = t * SL + slot;
    next_live = t < tiles && row < a.n && (!a.valid || a.valid[row]);
    if constexpr (MODE != kWide) next.template load<MODE == kPlain>(a.logits + row * a.K, a.K, g, loose, next_live);
  };
  int64_t t = (int64_t)blockIdx.x * (blockDim.x >> 6) + (threadIdx.x >> 6);
  if constexpr (MODE != kWide) fetch(t);
  // the bias, with zeros where there is none, for all of the workgroup's waves
  const float* bias = lds_all + (blockDim.x >> 6) * o.total;
  bool bias_nan = false;
  float bias_max = 0.f;  // largest finite magnitude
  if constexpr (MODE == kScored) {
    float* b = lds_all + (blockDim.x >> 6) * o.total;
    float* high = b + LPR * E;  // of each wave
    bool nan = false;
    float mine = 0.f;
    for (int k = threadIdx.x; k < LPR * E; k += blockDim.x) {
      const float f = a.bias && k < a.K ? a.bias[k] : 0.f;
      b[k] = f;
      nan |= is_nan_bits(f);
      if (fabsf(f) < INFINITY) mine = fmaxf(mine, fabsf(f));
    }
    mine = team_max<64>(mine);
    const bool none = __ballot(nan) != 0;
    if (lane == 0) high[threadIdx.x >> 6] = none ? -1.f : mine;
    __syncthreads();
    for (int w = 0; w < (int)(blockDim.x >> 6); ++w) bias_nan |= high[w] < 0.f, bias_max = fmaxf(bias_max, high[w]);
  }
  for (; t < tiles; t += waves) {
    const int64_t row0 = t * SL, row = row0 + slot;
    // (what a lane's columns say is formed anew for every tile: kept in registers, it would push out the row)
    asm volatile("" : "+v"(g), "+s"(a.K), "+s"(a.G));
    if constexpr (MODE == kWide) fetch(t);
    const Sl now = next;
    const bool live = next_live;
    if constexpr (MODE == kPlain) fetch(t + waves);
    double top[L];
    float high = -INFINITY, inv = 0.f;
    bool bad = false;
    if constexpr (MODE == kWide) {
      float sum = 0.f;
      for (int64_t off = 0; off < a.K; off += LPR * E) {
        const int left = a.K - off < LPR * E ? (int)(a.K - off) : LPR * E;
        Sl s;
        s.template load<true>(a.logits + row * a.K + off, left, g, loose, live);
        if (!sums) bad |= s.has_nan();
        float x[E];
        s.values(x);
        if (sums) {
          const float m = fmaxf(high, max_of(x));
          const float shift = m == -INFINITY ? 0.f : m;
          float e[E];
#pragma unroll
          for (int i = 0; i < E; ++i) e[i] = quick_exp(x[i], shift);
          sum = fmaf(sum, high == -INFINITY ? 0.f : exp_diff<F32>(high, shift), pair_sum(e));
          high = m;
        }
        add_keys<T, E, LPR, L>(top, x, (int)off + g * V, off == 0);
      }
      if (sums) {
        const float m = team_max<LPR>(high);
        // (a lane of -inf only has nothing, but for the NaN that maxima pass over and that its sum holds)
        sum = team_sum<LPR>(high == -INFINITY && sum == sum ? 0.f : sum * exp_diff<F32>(high, m));
        high = m, inv = 1.f / sum;
        bad = sum != sum;
      } else {
        bad = (__ballot(bad) & team) != 0;
      }
      join_lists<L, LPR>(top);
    } else {
      float x[E];
      now.values(x);
      // x = f(i, bias of element i), but for choices that are out (all is computed and then chosen from: no branches)
      auto add_bias = [&](auto f) {
#pragma unroll
        for (int i = 0; i < E; i += 4) {
          const float4 b = *reinterpret_cast<const float4*>(bias + Sl::first(i / V, g) + i % V);
          const float c[4] = {f(i, b.x), f(i + 1, b.y), f(i + 2, b.z), f(i + 3, b.w)};
#pragma unroll
          for (int v = 0; v < 4; ++v) x[i + v] = x[i + v] == -INFINITY ? -INFINITY : c[v];
        }
      };
      if (!sums) {
        bad = (__ballot(now.has_nan()) & team) != 0;
      } else {
        high = team_max<LPR>(max_of(x));
        const float shift = high == -INFINITY ? 0.f : high;
        float e[E];
#pragma unroll
        for (int i = 0; i < E; ++i) e[i] = quick_exp(x[i], shift);
        const float sum = team_sum<LPR>(pair_sum(e));
        inv = 1.f / sum;
        bad = sum != sum;  // (a NaN, or +inf - inf)
        if constexpr (MODE == kScored) {
          if (arith) {
            add_bias([&](int i, float b) { return fmaf(e[i], inv, b); });
          }
        }
      }
      if constexpr (MODE == kPlain) {
        add_keys<T, E, LPR, L>(top, x, g * V, true);
        join_lists<L, LPR>(top);
      } else {
        int unsure = 0;
        bool copies = false;
        if (arith && !a.softmax) {
          add_bias([&](int i, float b) { return quick_sigmoid(x[i]) + b; });
        }
        bad = live && (bad || bias_nan);
        const float base = score_error(a.softmax, inv);
        if (a.G > 1) {
          // the scores change hands: lanes take a group each, and say which of them stay
          const int gs = a.K / a.G;
          const float per = 1.f / (float)gs;
          auto group_of = [&](int k) { return (int)(((float)k + 0.5f) * per); };  // (exact: k < 2,048)
          float *worth = lds + o.worth, *keep = worth + SL * a.G;
          wave_sync();  // (the tile before is done with it)
          if (g == 0) info[2 * slot] = base;
          if (lane < SL) flag[lane] = 0;
          const bool fours = gs % 4 == 0;
          if (fours) {
            // four neighbours of a group leave their largest two; between groups one place stays empty (banks)
            float2* mine = reinterpret_cast<float2*>(lds) + slot * (a.K / 4 + a.G);
#pragma unroll
            for (int i = 0; i < E; i += 4) {
              const int c = Sl::first(i / V, g) + i % V;
              const float h0 = fmaxf(x[i], x[i + 1]), l0 = fminf(x[i], x[i + 1]);
              const float h1 = fmaxf(x[i + 2], x[i + 3]), l1 = fminf(x[i + 2], x[i + 3]);
              if (c < a.K)
                mine[c / 4 + group_of(c)] = make_float2(fmaxf(h0, h1), fmaxf(fminf(h0, h1), fmaxf(l0, l1)));
            }
          } else {
            float* mine = lds + slot * ((a.K + 3) & ~3);
#pragma unroll
            for (int i = 0; i < E; i += 4) {
              const int c = Sl::first(i / V, g) + i % V;  // (a row's last words may run into its padding)
              if (c < a.K) *reinterpret_cast<float4*>(mine + c) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
            }
          }
          wave_sync();
          for (int it = lane; it < SL * a.G; it += 64) {
            const int r = (int)(((uint32_t)it * group_magic) >> 20), gr = it - r * a.G;
            float m1 = -INFINITY, m2 = -INFINITY;
            if (fours) {
              const float2* p = reinterpret_cast<const float2*>(lds) + r * (a.K / 4 + a.G) + gr * (gs / 4 + 1);
#pragma unroll 4
              for (int i = 0; i < gs / 4; ++i) {
                const float2 c = p[i];
                m2 = fmaxf(fmaxf(m2, c.y), fminf(m1, c.x));
                m1 = fmaxf(m1, c.x);
              }
            } else {
              const float* p = lds + r * ((a.K + 3) & ~3) + gr * gs;
#pragma unroll 4
              for (int i = 0; i < gs; ++i) {
                const float c = p[i];
                m2 = fmaxf(m2, fminf(m1, c));
                m1 = fmaxf(m1, c);
              }
            }
            // (a sum below fp32 is no -inf, which is a group without choices; biases of that size leave all for the end)
            worth[it] = a.best == 2 && m2 > -INFINITY ? fmaxf(m1 + m2, -0x1.fffffep127f) : m1;
          }
          wave_sync();
          for (int it = lane; it < SL * a.G; it += 64) {
            const int r = (int)(((uint32_t)it * group_magic) >> 20), gr = it - r * a.G;
            const float w = worth[it];
            int better = 0;
            float gap = INFINITY;  // the distance to the next group down
#pragma unroll 4
            for (int q = 0; q < a.G; ++q) {
              const float other = worth[r * a.G + q];
              const bool b = other > w || (other == w && q < gr);
              better += b;
              if (!b && q != gr) gap = fminf(gap, w - other);
            }
            // the last group that stays and the first that goes (worths of two groups without choices are not compared);
            // a worth is the sum of two c, none of them larger than 1 and the largest finite bias, whose errors add up
            const float err = kU * (2.f * info[2 * r] + 4.f * (1.f + bias_max)) + 0x1p-119f;
            if (arith && better == a.keep - 1 && w > -INFINITY && gap <= 2.2f * err) flag[r] = kLast;
            keep[it] = better < a.keep ? 1.f : 0.f;
          }
          wave_sync();
#pragma unroll
          for (int i = 0; i < E; i += 4) {
            const int c = Sl::first(i / V, g) + i % V;
            if (fours) {
              const float stays = keep[slot * a.G + group_of(c < a.K ? c : 0)];  // (beyond K all is -inf)
#pragma unroll
              for (int v = 0; v < 4; ++v) x[i + v] = stays != 0.f ? x[i + v] : -INFINITY;
            } else {
#pragma unroll
              for (int v = 0; v < 4; ++v)
                x[i + v] = keep[slot * a.G + group_of(c + v < a.K ? c + v : 0)] != 0.f ? x[i + v] : -INFINITY;
            }
          }
          unsure = flag[slot];
        }
        add_keys<T, E, LPR, L>(top, x, g * V, true);
        join_lists<L, LPR>(top);
        double extra = __hiloint2double((int)0xFF800000u, 0);  // (a score of -inf: none)
        if (arith) {
          // choices that are not selected and no further from the last one than rounding goes
          double last = top[0];
#pragma unroll
          for (int i = 1; i < L; ++i) last = i == S - 1 ? top[i] : last;
          const float vs = key_score(last);
          const float border = vs - 2.2f * (kU * (base + fabsf(vs)) + 0x1p-120f);
          uint32_t count = 0;  // (a comparison and an addition of its bit each; the compiler puts the waits between them)
#pragma unroll
          for (int i = 0; i < E; ++i) count += x[i] >= border;
          count = (uint32_t)team_sum<LPR>((float)count);
          const bool many = vs > -INFINITY && (int)count > S && live && !bad;
          copies = many && (int)count > S + 1;
          if (__ballot(many)) {  // the largest of them joins; others than it and its copies are for the end
            auto score = [&](int k, float& f, float& b) {
              f = T::to_f32(a.logits[row * a.K + k]), b = bias[k];
              const bool out = a.G > 1 && lds[o.worth + (SL + slot) * a.G + k / (a.K / a.G)] == 0.f;  // (stays?)
              return out || f == -INFINITY ? -INFINITY
                     : a.softmax           ? fmaf(quick_exp(f, high), inv, b)
                                           : quick_sigmoid(f) + b;
            };
            double best[1] = {extra};
            float f, b;
            if (many)
              for (int k = g; k < a.K; k += LPR) {
                const double key = key_of(score(k, f, b), k);
                if (key_score(key) >= border && key < last && key > best[0]) best[0] = key;
              }
            join_lists<1, LPR>(best);
            extra = best[0];
            if (copies) {
              const float fe = T::to_f32(a.logits[row * a.K + key_col(extra)]), be = bias[key_col(extra)];
              for (int k = g; k < a.K; k += LPR) {
                const double key = key_of(score(k, f, b), k);
                if (key_score(key) >= border && key < extra && (f != fe || b != be)) unsure = 1;
              }
            }
          }
          unsure = (__ballot(unsure) & team) != 0;
        }
        wave_sync();
        if (g == 0) {
          flag[slot] = !arith || !live || bad               ? 0
                       : unsure                              ? kLast
                       : key_score(extra) > -INFINITY ? (copies ? kOpen | kCopies : kOpen)
                                                             : 0;
          reinterpret_cast<double*>(lds + o.extra)[slot] = extra;
        }
      }
    }
    if (a.softmax && !sums && key_score(top[0]) == INFINITY) bad = true;
    if constexpr (MODE == kScored) fetch(t + waves);  // (no earlier: it would push the row out)
    // ---- the selections change hands: item it is selection it % S of row it / S
    wave_sync();
#pragma unroll
    for (int i = 0; i < L; ++i)
      if (i < S && g == i % LPR) sel[slot * S + i] = bad ? __hiloint2double(0x7FC00000, 0) : top[i];
    if (g == 0) info[2 * slot] = high, info[2 * slot + 1] = inv;
    wave_sync();
    const int items = (int)(a.n - row0 < SL ? a.n - row0 : SL) * S;
    auto row_of = [&](int it) { return (int)(((uint32_t)it * magic) >> 20); };
    for (int it = lane; it < items; it += 64) {
      const int r = row_of(it);
      const double k = sel[it];
      float z = key_score(k);
      if (arith && z > -INFINITY && !is_nan_bits(z)) z = T::to_f32(a.logits[(row0 + r) * a.K + key_col(k)]);
      zs[it] = z;
    }
    wave_sync();
    if constexpr (MODE == kScored) {
      if (arith) {
        for (int it = lane; it < items; it += 64) {
          const int r = row_of(it);
          if (it + 1 >= (r + 1) * S) continue;
          const double k = sel[it], k1 = sel[it + 1];
          const float c = key_score(k), c1 = key_score(k1), z = zs[it], z1 = zs[it + 1];
          if (is_nan_bits(c) || !(c1 > -INFINITY)) continue;
          const float m = info[2 * r], pi = info[2 * r + 1];
          const float err = pair_error(a.softmax, m, pi, z, c) + pair_error(a.softmax, m, pi, z1, c1);
          if (c - c1 <= 1.1f * err && (z != z1 || bias[key_col(k)] != bias[key_col(k1)])) atomicOr(&flag[r], kOpen);
        }
        wave_sync();
        const int state = lane < SL ? flag[lane] : 0;
        uint64_t open = __ballot((state & (kOpen | kLast)) == kOpen), whole = __ballot(state & kLast);
        while (open) {  // lane j takes candidate j, the extra one is the last
          const int r = __builtin_ctzll(open);
          open &= open - 1;
          const double k = lane < S ? sel[r * S + lane] : reinterpret_cast<double*>(lds + o.extra)[r];
          const bool some = lane <= S && key_score(k) > -INFINITY;
          const int ck = some ? (int)key_col(k) : -1;
          float z = -INFINITY, b = 0.f;
          double p = 0.0, c = -INFINITY;
          if (some) {
            z = lane < S ? zs[r * S + lane] : T::to_f32(a.logits[(row0 + r) * a.K + ck]);
            b = bias[ck];
            const double e = exp(a.softmax ? (double)z - (double)info[2 * r] : -(double)z);
            p = a.softmax ? e * (double)info[2 * r + 1] : 1.0 / (1.0 + e);
            c = p + (double)b;
          }
          int rank = 0;
          bool last = false;
          for (int i = 0; i <= S; ++i) {
            const double ci = lane_value(c, i);
            const int ki = __builtin_amdgcn_readlane(ck, i);
            rank += ci > c || (ci == c && (some ? ki < ck : i < lane));
            // (the error of 1 / sum is the same in both: 20 u of the probabilities' difference)
            if (a.softmax && some && ki >= 0) {
              const double pi = lane_value(p, i);
              if (fabs(ci - c) <= 0x1p-19 * fabs(pi - p) + 0x1p-48 * (pi + p))
                last |= lane_value(z, i) != z || lane_value(b, i) != b;
            }
          }
          // (behind the extra one there may be room for its copies)
          last |= lane == S && some && rank < S - 1 && (flag[r] & kCopies);
          if (__ballot(last)) {
            whole |= 1ull << r;
          } else if (lane <= S && rank < S) {
            sel[r * S + rank] = some ? key_of(0.f, ck) : __hiloint2double((int)0xFF800000u, 0);
            zs[r * S + rank] = z;
          }
        }
        while (whole) {
          const int r = __builtin_ctzll(whole);
          whole &= whole - 1;
          const int id = decide_row(a, row0 + r, bias, reinterpret_cast<double*>(lds + o.exact));
          if (lane < S) {
            sel[r * S + lane] = id < 0 ? __hiloint2double((int)0xFF800000u, 0) : key_of(0.f, id);
            zs[r * S + lane] = id < 0 ? -INFINITY : T::to_f32(a.logits[(row0 + r) * a.K + id]);
          }
        }
        wave_sync();
      }
    }
    // a row's selections are neighbouring lanes where S divides 64: their sums need no LDS
    const bool lanes = a.renorm && S <= 16 && (S & (S - 1)) == 0;
    auto over_row = [&](float v, auto op) {
      if (S >= 2) v = op(v, dpp<0xB1>(v));
      if (S >= 4) v = op(v, dpp<0x4E>(v));
      if (S >= 8) v = op(v, dpp<0x141>(v));
      if (S >= 16) v = op(v, dpp<0x140>(v));
      return v;
    };
    if (a.renorm && !lanes) {
      for (int it = lane; it < items; it += 64) {
        const int r = row_of(it);
        float m = -INFINITY;
        for (int j = 0; j < S; ++j) m = fmaxf(m, zs[r * S + j]);
        es[it] = zs[it] == -INFINITY ? 0.f : share_term(zs[it], share_shift(m, a.softmax), a.softmax);
      }
      wave_sync();
    }
    for (int it0 = 0; it0 < items; it0 += 64) {
      const int it = it0 + lane;
      const float z = it < items ? zs[it] : -INFINITY;
      float w;
      if (lanes) {
        const float m = over_row(z, [](float a, float b) { return fmaxf(a, b); });
        const float t = z == -INFINITY ? 0.f : share_term(z, share_shift(m, a.softmax), a.softmax);
        w = a.scale * (t * __builtin_amdgcn_rcpf(over_row(t, [](float a, float b) { return a + b; })));
      }
      if (it >= items) continue;
      const int r = row_of(it);
      if (a.renorm && !lanes) {
        float sum = 0.f;
        for (int j = 0; j < S; ++j) sum += es[r * S + j];
        w = a.scale * (es[it] * __builtin_amdgcn_rcpf(sum));
      } else if (!a.renorm) {
        w = a.scale * (a.softmax ? exp_diff<F32>(z, info[2 * r]) * info[2 * r + 1] : __builtin_amdgcn_rcpf(1.f + exp_to(-z)));
      }
      const int64_t at = row0 * S + it;
      const bool nan = is_nan_bits(z);
      const bool out = nan || !(z > -INFINITY);
      a.ids[at] = out ? -1 : (int32_t)key_col(sel[it]);
      a.weights[at] = nan ? __uint_as_float(0x7FC00000u) : out ? 0.f : w;
      a.chosen[at] = nan ? __uint_as_float(0x7FC00000u) : out ? -INFINITY : z;
    }
  }
}

}  // namespace fkm
