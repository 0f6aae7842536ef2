// Balance loss of the use of K choices by N rows, with counts, and its
// gradient (formulas in flashkm_codebook.h).  Both are bound by reading the
// logits (and writing the gradient) once.
//
// Rows up to kBalanceMaxK choices stay in registers.  A team of LPR lanes, or
// of W whole waves, holds one row, E elements a lane, loaded 16 bytes at a time.
// Forward, a lane owns its columns: after the row's maximum and sum it adds its
// probabilities to its own column sums, so the probabilities are never written
// and the logits are read once.  A column sum is fp32 over blocks of kFold rows,
// over at most kFold such blocks and over a wave's lanes, and fp64 over the waves
// of a workgroup (a team of whole waves has none to add).  A workgroup covers a
// chunk of rows of one instance and leaves one partial sum per column, rounded
// to fp32 (half the workspace of fp64, for half a step of a sum that already has
// the roundings above), and its counts, from an LDS histogram of integers; a
// second launch adds the chunks in fp64 in a fixed order.  An instance of one
// chunk is finished by its own workgroup.  Longer rows take two reads: row
// statistics (fp32 over a load, then fp64), then column sums of 64 rows (fp32).
//
// Exponentials are taken of differences from a row's maximum (forward) or
// lse (backward), formed before the scaling by log2(e), so logits of the
// type's lowest value stay finite differences.  The backward pass divides by
// the sum of those exponentials again: an lse of large magnitude does not
// hold the sum's logarithm, but any shift near it gives the same quotients.
#include "kernels.h"
#include "teams.h"
#include "vecio.h"

namespace fkm {

namespace {

constexpr int kFold = kBalanceFold;
// Rows in flight per team, forward and backward (1,048,576 x 1,024 bf16:
// forward 397 us with 1, 396 with 2, 513 with 4; backward 863 us with 2, 806
// with 4).
constexpr int kAheadF = 2, kAheadB = 4;
constexpr int kEarly = 2;  // labels a thread reads ahead of the rows

// v summed over the 64 / LPR lanes of a wave that are LPR apart, in every one of
// them (rotations within 16 lanes, then swaps of 16 and 32).
template <int LPR>
__device__ __forceinline__ float slot_sum(float v) {
  if constexpr (LPR <= 1) v += dpp<0xB1>(v);   // quad_perm 1,0,3,2
  if constexpr (LPR <= 2) v += dpp<0x4E>(v);   // quad_perm 2,3,0,1
  if constexpr (LPR <= 4) v += dpp<0x124>(v);  // row_ror 4
  if constexpr (LPR <= 8) v += dpp<0x128>(v);  // row_ror 8
  if constexpr (LPR <= 16) {
    const auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(p[0]) + __uint_as_float(p[1]);
  }
  if constexpr (LPR <= 32) {
    const auto p = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(p[0]) + __uint_as_float(p[1]);
  }
  return v;
}

// What the forward pass writes for one instance.
struct BalanceOut {
  float* loss;
  int32_t* counts;
  float* prob;
  float* coef;
};
// Entry k of an instance from its column sum, count and valid rows; returns
// its term of the loss.
__device__ __forceinline__ double balance_entry(const BalanceOut& o, int64_t at, int K, int S, double T, double sum,
                                                int count) {
  const double per = T > 0 ? 1.0 / T : 0.0;
  const double p = sum * per;
  const double share = (double)count * ((double)K / S) * per;
  o.counts[at] = count;
  o.prob[at] = (float)p;
  o.coef[at] = (float)(share * per);
  return share * p;
}

// Sum over the workgroup in a fixed order (WAVES waves); every thread gets it.
template <int WAVES>
__device__ __forceinline__ double block_sum_f64(double v, double* tmp) {
  v = wave_sum_f64(v);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) tmp[threadIdx.x >> 6] = v;
  __syncthreads();
  double s = 0.0;
#pragma unroll
  for (int i = 0; i < WAVES; ++i) s += tmp[i];
  return s;
}

// ---------------------------------------------------------------------------
// rows in registers
// ---------------------------------------------------------------------------
// T type, V elements (16 bytes) per load, NV loads per lane, LPR lanes per row
// (W = 1) or W whole waves per row (LPR = 64).  LOOSE: rows that are no multiple
// of 16 bytes or start anywhere: loads at element alignment, the last one of a
// row ending with it, its elements that the load before has too left out
// (65,536 x 5,001 bf16 forward 295 us, 1,048,576 x 100 75 us.  When they took 295
// and 90 us, loads of single elements took 425 and 95 us, and single elements at
// a row's end only, whose branches break the ring, 304 and 162 us).  What it
// costs: 1,048,576 x 189 159 us, x 192 124 us, with as many lanes idle.
template <class T, int NV, int LPR, int W, bool LOOSE>
struct Rows {
  static constexpr int V = 16 / T::SZ;
  static constexpr int E = V * NV;
  static constexpr int MAXK = LPR * W * E;
  static constexpr int BLOCK = W > 4 ? 64 * W : 256;
  static constexpr int WAVES = BLOCK / 64;
  static constexpr int TEAMS = WAVES / W;       // teams of whole waves per workgroup
  static constexpr int SL = 64 / LPR;           // rows per wave and step
  static constexpr int STEP = TEAMS * SL;       // rows per workgroup and step
  static_assert(W == 1 || (LPR == 64 && TEAMS == 1), "a wide team is the workgroup");
  // The columns of lane g of a team: load j takes V from first[j], of which
  // those from skip[j] to before end are the lane's own.
  struct Cols {
    int first[NV], skip[NV], end, K;
    __device__ __forceinline__ Cols(int g, int K_) : K(K_) {
      end = LOOSE && K < V ? K : V;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = (j * LPR * W + g) * V;
        first[j] = c, skip[j] = c < K ? 0 : V;
        if (LOOSE && c + V > K && K >= V) {
          first[j] = K - V;
          skip[j] = c + V - K < V ? c + V - K : V;
        }
      }
    }
    // column of the lane's element e, or -1
    __device__ __forceinline__ int at(int e) const {
      const int v = e % V;
      return v >= skip[e / V] && v < end ? first[e / V] + v : -1;
    }
  };
  Pack<T, V> p[NV];
  // the row's words; -inf for columns that are not the lane's (where a whole
  // load has none) and for a row that is not live
  __device__ __forceinline__ void load(const typename T::raw* row, const Cols& c, bool live) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if constexpr (LOOSE) {
        if (c.end == V) {  // uniform over the launch
          if (live) p[j].load_loose(row + c.first[j]);
          else p[j].fill_neg_inf();
        } else {
          p[j].fill_neg_inf();
          if (live && c.skip[j] == 0) p[j].load_head(row + c.first[j], c.K);
        }
      } else {
        if (live && c.skip[j] == 0) p[j].load_nt(row + c.first[j]);
        else p[j].fill_neg_inf();
      }
    }
  }
  // values as fp32, -inf for columns that are not the lane's
  __device__ __forceinline__ void values(float (&x)[E], const Cols& c) const {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float f[V];
      p[j].unpack(f);
#pragma unroll
      for (int v = 0; v < V; ++v) x[j * V + v] = LOOSE && v < c.skip[j] ? -INFINITY : f[v];
    }
  }
};

// Bound by the logits' bytes where rows are long (1,048,576 x 1,024 bf16: 2.15
// GB in 0.395 ms, 5.4 TB/s) and by the vector instructions, about 9 a value,
// where they are short (8,388,608 x 8, 2 labels: 60 us, 3.9 TB/s).  Waves of 16
// values a lane: five per SIMD instead of four, 396 against 411 us.
template <class T, int NV, int LPR, int W, bool LOOSE>
__global__ __launch_bounds__((Rows<T, NV, LPR, W, LOOSE>::BLOCK),
                             (W == 1 && Rows<T, NV, LPR, W, LOOSE>::E == 16 && !LOOSE ? 5 : 1))
void balance_rows_kernel(
    const typename T::raw* __restrict__ logits, int64_t N, int K, const int32_t* __restrict__ labels, int S,
    const uint8_t* __restrict__ valid, float* __restrict__ lse, int64_t chunks, int steps, float* __restrict__ part,
    int32_t* __restrict__ cpart, int32_t* __restrict__ vpart, BalanceOut out) {
  using R = Rows<T, NV, LPR, W, LOOSE>;
  constexpr int V = R::V, E = R::E, WAVES = R::WAVES;
  __shared__ int hist[R::MAXK];
  __shared__ float col[W == 1 ? WAVES * R::MAXK : 1];
  __shared__ float2 xch[2][W == 1 ? 1 : W];
  __shared__ double tmp[WAVES];
  __shared__ int nval;
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  const int g = W == 1 ? lane % LPR : tid;          // lane of the team
  const typename R::Cols cols(g, K);
  const int slot = W == 1 ? w * R::SL + lane / LPR : 0;
  const int64_t b = blockIdx.x / chunks, c = blockIdx.x - b * chunks;
  const int64_t i0 = c * steps * R::STEP;
  const int64_t i1 = i0 + (int64_t)steps * R::STEP < N ? i0 + (int64_t)steps * R::STEP : N;
  const int64_t base = b * N;

  for (int k = tid; k < K; k += R::BLOCK) hist[k] = 0;
  if (tid == 0) nval = 0;

  float acc[E], sum[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = sum[e] = 0.f;
  int mine = 0;  // valid rows of this team
  auto is_live = [&](int64_t i) { return i < i1 && (!valid || valid[base + i]); };
  // a ring of kAheadF rows: a slot is refilled as soon as its values are out
  R ring[kAheadF];
  bool live_at[kAheadF];
  auto refill = [&](int h, int t) {
    const int64_t i = i0 + (int64_t)t * R::STEP + slot;
    live_at[h] = t < steps && is_live(i);
    ring[h].load(logits + (base + i) * K, cols, live_at[h]);
  };
#pragma unroll
  for (int h = 0; h < kAheadF; ++h) refill(h, h);
  // the first labels are read now and counted after the rows
  const int64_t l0 = (base + i0) * S, l1 = (base + i1) * S;
  auto label_at = [&](int64_t l) -> uint32_t {  // ~0 if it names nothing
    if (l >= l1 || (valid && !valid[(uint32_t)l / (uint32_t)S])) return ~0u;
    return (uint32_t)labels[l];
  };
  uint32_t early[kEarly];
#pragma unroll
  for (int q = 0; q < kEarly; ++q) early[q] = label_at(l0 + tid + q * R::BLOCK);
  __syncthreads();  // the histogram is clear
  int fold = 0;
  auto step = [&](int t, int h) {
    const int64_t i = i0 + (int64_t)t * R::STEP + slot;
    const bool live = live_at[h];
    float x[E];
    ring[h].values(x, cols);
    refill(h, t + kAheadF);
    float m = team_max<LPR>(max_of(x));
    // a wave (or team) without a finite maximum: shift by 0, so that -inf
    // gives 0 (and NaN and +inf stay what they are)
    float shift = m == -INFINITY ? 0.f : m;
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      x[e] = exp_diff<T>(x[e], shift);
      s += x[e];
    }
    s = team_sum<LPR>(s);
    float scale = 1.f;  // from this wave's exponentials to the row's
    if constexpr (W > 1) {
      if (lane == 0) xch[t & 1][w] = make_float2(m, s);
      __syncthreads();
      float mm = -INFINITY;
#pragma unroll
      for (int q = 0; q < W; ++q) mm = fmaxf(mm, xch[t & 1][q].x);
      const float sh = mm == -INFINITY ? 0.f : mm;
      float ss = 0.f;
#pragma unroll
      for (int q = 0; q < W; ++q) {
        const float2 o = xch[t & 1][q];
        // a wave's sum is relative to its own shift (0 if it had none)
        ss += o.y * exp_diff<T>(o.x == -INFINITY ? (o.y == 0.f ? sh : 0.f) : o.x, sh);
      }
      scale = exp_diff<T>(m == -INFINITY ? sh : m, sh);
      m = mm, s = ss;
    }
    if (g == 0 && i < i1) {
      lse[base + i] = !live ? INFINITY : s == 0.f ? -INFINITY : fmaf(__builtin_amdgcn_logf(s), kLn2, m);
      mine += live;
    }
    // a row that leaves no probability has exponentials of 0 only
    const float q = s != 0.f ? scale * __builtin_amdgcn_rcpf(s) : 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = fmaf(x[e], q, acc[e]);
    if (++fold == kFold) {
      fold = 0;
#pragma unroll
      for (int e = 0; e < E; ++e) sum[e] += acc[e], acc[e] = 0.f;
    }
  };
  for (int t = 0; t < steps; t += kAheadF) {
#pragma unroll
    for (int h = 0; h < kAheadF; ++h)
      if (t + h < steps && i0 + (int64_t)(t + h) * R::STEP < i1) step(t + h, h);  // uniform over the workgroup
  }
#pragma unroll
  for (int e = 0; e < E; ++e) sum[e] += acc[e];

  // counts of the chunk's labels: integer LDS atomics, exact in any order
#pragma unroll
  for (int q = 0; q < kEarly; ++q)
    if (early[q] < (uint32_t)K) atomicAdd(&hist[early[q]], 1);
  for (int64_t l = l0 + tid + kEarly * R::BLOCK; l < l1; l += R::BLOCK) {
    const uint32_t k = label_at(l);
    if (k < (uint32_t)K) atomicAdd(&hist[k], 1);
  }
  if (mine) atomicAdd(&nval, mine);

  // column sums: lanes of one column, then (below) the waves, in fixed orders
  if constexpr (W == 1) {
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const float total = slot_sum<LPR>(sum[e]);
      const int k = cols.at(e);
      if (lane < LPR && k >= 0) col[w * R::MAXK + k] = total;
    }
  }
  __syncthreads();
  auto column = [&](int k) {
    double s = 0.0;
#pragma unroll
    for (int q = 0; q < WAVES; ++q) s += (double)col[q * R::MAXK + k];
    return s;
  };
  const double T_ = nval;
  const int64_t at = (b * chunks + c) * K;
  double term = 0.0;
  if constexpr (W == 1) {
    for (int k = tid; k < K; k += R::BLOCK) {
      if (chunks == 1) {
        term += balance_entry(out, b * K + k, K, S, T_, column(k), hist[k]);
      } else {
        part[at + k] = (float)column(k);
        cpart[at + k] = hist[k];
      }
    }
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int k = cols.at(e);
      if (k < 0) continue;
      if (chunks == 1) {
        term += balance_entry(out, b * K + k, K, S, T_, (double)sum[e], hist[k]);
      } else {
        part[at + k] = sum[e];
        cpart[at + k] = hist[k];
      }
    }
  }
  if (chunks == 1) {
    term = block_sum_f64<WAVES>(term, tmp);
    if (tid == 0) out.loss[b] = (float)term;
  } else if (tid == 0) {
    vpart[b * chunks + c] = nval;
  }
}

// Chunk sums joined: 1,024 threads take CB columns of one instance, 1024 / CB
// groups of chunks in order, joined by halving.  With one column block the
// loss is finished here, else each block leaves its term.
template <int CB>
__global__ __launch_bounds__(1024) void balance_join_kernel(const float* __restrict__ part, int64_t chunks,
                                                            const int32_t* cpart, int64_t cchunks,
                                                            const int32_t* __restrict__ vpart, int64_t vchunks,
                                                            uint32_t K, int S, int kblocks, int64_t units,
                                                            BalanceOut out, double* __restrict__ terms) {
  constexpr int G = 1024 / CB;
  __shared__ double sp[1024];
  __shared__ int sc[1024];
  __shared__ double tmp[16];
  const int tid = threadIdx.x;
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int64_t b = u / kblocks;
    const int kb = (int)(u - b * kblocks);
    const uint32_t k = (uint32_t)kb * CB + tid % CB;
    const int g = tid / CB;
    int64_t nv = 0;
    for (int64_t c = tid; c < vchunks; c += 1024) nv += vpart[b * vchunks + c];
    double p = 0.0;
    int n = 0;
    if (k < K) {
#pragma unroll 8
      for (int64_t c = g; c < chunks; c += G) p += (double)part[(b * chunks + c) * K + k];
#pragma unroll 8
      for (int64_t c = g; c < cchunks; c += G) n += cpart[(b * cchunks + c) * K + k];
    }
    const double T_ = block_sum_f64<16>((double)nv, tmp);
    sp[tid] = p;
    sc[tid] = n;
    for (int h = 512; h >= CB; h >>= 1) {
      __syncthreads();
      if (tid < h) sp[tid] += sp[tid + h], sc[tid] += sc[tid + h];
    }
    double term = 0.0;
    if (tid < CB && k < K) term = balance_entry(out, b * K + k, (int)K, S, T_, sp[tid], sc[tid]);
    term = block_sum_f64<16>(term, tmp);  // its barriers also end this unit's use of sp and sc
    if (tid == 0) {
      if (kblocks == 1) out.loss[b] = (float)term;
      else terms[u] = term;
    }
  }
}

// loss[b] = the column blocks' terms in a fixed order; one wave per instance.
__global__ __launch_bounds__(256) void balance_loss_kernel(const double* __restrict__ terms, int kblocks, int B,
                                                           float* __restrict__ loss) {
  const int lane = lane_id();
  for (int64_t b = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); b < B; b += (int64_t)gridDim.x * 4) {
    double s = 0.0;
    for (int k = lane; k < kblocks; k += 64) s += terms[b * kblocks + k];
    s = wave_sum_f64(s);
    if (lane == 0) loss[b] = (float)s;
  }
}

// Bound by the bytes read and written: 1,048,576 x 1,024 bf16 4.3 GB in 0.81 ms,
// 5.3 TB/s.
template <class T, int NV, int LPR, int W, bool LOOSE>
__global__ __launch_bounds__((Rows<T, NV, LPR, W, LOOSE>::BLOCK)) void balance_grad_rows_kernel(
    const typename T::raw* __restrict__ logits, int64_t N, int K, const float* __restrict__ lse,
    const float* __restrict__ coef, const float* __restrict__ dloss, int64_t chunks, int steps,
    typename T::raw* __restrict__ dlogits) {
  using R = Rows<T, NV, LPR, W, LOOSE>;
  constexpr int V = R::V, E = R::E;
  __shared__ float2 xch[2][W == 1 ? 1 : W];
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  const int g = W == 1 ? lane % LPR : tid;
  const typename R::Cols cols(g, K);
  const int slot = W == 1 ? w * R::SL + lane / LPR : 0;
  const int64_t b = blockIdx.x / chunks, c = blockIdx.x - b * chunks;
  const int64_t i0 = c * steps * R::STEP;
  const int64_t i1 = i0 + (int64_t)steps * R::STEP < N ? i0 + (int64_t)steps * R::STEP : N;
  const int64_t base = b * N;
  const float dl = dloss[b];
  float cf[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int k = cols.at(e);
    cf[e] = k >= 0 ? coef[b * K + k] : 0.f;
  }
  auto z_of = [&](int64_t i) { return i < i1 ? lse[base + i] : INFINITY; };
  auto is_live = [](float z) { return z != INFINITY && z != -INFINITY; };
  R ring[kAheadB];
  float z_at[kAheadB];
  auto refill = [&](int h, int t) {
    const int64_t i = i0 + (int64_t)t * R::STEP + slot;
    z_at[h] = t < steps ? z_of(i) : INFINITY;
    ring[h].load(logits + (base + i) * K, cols, is_live(z_at[h]));
  };
#pragma unroll
  for (int h = 0; h < kAheadB; ++h) refill(h, h);
  auto step = [&](int t, int h) {
    const int64_t i = i0 + (int64_t)t * R::STEP + slot;
    const float z = z_at[h];
    float x[E];
    ring[h].values(x, cols);
    refill(h, t + kAheadB);
    float s = 0.f, d = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      x[e] = exp_diff<T>(x[e], z);
      s += x[e];
      d = fmaf(x[e], cf[e], d);
    }
    s = team_sum<LPR>(s);
    d = team_sum<LPR>(d);
    if constexpr (W > 1) {
      if (lane == 0) xch[t & 1][w] = make_float2(s, d);
      __syncthreads();
      s = 0.f, d = 0.f;
#pragma unroll
      for (int q = 0; q < W; ++q) s += xch[t & 1][q].x, d += xch[t & 1][q].y;
    }
    const float inv = __builtin_amdgcn_rcpf(s);
    const float mean = d * inv, scale = dl * inv;
    const bool live = is_live(z);
    if (i < i1) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        if (cols.skip[j] == V) continue;
        float o[V];
#pragma unroll
        for (int v = 0; v < V; ++v) o[v] = live ? scale * x[j * V + v] * (cf[j * V + v] - mean) : 0.f;
        Pack<T, V> q;
        q.pack(o);
        typename T::raw* at = dlogits + (base + i) * K + cols.first[j];
        if constexpr (LOOSE) {
          if (cols.skip[j] == 0 && cols.end == V) q.store_loose(at);
          else q.store_range(at, cols.skip[j], cols.end);
        } else {
          q.store_nt(at);
        }
      }
    }
  };
  for (int t = 0; t < steps; t += kAheadB) {
#pragma unroll
    for (int h = 0; h < kAheadB; ++h)
      if (t + h < steps && i0 + (int64_t)(t + h) * R::STEP < i1) step(t + h, h);  // uniform over the workgroup
  }
}

// ---------------------------------------------------------------------------
// rows longer than the registers hold
// ---------------------------------------------------------------------------
// Columns are unsigned: K may be 2^31 - 1, and a step past it must not wrap.
// One workgroup per row, V elements per load; f(values, first column) over the
// row's elements that thread tid takes, in order.
template <class T, int V, class F>
__device__ __forceinline__ void over_row(const typename T::raw* __restrict__ row, uint32_t K, F&& f) {
#pragma unroll 4
  for (uint32_t k = threadIdx.x * V; k < K; k += 256 * V) {
    Pack<T, V> p;
    float x[V];
    p.load(row + k);
    p.unpack(x);
    f(x, k);
  }
}
// (a, b) summed over the workgroup's 4 waves, in every thread.
__device__ __forceinline__ float2 block_sum2(float a, float b, float2* tmp) {
  a = team_sum<64>(a);
  b = team_sum<64>(b);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) tmp[threadIdx.x >> 6] = make_float2(a, b);
  __syncthreads();
  return make_float2((tmp[0].x + tmp[1].x) + (tmp[2].x + tmp[3].x), (tmp[0].y + tmp[1].y) + (tmp[2].y + tmp[3].y));
}

// lse of every row (+inf for an invalid one) and its (maximum, 1 / sum of
// exponentials), (0, 0) for a row that leaves no probability: the
// probabilities come from these, since a large lse has lost the sum's low
// bits.  One read: a thread keeps a running maximum and the sum relative to it,
// fp32 over a load's elements and fp64 over its loads (in fp32 alone a row of
// 2^24 equal values rounds the same way 65,536 times: lse off by 1.6e-4).
// Loads of single elements go in groups of G, to share one step in fp64.
template <class T, int V>
__global__ __launch_bounds__(256) void balance_lse_kernel(const typename T::raw* __restrict__ logits, int64_t n, int K,
                                                          const uint8_t* __restrict__ valid, float* __restrict__ lse,
                                                          float2* __restrict__ ms) {
  constexpr int G = V == 1 ? 4 : 1;
  __shared__ float2 tmp[4];
  const uint32_t tid = threadIdx.x, Ku = K;
  for (int64_t i = blockIdx.x; i < n; i += gridDim.x) {
    if (valid && !valid[i]) {  // uniform over the workgroup
      if (threadIdx.x == 0) lse[i] = INFINITY, ms[i] = make_float2(0.f, 0.f);
      continue;
    }
    float m = -INFINITY;
    double s = 0.0;
    const typename T::raw* row = logits + i * K;
#pragma unroll G == 1 ? 4 : 2
    for (uint32_t k = tid * V; k < Ku; k += 256 * V * G) {
      float x[V * G];
#pragma unroll
      for (int g = 0; g < G; ++g) {
        const uint32_t at = k + 256 * V * g;
        Pack<T, V> p;
        p.load(row + (G == 1 || at < Ku ? at : k));  // (no branch: the loads of a group are in flight together)
        p.unpack(x + g * V);
        if (G > 1 && at >= Ku) x[g] = -INFINITY;
      }
      float top = x[0];
#pragma unroll
      for (int v = 1; v < V * G; ++v) top = fmaxf(top, x[v]);
      if (top > m) {  // the sum moves to the new maximum (from nothing, if that was -inf)
        s *= (double)exp_diff<T>(m, top);
        m = top;
      }
      const float shift = m == -INFINITY ? 0.f : m;
      float e = 0.f;
#pragma unroll
      for (int v = 0; v < V * G; ++v) e += exp_diff<T>(x[v], shift);
      s += (double)e;
    }
    // the workgroup's maximum, then the sums relative to it
    const float wm = team_max<64>(m);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) tmp[threadIdx.x >> 6].x = wm;
    __syncthreads();
    const float top = fmaxf(fmaxf(tmp[0].x, tmp[1].x), fmaxf(tmp[2].x, tmp[3].x));
    const float shift = top == -INFINITY ? 0.f : top;
    // a thread without a maximum holds 0 (or NaN), relative to 0
    const float sum = block_sum2(m == -INFINITY ? (float)s : (float)s * exp_diff<T>(m, shift), 0.f, tmp).x;
    if (threadIdx.x == 0) {
      lse[i] = sum == 0.f ? -INFINITY : top + logf(sum);
      ms[i] = sum == 0.f ? make_float2(0.f, 0.f) : make_float2(shift, 1.f / sum);
    }
  }
}

// part[b, chunk, k] = sum of p[b, i, k] over the chunk's valid rows; V columns
// per thread.
template <class T, int V>
__global__ __launch_bounds__(256) void balance_cols_kernel(const typename T::raw* __restrict__ logits, int64_t N,
                                                           uint32_t K, int64_t chunks, uint32_t kblocks, int64_t units,
                                                           const float2* __restrict__ ms, float* __restrict__ part) {
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int64_t bc = u / kblocks;
    const uint32_t k = ((uint32_t)(u - bc * kblocks) * 256 + threadIdx.x) * V;
    if (k >= K) continue;
    const int64_t b = bc / chunks, c = bc - b * chunks;
    const int64_t i0 = c * kBalanceRows, i1 = i0 + kBalanceRows < N ? i0 + kBalanceRows : N;
    float sum[V];
#pragma unroll
    for (int v = 0; v < V; ++v) sum[v] = 0.f;
#pragma unroll 4
    for (int64_t i = i0; i < i1; ++i) {
      const float2 z = ms[b * N + i];
      Pack<T, V> p;
      float x[V];
      p.load_nt(logits + (b * N + i) * K + k);
      p.unpack(x);
      // (a row that leaves nothing may hold anything)
#pragma unroll
      for (int v = 0; v < V; ++v) sum[v] += z.y == 0.f ? 0.f : exp_diff<T>(x[v], z.x) * z.y;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) part[bc * K + k + v] = sum[v];
  }
}

__global__ __launch_bounds__(256) void balance_zero_kernel(int32_t* __restrict__ counts, int64_t entries,
                                                           int32_t* __restrict__ nvalid, int B) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < entries; i += (int64_t)gridDim.x * 256) {
    counts[i] = 0;
    if (i < B) nvalid[i] = 0;
  }
}

// Integer counts by atomics: exact, whatever their order.
__global__ __launch_bounds__(256) void balance_count_kernel(const int32_t* __restrict__ labels, int64_t n, uint32_t N,
                                                            uint32_t K, int S, const uint8_t* __restrict__ valid,
                                                            int32_t* __restrict__ counts,
                                                            int32_t* __restrict__ nvalid) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
    if (valid && !valid[i]) continue;
    const int64_t b = (uint32_t)i / N;
    atomicAdd(&nvalid[b], 1);
    for (int s = 0; s < S; ++s) {
      const uint32_t l = (uint32_t)labels[i * S + s];
      if (l < K) atomicAdd(&counts[b * K + l], 1);
    }
  }
}

template <class T, int V>
__global__ __launch_bounds__(256) void balance_grad_wide_kernel(const typename T::raw* __restrict__ logits, int64_t n,
                                                                uint32_t N, int K, const float* __restrict__ lse,
                                                                const float* __restrict__ coef,
                                                                const float* __restrict__ dloss,
                                                                typename T::raw* __restrict__ dlogits) {
  __shared__ float2 tmp[4];
  for (int64_t i = blockIdx.x; i < n; i += gridDim.x) {
    const int64_t b = (uint32_t)i / N;
    const float z = lse[i];
    const bool none = z == INFINITY || z == -INFINITY;  // uniform over the workgroup
    const float* cf = coef + b * K;
    float mean = 0.f, scale = 0.f;
    if (!none) {
      double s = 0.0, d = 0.0;  // as in the forward pass
      over_row<T, V>(logits + i * K, K, [&](const float (&x)[V], uint32_t k) {
        float es = 0.f, ds = 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const float e = exp_diff<T>(x[v], z);
          es += e;
          ds = fmaf(e, cf[k + v], ds);
        }
        s += (double)es, d += (double)ds;
      });
      const float2 t = block_sum2((float)s, (float)d, tmp);
      const float inv = 1.f / t.x;
      mean = t.y * inv, scale = dloss[b] * inv;
    }
    // the row again for the gradient (from the cache only while the rows of all
    // resident workgroups fit it: 8,192 x 65,536 bf16 1,181 us)
    over_row<T, V>(logits + i * K, K, [&](const float (&x)[V], uint32_t k) {
      float o[V];
#pragma unroll
      for (int v = 0; v < V; ++v) o[v] = none ? 0.f : scale * exp_diff<T>(x[v], z) * (cf[k + v] - mean);
      Pack<T, V> q;
      q.pack(o);
      q.store_nt(dlogits + i * K + k);
    });
  }
}

int64_t capped(int64_t blocks) { return blocks < 1 ? 1 : blocks < (1 << 22) ? blocks : (1 << 22); }

// Chunk sums in `part`, counts in `cpart` (cchunks of them), valid rows in
// vpart, to the outputs.
struct JoinIn {
  const float* part;
  int64_t chunks;
  const int32_t* cpart;
  int64_t cchunks;
  const int32_t* vpart;
  int64_t vchunks;
};
template <int CB>
void join_launch(const JoinIn& in, int K, int S, int B, const BalanceOut& out, double* terms, hipStream_t s) {
  const int kblocks = (int)(((uint32_t)K + CB - 1) / CB);
  const int64_t units = (int64_t)B * kblocks;
  const int64_t grid = units < (1 << 20) ? units : (1 << 20);
  balance_join_kernel<CB><<<dim3((unsigned)grid), dim3(1024), 0, s>>>(in.part, in.chunks, in.cpart, in.cchunks,
                                                                      in.vpart, in.vchunks, K, S, kblocks, units, out,
                                                                      terms);
  if (kblocks > 1)
    balance_loss_kernel<<<dim3((unsigned)capped((B + 3) / 4)), dim3(256), 0, s>>>(terms, kblocks, B, out.loss);
}
hipError_t join(const JoinIn& in, int K, int S, int B, const BalanceOut& out, double* terms, hipStream_t s) {
  // one workgroup per instance while it reads little, else 32 columns each and
  // a launch for the loss (8 x 4,095 x 128: 10.9 us in all, 13.4 by 32 columns;
  // 16,384 x 1,024: 109 us with one workgroup, 25.1 by 32 columns)
  const bool one = K <= 1024 && in.chunks * K <= 65536;
  if (K <= 32 || !one) join_launch<kBalanceJoinCols>(in, K, S, B, out, terms, s);
  else if (K <= 64) join_launch<64>(in, K, S, B, out, terms, s);
  else if (K <= 128) join_launch<128>(in, K, S, B, out, terms, s);
  else if (K <= 256) join_launch<256>(in, K, S, B, out, terms, s);
  else if (K <= 512) join_launch<512>(in, K, S, B, out, terms, s);
  else join_launch<1024>(in, K, S, B, out, terms, s);
  return hipGetLastError();
}

template <class T, int NV, int LPR, int W, bool LOOSE>
hipError_t rows_forward(const void* logits, int64_t N, int K, int B, const int32_t* labels, int S,
                        const uint8_t* valid, float* lse, const BalanceOut& out, const BalanceBuffers& buf,
                        hipStream_t s) {
  using R = Rows<T, NV, LPR, W, LOOSE>;
  static_assert(R::STEP == balance_step(R::MAXK), "the workspace's chunks are these");
  const BalanceSplit sp = balance_split(N, B, K);
  balance_rows_kernel<T, NV, LPR, W, LOOSE><<<dim3((unsigned)(B * sp.chunks)), dim3(R::BLOCK), 0, s>>>(
      static_cast<const typename T::raw*>(logits), N, K, labels, S, valid, lse, sp.chunks, sp.steps, buf.part,
      buf.cpart, buf.vpart, out);
  if (sp.chunks == 1) return hipGetLastError();
  return join(JoinIn{buf.part, sp.chunks, buf.cpart, sp.chunks, buf.vpart, sp.chunks}, K, S, B, out, buf.terms, s);
}

template <class T, int NV, int LPR, int W, bool LOOSE>
hipError_t rows_backward(const void* logits, int64_t N, int K, int B, const float* lse, const float* coef,
                         const float* dloss, void* dlogits, hipStream_t s) {
  using R = Rows<T, NV, LPR, W, LOOSE>;
  static_assert(R::STEP == balance_step(R::MAXK), "the workspace's chunks are these");
  const BalanceSplit sp = balance_split(N, B, K);
  balance_grad_rows_kernel<T, NV, LPR, W, LOOSE><<<dim3((unsigned)(B * sp.chunks)), dim3(R::BLOCK), 0, s>>>(
      static_cast<const typename T::raw*>(logits), N, K, lse, coef, dloss, sp.chunks, sp.steps,
      static_cast<typename T::raw*>(dlogits));
  return hipGetLastError();
}

// f(Team) with the smallest team that holds a row of K elements; A loads of 16
// bytes make 8 elements, and a lane holds 8, or 16 where a team takes 2 A loads.
template <int NV_, int LPR_, int W_, bool LOOSE_>
struct Team {
  static constexpr int NV = NV_, LPR = LPR_, W = W_;
  static constexpr bool LOOSE = LOOSE_;
};
template <int A, bool LOOSE, class F>
hipError_t with_team(int K, F&& f) {
  if (K <= 8) return f(Team<A, 1, 1, LOOSE>{});
  if (K <= 16) return f(Team<A, 2, 1, LOOSE>{});
  if (K <= 32) return f(Team<A, 4, 1, LOOSE>{});
  if (K <= 64) return f(Team<A, 8, 1, LOOSE>{});
  if (K <= 128) return f(Team<A, 16, 1, LOOSE>{});
  if (K <= 256) return f(Team<A, 32, 1, LOOSE>{});
  if (K <= 512) return f(Team<A, 64, 1, LOOSE>{});
  if (K <= 1024) return f(Team<2 * A, 64, 1, LOOSE>{});
  // (a barrier a row: the fewer waves share one, the more rows a CU works on)
  if (K <= 2048) return f(Team<A, 64, 4, LOOSE>{});
  if (K <= 4096) return f(Team<2 * A, 64, 4, LOOSE>{});
  if (K <= 8192) return f(Team<2 * A, 64, 8, LOOSE>{});
  return f(Team<2 * A, 64, 16, LOOSE>{});
}

template <class T, int V>
hipError_t wide_forward(const void* logits, int64_t N, int K, int B, const int32_t* labels, int S,
                        const uint8_t* valid, float* lse, const BalanceOut& out, const BalanceBuffers& buf,
                        hipStream_t s) {
  const int64_t n = N * B;
  const auto* x = static_cast<const typename T::raw*>(logits);
  const int64_t entries = (int64_t)B * K;
  balance_zero_kernel<<<dim3((unsigned)capped((entries + 255) / 256)), dim3(256), 0, s>>>(out.counts, entries,
                                                                                           buf.vpart, B);
  if (n) {
    balance_lse_kernel<T, V><<<dim3((unsigned)capped(n)), dim3(256), 0, s>>>(x, n, K, valid, lse, buf.ms);
    balance_count_kernel<<<dim3((unsigned)capped((n + 255) / 256)), dim3(256), 0, s>>>(
        labels, n, (uint32_t)N, (uint32_t)K, S, valid, out.counts, buf.vpart);
  }
  const int64_t chunks = balance_wide_chunks(N);
  const uint32_t kblocks = ((uint32_t)K + 256 * V - 1) / (256 * V);
  const int64_t units = B * chunks * kblocks;
  balance_cols_kernel<T, V><<<dim3((unsigned)capped(units)), dim3(256), 0, s>>>(x, N, K, chunks, kblocks, units,
                                                                                 buf.ms, buf.part);
  return join(JoinIn{buf.part, chunks, out.counts, 1, buf.vpart, 1}, K, S, B, out, buf.terms, s);
}

template <class T>
hipError_t balance_t(const void* logits, int64_t N, int K, int B, const int32_t* labels, int S, const uint8_t* valid,
                     float* lse, const BalanceOut& out, const BalanceBuffers& buf, hipStream_t s) {
  constexpr int VEC = 16 / T::SZ;
  if (K <= kBalanceMaxK) {
    auto go = [&](auto team) {
      using P = decltype(team);
      return rows_forward<T, P::NV, P::LPR, P::W, P::LOOSE>(logits, N, K, B, labels, S, valid, lse, out, buf, s);
    };
    return vec_width(K, VEC, logits, T::SZ, logits, T::SZ) == VEC ? with_team<8 / VEC, false>(K, go)
                                                                  : with_team<8 / VEC, true>(K, go);
  }
  return vec_width(K, VEC, logits, T::SZ, logits, T::SZ) == VEC
             ? wide_forward<T, VEC>(logits, N, K, B, labels, S, valid, lse, out, buf, s)
             : wide_forward<T, 1>(logits, N, K, B, labels, S, valid, lse, out, buf, s);
}

template <class T>
hipError_t balance_grad_t(const void* logits, int64_t N, int K, int B, const float* lse, const float* coef,
                          const float* dloss, void* dlogits, hipStream_t s) {
  constexpr int VEC = 16 / T::SZ;
  if (K <= kBalanceMaxK) {
    auto go = [&](auto team) {
      using P = decltype(team);
      return rows_backward<T, P::NV, P::LPR, P::W, P::LOOSE>(logits, N, K, B, lse, coef, dloss, dlogits, s);
    };
    return vec_width(K, VEC, logits, T::SZ, dlogits, T::SZ) == VEC ? with_team<8 / VEC, false>(K, go)
                                                                   : with_team<8 / VEC, true>(K, go);
  }
  const int64_t n = N * B;
  const dim3 grid((unsigned)capped(n));
  const auto* x = static_cast<const typename T::raw*>(logits);
  auto* dx = static_cast<typename T::raw*>(dlogits);
  if (vec_width(K, VEC, logits, T::SZ, dlogits, T::SZ) == VEC)
    balance_grad_wide_kernel<T, VEC><<<grid, dim3(256), 0, s>>>(x, n, (uint32_t)N, K, lse, coef, dloss, dx);
  else
    balance_grad_wide_kernel<T, 1><<<grid, dim3(256), 0, s>>>(x, n, (uint32_t)N, K, lse, coef, dloss, dx);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_balance(int dt, const void* logits, int64_t N, int K, int B, const int32_t* labels, int S,
                          const uint8_t* valid, float* loss, int32_t* counts, float* prob, float* lse, float* coef,
                          const BalanceBuffers& buf, hipStream_t s) {
  const BalanceOut out{loss, counts, prob, coef};
  switch (dt) {
    case DT_F32: return balance_t<F32>(logits, N, K, B, labels, S, valid, lse, out, buf, s);
    case DT_F16: return balance_t<F16>(logits, N, K, B, labels, S, valid, lse, out, buf, s);
    case DT_BF16: return balance_t<BF16>(logits, N, K, B, labels, S, valid, lse, out, buf, s);
    default: return hipErrorInvalidValue;
  }
}

hipError_t launch_balance_grad(int dt, const void* logits, int64_t N, int K, int B, const float* lse,
                               const float* coef, const float* dloss, void* dlogits, hipStream_t s) {
  switch (dt) {
    case DT_F32: return balance_grad_t<F32>(logits, N, K, B, lse, coef, dloss, dlogits, s);
    case DT_F16: return balance_grad_t<F16>(logits, N, K, B, lse, coef, dloss, dlogits, s);
    case DT_BF16: return balance_grad_t<BF16>(logits, N, K, B, lse, coef, dloss, dlogits, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace fkm
