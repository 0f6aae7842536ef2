// Gradient of the routing weights with respect to the logits (formulas in flashkm_train.h).
//
// Renormalised weights and sigmoids reach only the selected logits: a thread takes a selection, a row's sums are taken
// over LDS, and what is left is to write the rows (or, accumulating, to add to S elements of each).  Softmax without
// renormalisation reaches every choice: a team of lanes holds a row and its probabilities, and finds the selections'
// derivatives in LDS.
#include "route_rows.h"

namespace fkm {

namespace {

template <class T>
struct GradArgs {
  const typename T::raw* logits;
  int64_t n;
  int K;
  const int32_t* ids;
  const float* chosen;
  const float* dweights;
  int S, softmax, renorm;
  float scale;
  int accumulate;
  typename T::raw* dlogits;
};

// ---------------------------------------------------------------------------
// gradients of the selected logits only
// ---------------------------------------------------------------------------
// A workgroup takes R rows, a thread one selection of them.  Fresh gradients are laid out in LDS as the rows are in
// memory (with the same address modulo 16), zeros with the selections' derivatives among them, and leave in 16-byte
// words whatever K and the address; of rows longer than the tile a workgroup takes `width` columns of one.  Bound by the
// bytes written (8 x 4,095 x 128 bf16, eight a row, 5.7 us, most of it latency; 262,144 x 1,024 bf16 94 us, 5.7 TB/s; 16 KB
// of rows leave LDS for seven workgroups a CU).  Accumulated, a selection's element is read, added to and written by its
// thread: bound by the chain of two reads, ids and then elements, that all
// workgroups are in at once (65,536 x 256 fp32, eight a row, 14.0 us; fresh 15.5; the sectors of 32 bytes that are read and
// written alone are 8.1).
constexpr int kGradTile = 16384;  // bytes of rows in LDS

template <class T, bool ACC>
__global__ __launch_bounds__(256) void route_grad_items_kernel(GradArgs<T> a, int R, int width, int parts,
                                                               int64_t tiles) {
  constexpr int V = 16 / T::SZ;
  __shared__ __align__(16) uint4 tile[ACC ? 1 : kGradTile / 16 + 2];
  __shared__ float zs[256], es[256], gs[256];
  __shared__ uint32_t is[256];
  const int tid = threadIdx.x, S = a.S;
  const int r = tid / S, first = r * S;  // the thread's row, and its first selection's thread
  for (int64_t u = blockIdx.x; u < tiles; u += gridDim.x) {
    const int64_t row0 = parts == 1 ? u * R : u / parts;
    const int c0 = parts == 1 ? 0 : (int)(u - row0 * parts) * width;
    const int rows = (int)(a.n - row0 < R ? a.n - row0 : R);
    const int cols = a.K - c0 < width ? a.K - c0 : width;
    const bool item = tid < rows * S;
    const int64_t at = row0 * S + tid;
    const uint32_t id = item ? (uint32_t)a.ids[at] : ~0u;
    const bool live = id < (uint32_t)a.K;
    const float g = live ? a.scale * a.dweights[at] : 0.f;
    const float z = live ? a.chosen[at] : -INFINITY;
    typename T::raw* mine = a.dlogits + (row0 + r) * a.K + id;  // (live only)
    float old = 0.f;
    if constexpr (ACC) old = live ? T::to_f32(*mine) : 0.f;
    typename T::raw* from = a.dlogits + row0 * a.K + c0;
    const int shift = (int)(((uintptr_t)from & 15) / T::SZ);
    const int count = parts == 1 ? rows * a.K : cols;
    const int words = (shift + count + V - 1) / V;
    if constexpr (!ACC) {
      for (int i = tid; i < words; i += 256) tile[i] = make_uint4(0, 0, 0, 0);
    }
    is[tid] = id;
    float d;
    if (a.renorm) {
      zs[tid] = z;
      __syncthreads();
      float m = -INFINITY;
      if (item)
        for (int j = 0; j < S; ++j) m = fmaxf(m, zs[first + j]);
      const float t = live ? share_term(z, share_shift(m, a.softmax), a.softmax) : 0.f;
      es[tid] = t, gs[tid] = t * g;
      __syncthreads();
      float sum = 0.f, dot = 0.f;
      if (item)
        for (int j = 0; j < S; ++j) sum += es[first + j], dot += gs[first + j];
      d = live ? t / sum * (g - dot / sum) : 0.f;
      if (!a.softmax && live) d *= 1.f / (1.f + exp_to(z));
    } else {
      d = live ? g * (1.f / (1.f + exp_to(-z))) * (1.f / (1.f + exp_to(z))) : 0.f;
    }
    zs[tid] = d;  // (every thread has read its row's logits before the barrier above)
    __syncthreads();
    // the same id again in a row adds up, and its first selection writes
    if (live) {
      float total = 0.f;
      bool lead = true;
      for (int j = 0; j < S; ++j)
        if (is[first + j] == id) {
          total += zs[first + j];
          if (first + j < tid) lead = false;
        }
      if constexpr (ACC) {
        if (lead) *mine = round_to<T>(old + total);
      } else if (lead && id - (uint32_t)c0 < (uint32_t)cols) {
        reinterpret_cast<typename T::raw*>(tile)[shift + (parts == 1 ? r * a.K : 0) + (id - c0)] = round_to<T>(total);
      }
    }
    __syncthreads();
    if constexpr (!ACC) {
      for (int i = tid; i < words; i += 256) {
        typename T::raw* to = from - shift + i * V;
        Pack<T, V> p;
        p.load(reinterpret_cast<const typename T::raw*>(tile + i));
        if (i * V >= shift && (i + 1) * V <= shift + count) p.store_nt(to);
        else p.store_range(to, shift - i * V > 0 ? shift - i * V : 0, shift + count - i * V < V ? shift + count - i * V : V);
      }
      __syncthreads();  // the tile is laid out again
    }
  }
}

// ---------------------------------------------------------------------------
// gradients of whole rows
// ---------------------------------------------------------------------------
// d = p (g - sum p g), g the derivatives of the selections of a choice.  Rows of K <= LPR * E choices stay in a team's
// registers; a wave's rows have their g in its LDS, zero but for the selections, which clear it again.
// Bound by the bytes of a read and a write: 262,144 x 1,024 bf16, two a row, 214 us (5.0 TB/s), onto a gradient 301 (5.3).
template <class T, int E, int LPR>
__global__ __launch_bounds__(256) void route_grad_rows_kernel(GradArgs<T> a, bool loose, uint32_t magic) {
  using Sl = Slice<T, E, LPR>;
  constexpr int V = Sl::V, NV = Sl::NV, SL = 64 / LPR, ROW = LPR * E;
  __shared__ __align__(16) float lds_all[4 * SL * ROW];
  const int lane = lane_id(), slot = lane / LPR, g = lane % LPR, S = a.S;
  float* lds = lds_all + (threadIdx.x >> 6) * SL * ROW;
  for (int i = lane; i < SL * ROW; i += 64) lds[i] = 0.f;
  wave_sync();
  const int64_t tiles = (a.n + SL - 1) / SL, waves = (int64_t)gridDim.x * 4;
  for (int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); t < tiles; t += waves) {
    const int64_t row0 = t * SL, row = row0 + slot;
    const int items = (int)(a.n - row0 < SL ? a.n - row0 : SL) * S;
    Sl s;
    s.template load<true>(a.logits + row * a.K, a.K, g, loose, row < a.n);
    // selections of one id add up in their order: a row's by one lane where an id comes again
    bool again = false;
    for (int it = lane; it < items; it += 64) {
      const int r = (int)(((uint32_t)it * magic) >> 20);
      const uint32_t id = (uint32_t)a.ids[row0 * S + it];
      if (id < (uint32_t)a.K) {
        const float w = a.scale * a.dweights[row0 * S + it];
        again |= atomicExch(&lds[r * ROW + id], w) != 0.f;
      }
    }
    wave_sync();
    if (__ballot(again)) {
      for (int it = lane; it < items; it += 64) {
        const uint32_t id = (uint32_t)a.ids[row0 * S + it];
        if (id < (uint32_t)a.K) lds[(int)(((uint32_t)it * magic) >> 20) * ROW + id] = 0.f;
      }
      wave_sync();
      if (lane < SL && row0 + lane < a.n)
        for (int j = 0; j < S; ++j) {
          const int64_t at = (row0 + lane) * S + j;
          const uint32_t id = (uint32_t)a.ids[at];
          if (id < (uint32_t)a.K) lds[lane * ROW + id] += a.scale * a.dweights[at];
        }
      wave_sync();
    }
    // rows with a selection
    uint64_t some = 0;
    for (int it = lane; it < ((items + 63) & ~63); it += 64) {
      const bool in = it < items && (uint32_t)a.ids[row0 * S + it] < (uint32_t)a.K;
      const int r = (int)(((uint32_t)it * magic) >> 20);
      some |= in ? 1ull << (r & 63) : 0ull;
    }
    some |= (uint64_t)__shfl_xor((long long)some, 1), some |= (uint64_t)__shfl_xor((long long)some, 2);
    some |= (uint64_t)__shfl_xor((long long)some, 4), some |= (uint64_t)__shfl_xor((long long)some, 8);
    some |= (uint64_t)__shfl_xor((long long)some, 16), some |= (uint64_t)__shfl_xor((long long)some, 32);
    const bool any = some >> slot & 1;
    float x[E], w[E];
    s.values(x);
    const float high = team_max<LPR>(max_of(x));
#pragma unroll
    for (int i = 0; i < E; i += 4) {
      const float4 f = *reinterpret_cast<const float4*>(lds + slot * ROW + Sl::first(i / V, g) + i % V);
      w[i] = f.x, w[i + 1] = f.y, w[i + 2] = f.z, w[i + 3] = f.w;
    }
    const float shift = high == -INFINITY ? 0.f : high;
#pragma unroll
    for (int i = 0; i < E; ++i) x[i] = exp_diff<T>(x[i], shift);
    const float inv = 1.f / team_sum<LPR>(pair_sum(x));
    float pw[E];
#pragma unroll
    for (int i = 0; i < E; ++i) x[i] *= inv, pw[i] = x[i] * w[i];
    const float mean = team_sum<LPR>(pair_sum(pw));
    wave_sync();
    for (int it = lane; it < items; it += 64) {
      const uint32_t id = (uint32_t)a.ids[row0 * S + it];
      if (id < (uint32_t)a.K) lds[(int)(((uint32_t)it * magic) >> 20) * ROW + id] = 0.f;
    }
    wave_sync();
    if (row < a.n && (any || !a.accumulate)) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = Sl::first(j, g), left = a.K - c;
        if (left <= 0) continue;
        typename T::raw* to = a.dlogits + row * a.K + c;
        float o[V];
#pragma unroll
        for (int v = 0; v < V; ++v) o[v] = any ? x[j * V + v] * (w[j * V + v] - mean) : 0.f;
        Pack<T, V> p;
        if (a.accumulate) {
          float f[V];
          p.zero();
          if (!loose) p.load(to);
          else if (left >= V) p.load_loose(to);
          else p.load_head(to, left);
          p.unpack(f);
#pragma unroll
          for (int v = 0; v < V; ++v) o[v] += f[v];
        }
        p.pack(o);
        if (!loose) p.store_nt(to);
        else if (left >= V) p.store_loose(to);
        else p.store_range(to, 0, left);
      }
    }
  }
}

// Rows of any length, a workgroup each: a thread's running maximum and sum (fp32 over the elements of a load, in 64 bits
// over its loads), then the row again.  16 bytes a load at element alignment, a row's last few elements one by one.  The
// selections' elements are written last, by their threads.
// 8,192 x 4,096 bf16 41 us, 1,024 x 65,536 73 (three bytes moved for each in a row: 4.9 and 5.5 TB/s).
template <class T>
__global__ __launch_bounds__(256) void route_grad_wide_kernel(GradArgs<T> a) {
  __shared__ float tmp[2][4];
  __shared__ uint32_t is[64];
  __shared__ float gs[64];
  constexpr int V = 16 / T::SZ;
  const int tid = threadIdx.x, S = a.S;
  const uint32_t K = a.K, whole = K / V * V;
  auto join = [&](float v, bool largest, int k) {
    v = largest ? team_max<64>(v) : team_sum<64>(v);
    if ((tid & 63) == 0) tmp[k][tid >> 6] = v;
    __syncthreads();
    const float* p = tmp[k];
    return largest ? fmaxf(fmaxf(p[0], p[1]), fmaxf(p[2], p[3])) : (p[0] + p[1]) + (p[2] + p[3]);
  };
  for (int64_t row = blockIdx.x; row < a.n; row += gridDim.x) {
    __syncthreads();  // the row before is done with the LDS
    if (tid < S) {
      is[tid] = (uint32_t)a.ids[row * S + tid];
      gs[tid] = is[tid] < K ? a.scale * a.dweights[row * S + tid] : 0.f;
    }
    const bool any = __syncthreads_or(tid < S && is[tid] < K);
    const typename T::raw* x = a.logits + row * K;
    typename T::raw* out = a.dlogits + row * K;
    if (!any) {
      if (!a.accumulate) {
        Pack<T, V> none;
        none.zero();
        for (uint32_t k = tid * V; k < whole; k += 256 * V) none.store_loose(out + k);
        if (tid < K - whole) out[whole + tid] = round_to<T>(0.f);
      }
      continue;
    }
    float m = -INFINITY;
    double sum = 0.0;
    auto add = [&](auto& e) {
      const float high = fmaxf(m, max_of(e));
      const float shift = high == -INFINITY ? 0.f : high;
      for (float& f : e) f = exp_diff<F32>(f, shift);
      sum = sum * (double)(m == -INFINITY ? 0.f : exp_diff<F32>(m, shift)) + (double)pair_sum(e);
      m = high;
    };
#pragma unroll 4
    for (uint32_t k = tid * V; k < whole; k += 256 * V) {
      Pack<T, V> p;
      p.load_loose(x + k);
      float e[V];
      p.unpack(e);
      add(e);
    }
    if (tid < K - whole) {
      float e[2] = {T::to_f32(x[whole + tid]), -INFINITY};
      add(e);
    }
    const float high = join(m, true, 0), shift = high == -INFINITY ? 0.f : high;
    const float inv = 1.f / join((float)(sum * (double)(m == -INFINITY ? 0.f : exp_diff<F32>(m, shift))), false, 1);
    // the sum of a choice's derivatives, its probability, and its old value
    float mine = 0.f, p = 0.f, old = 0.f;
    bool lead = false;
    if (tid < S && is[tid] < K) {
      lead = true;
      for (int j = 0; j < S; ++j)
        if (is[j] == is[tid]) {
          mine += gs[j];
          if (j < tid) lead = false;
        }
      p = exp_diff<F32>(T::to_f32(x[is[tid]]), shift) * inv;
      if (a.accumulate) old = T::to_f32(out[is[tid]]);
    }
    __syncthreads();  // (tmp is free, and the old values are read)
    const float mean = join(lead ? p * mine : 0.f, false, 0);
    auto grad = [&](float f, float was) {
      const float d = -mean * (exp_diff<F32>(f, shift) * inv);
      return a.accumulate ? was + d : d;
    };
#pragma unroll 2
    for (uint32_t k = tid * V; k < whole; k += 256 * V) {
      Pack<T, V> p, q;
      p.load_loose(x + k);
      q.zero();
      if (a.accumulate) q.load_loose(out + k);
      float f[V], was[V];
      p.unpack(f), q.unpack(was);
#pragma unroll
      for (int v = 0; v < V; ++v) f[v] = grad(f[v], was[v]);
      p.pack(f);
      p.store_loose(out + k);
    }
    if (tid < K - whole) {
      const uint32_t k = whole + tid;
      out[k] = round_to<T>(grad(T::to_f32(x[k]), a.accumulate ? T::to_f32(out[k]) : 0.f));
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // the row's values have arrived before the selections' are sent
    __syncthreads();
    if (lead) out[is[tid]] = round_to<T>(old + p * (mine - mean));
  }
}

template <class T, int E, int LPR>
hipError_t grad_rows(const GradArgs<T>& a, hipStream_t s) {
  constexpr int SL = 64 / LPR, V = 16 / T::SZ;
  const int64_t blocks = ((a.n + SL - 1) / SL + 3) / 4, most = 256 * 16;
  const bool loose = a.K % V != 0 || (uintptr_t)a.logits % 16 != 0 || (uintptr_t)a.dlogits % 16 != 0;
  route_grad_rows_kernel<T, E, LPR><<<dim3((unsigned)(blocks < most ? blocks : most)), dim3(256), 0, s>>>(
      a, loose, ((1u << 20) + a.S - 1) / a.S);
  return hipGetLastError();
}

int64_t grid_of(int64_t tiles) { return tiles < (1 << 22) ? tiles : (1 << 22); }

template <class T>
hipError_t route_grad_t(const RouteGradCall& c, hipStream_t s) {
  const GradArgs<T> a{static_cast<const typename T::raw*>(c.logits), c.n, c.K, c.ids, c.chosen, c.dweights, c.S, c.softmax,
                      c.renorm, c.scale, c.accumulate, static_cast<typename T::raw*>(c.dlogits)};
  if (a.softmax && !a.renorm) {
    if (a.K <= 8) return grad_rows<T, 8, 1>(a, s);
    if (a.K <= 16) return grad_rows<T, 16, 1>(a, s);
    if (a.K <= 32) return grad_rows<T, 16, 2>(a, s);
    if (a.K <= 64) return grad_rows<T, 16, 4>(a, s);
    if (a.K <= 128) return grad_rows<T, 16, 8>(a, s);
    if (a.K <= 256) return grad_rows<T, 16, 16>(a, s);
    if (a.K <= 512) return grad_rows<T, 16, 32>(a, s);
    if (a.K <= 1024) return grad_rows<T, 16, 64>(a, s);
    if (a.K <= 2048) return grad_rows<T, 32, 64>(a, s);
    route_grad_wide_kernel<T><<<dim3((unsigned)grid_of(a.n)), dim3(256), 0, s>>>(a);
    return hipGetLastError();
  }
  int R = 256 / a.S;
  if (a.accumulate) {
    const int64_t tiles = (a.n + R - 1) / R;
    route_grad_items_kernel<T, true><<<dim3((unsigned)grid_of(tiles)), dim3(256), 0, s>>>(a, R, a.K, 1, tiles);
    return hipGetLastError();
  }
  constexpr int most = kGradTile / T::SZ;  // elements of a tile
  const int fit = a.K <= most ? most / a.K : 1;
  if (R > fit) R = fit;
  const int parts = (int)(((int64_t)a.K + most - 1) / most);
  const int64_t tiles = parts == 1 ? (a.n + R - 1) / R : a.n * parts;
  route_grad_items_kernel<T, false><<<dim3((unsigned)grid_of(tiles)), dim3(256), 0, s>>>(
      a, R, parts == 1 ? a.K : most, parts, tiles);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_route_grad(int dt, const RouteGradCall& c, hipStream_t s) {
  switch (dt) {
    case DT_F32: return route_grad_t<F32>(c, s);
    case DT_F16: return route_grad_t<F16>(c, s);
    case DT_BF16: return route_grad_t<BF16>(c, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace fkm
