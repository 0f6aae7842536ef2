// Table lookup with scaling, and its gradient by sorted ids.
//
// Forward:   out[i] = round(scale * table[ids[i]]), a row copy.
// Backward:  grad[k] = (old) + scale * sum of the rows i with ids[i] = k.  The ids are argsorted (stable), so
//            entry k owns a contiguous range of the sorted order and its sum is taken in that order: no atomics.
#include "kernels.h"
#include "vecio.h"

namespace fkm {

namespace {

constexpr int kVecs = 4;                  // vectors in flight per thread
constexpr int kTileVecs = 256 * kVecs;    // vectors per workgroup tile

// ---------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------
// A row is nv vectors.  A tile is rpt whole rows (nv <= kTileVecs) or one of
// the nslab slabs of a longer row; workgroups stride over the tiles.
template <class TI, class TO, int V>
__global__ __launch_bounds__(256) void embed_kernel(const typename TI::raw* __restrict__ table,
                                                    const int32_t* __restrict__ ids, int64_t n, uint32_t N, uint32_t K,
                                                    int nv, int rpt, int nslab, int64_t tiles, float scale,
                                                    typename TO::raw* __restrict__ out) {
  for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
    const int64_t row0 = nslab == 1 ? t * rpt : t / nslab;
    const int c0 = nslab == 1 ? 0 : (int)(t - row0 * nslab) * kTileVecs;
    const int width = nslab == 1 ? nv : kTileVecs;
    int64_t src[kVecs], dst[kVecs];
    Pack<TI, V> v[kVecs];
#pragma unroll
    for (int u = 0; u < kVecs; ++u) {
      const int l = threadIdx.x + 256 * u;
      const int r = l / width, c = c0 + l - r * width;
      const int64_t i = row0 + r;
      dst[u] = -1;
      src[u] = -1;
      if (r < rpt && i < n && c < nv) {
        dst[u] = (i * nv + c) * V;
        const uint32_t id = (uint32_t)ids[i];
        const int64_t b = N < n ? (int64_t)((uint32_t)i / N) : 0;
        if (id < K) src[u] = ((b * K + id) * nv + c) * V;
      }
    }
#pragma unroll
    for (int u = 0; u < kVecs; ++u) {
      v[u].zero();
      if (src[u] >= 0) v[u].load(table + src[u]);
    }
#pragma unroll
    for (int u = 0; u < kVecs; ++u) {
      if (dst[u] < 0) continue;
      float f[V];
      v[u].unpack(f);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        f[e] = src[u] >= 0 ? f[e] * scale : 0.f;
        // an fp32 product for every type: without this the compiler joins it
        // with the rounding to fp16 (and only to fp16) in one instruction
        if constexpr (TO::SZ == 2) asm("" : "+v"(f[e]));
      }
      Pack<TO, V> o;
      o.pack(f);
      o.store(out + dst[u]);
    }
  }
}

template <class TI, class TO, int V>
hipError_t embed_v(const void* table, const int32_t* ids, int64_t N, int K, int D, int B, float scale, void* out,
                   hipStream_t s) {
  const int64_t n = N * B;
  const int nv = D / V;
  const int nslab = (nv + kTileVecs - 1) / kTileVecs;
  const int rpt = nslab == 1 ? kTileVecs / nv : 1;
  const int64_t tiles = nslab == 1 ? (n + rpt - 1) / rpt : n * nslab;
  const int64_t grid = tiles < (1 << 22) ? tiles : (1 << 22);
  embed_kernel<TI, TO, V><<<dim3((unsigned)grid), dim3(256), 0, s>>>(
      static_cast<const typename TI::raw*>(table), ids, n, (uint32_t)N, (uint32_t)K, nv, rpt, nslab, tiles, scale,
      static_cast<typename TO::raw*>(out));
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// backward
// ---------------------------------------------------------------------------
// One wave per table entry and slab of 64 vectors.
template <class TI, class TO, int V>
__global__ __launch_bounds__(256) void embed_grad_kernel(const typename TI::raw* __restrict__ dout,
                                                         const uint2* __restrict__ kv, int64_t n, uint32_t K,
                                                         int64_t entries, int nv, int nslab, float scale, bool acc,
                                                         typename TO::raw* __restrict__ grad) {
  const int lane = lane_id();
  const int64_t units = entries * nslab;
  for (int64_t u = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); u < units; u += (int64_t)gridDim.x * 4) {
    const int64_t e = u / nslab;
    const int c = (int)(u - e * nslab) * 64 + lane;
    const uint32_t key = (uint32_t)(e + e / K);  // b * (K + 1) + id
    int64_t lo = 0, hi = n;                      // first sorted position with this key
    while (lo < hi) {
      const int64_t m = (lo + hi) >> 1;
      if (kv[m].x < key) lo = m + 1;
      else hi = m;
    }
    float a[V];
#pragma unroll
    for (int i = 0; i < V; ++i) a[i] = 0.f;
    int64_t j = lo;
    for (; j < n; ++j) {
      const uint2 q = kv[j];
      if (q.x != key) break;
      if (c < nv) {
        Pack<TI, V> p;
        float f[V];
        p.load(dout + ((int64_t)q.y * nv + c) * V);
        p.unpack(f);
#pragma unroll
        for (int i = 0; i < V; ++i) a[i] += f[i];
      }
    }
    if (c >= nv || (acc && j == lo)) continue;
    typename TO::raw* g = grad + (e * nv + c) * V;
    Pack<TO, V> o;
    float old[V];
#pragma unroll
    for (int i = 0; i < V; ++i) old[i] = 0.f;
    if (acc) {
      o.load(g);
      o.unpack(old);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) a[i] = j == lo ? 0.f : acc ? fmaf(scale, a[i], old[i]) : scale * a[i];
    o.pack(a);
    o.store(g);
  }
}

template <class TI, class TO, int V>
hipError_t embed_grad_v(const void* dout, const uint2* sorted, int64_t n, int K, int D, int B, float scale, bool acc,
                        void* grad, hipStream_t s) {
  const int nv = D / V;
  const int nslab = (nv + 63) / 64;
  const int64_t entries = (int64_t)B * K;
  const int64_t blocks = (entries * nslab + 3) / 4;
  const int64_t grid = blocks < (1 << 22) ? blocks : (1 << 22);
  embed_grad_kernel<TI, TO, V><<<dim3((unsigned)grid), dim3(256), 0, s>>>(
      static_cast<const typename TI::raw*>(dout), sorted, n, (uint32_t)K, entries, nv, nslab, scale, acc,
      static_cast<typename TO::raw*>(grad));
  return hipGetLastError();
}

}  // namespace

#define FKM_PAIR(FN, WIDTH, ...)                                                  \
  switch (WIDTH) {                                                                \
    case 8: return FN<TI, TO, 8>(__VA_ARGS__);                                    \
    case 4: return FN<TI, TO, 4>(__VA_ARGS__);                                    \
    default: return FN<TI, TO, 1>(__VA_ARGS__);                                   \
  }

// f(F32{} | F16{} | BF16{}) for a runtime type
template <class F>
static hipError_t with_type(int dt, F&& f) {
  switch (dt) {
    case DT_F32: return f(F32{});
    case DT_F16: return f(F16{});
    case DT_BF16: return f(BF16{});
    default: return hipErrorInvalidValue;
  }
}

hipError_t launch_embed(int tdt, int odt, const void* table, const int32_t* ids, int64_t N, int K, int D, int B,
                        float scale, void* out, hipStream_t s) {
  const int w = vec_width(D, table, dtype_size(tdt), out, dtype_size(odt));
  return with_type(tdt, [&](auto ti) {
    return with_type(odt, [&](auto to) {
      using TI = decltype(ti);
      using TO = decltype(to);
      FKM_PAIR(embed_v, w, table, ids, N, K, D, B, scale, out, s)
    });
  });
}

hipError_t launch_embed_grad(int idt, int gdt, const void* dout, const uint2* sorted, int64_t n, int K, int D, int B,
                             float scale, bool acc, void* grad, hipStream_t s) {
  const int w = vec_width(D, dout, dtype_size(idt), grad, dtype_size(gdt));
  return with_type(idt, [&](auto ti) {
    return with_type(gdt, [&](auto to) {
      using TI = decltype(ti);
      using TO = decltype(to);
      FKM_PAIR(embed_grad_v, w, dout, sorted, n, K, D, B, scale, acc, grad, s)
    });
  });
}

}  // namespace fkm
