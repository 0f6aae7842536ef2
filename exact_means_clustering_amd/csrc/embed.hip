// Table lookup with scaling, and its gradient by sorted ids.
//
// Forward:   out[i] = round(scale * table[ids[i]]), a row copy.
// Backward:  grad[k] = (old) + scale * sum of the rows i with ids[i] = k.  The ids are argsorted (stable), so
//            entry k owns a contiguous range of the sorted order and its sum is taken in that order: no atomics.
#include "kernels.h"
#include "vecio.h"

namespace fkm {

namespace {

// Entries a wave zeroes at a time: about 32 KB of them, 64 at most.
int zero_per(int64_t row_bytes) {
  const int64_t e = 32768 / row_bytes;
  return e < 1 ? 1 : e > 64 ? 64 : (int)e;
}
int64_t zero_grid(int64_t blocks) { return blocks < (1 << 20) ? blocks : (1 << 20); }

constexpr int kVecs = 4;                  // vectors in flight per thread
constexpr int kTileVecs = 256 * kVecs;    // vectors per workgroup tile

// ---------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------
// A row is nv vectors.  A tile is rpt whole rows (nv <= kTileVecs) or one of
// the nslab slabs of a longer row, either way consecutive vectors of the
// output; workgroups stride over the tiles.  The row of a vector comes from a
// multiplication by `magic` = ceil(2^32 / nv), exact below 2^16, and 64-bit
// products only address the table: with plain divisions and products the
// kernel spent 91 vector instructions per 8 elements and was bound by them
// (2^23 rows of 128 fp32 to bf16: 404 us; 392 so).  The output is streamed
// past the caches, which then keep the table (680 us without).
// LOOSE: rows that are no multiple of 16 bytes or start anywhere.  Vectors have
// element alignment, a row's last one ends with it, and of that one only the
// elements that the one before does not have are stored (65,536 rows of 2,049
// bf16: 95 us, of 2,048 53; element by element 288 us).
template <class TI, class TO, int V, bool LOOSE>
__global__ __launch_bounds__(256) void embed_kernel(const typename TI::raw* __restrict__ table,
                                                    const int32_t* __restrict__ ids, int64_t n, uint32_t N, uint32_t K,
                                                    int nv, int D, uint32_t magic, int rpt, int nslab,
                                                    int64_t tiles, float scale, typename TO::raw* __restrict__ out) {
  for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
    const int64_t row0 = nslab == 1 ? t * rpt : t / nslab;
    const int c0 = nslab == 1 ? 0 : (int)(t - row0 * nslab) * kTileVecs;
    const int64_t left = n - row0;
    const int limit = nslab == 1 ? (int)(left < rpt ? left : rpt) * nv : nv - c0 < kTileVecs ? nv - c0 : kTileVecs;
    typename TO::raw* dst = out + row0 * D;
    const int32_t* id0 = ids + row0;
    // instance of the tile's first row and the rows it has left in it
    const uint32_t b0 = N < n ? (uint32_t)row0 / N : 0u;
    const uint32_t in_b0 = N < n ? N - ((uint32_t)row0 - b0 * N) : ~0u;
    bool live[kVecs];
    uint32_t at[kVecs], row[kVecs];  // column of the vector's first element, and its row in the tile
    Pack<TI, V> v[kVecs];
#pragma unroll
    for (int u = 0; u < kVecs; ++u) {
      const uint32_t l = threadIdx.x + 256 * u;
      const uint32_t r = nslab != 1 ? 0u : nv == 1 ? l : __umulhi(l, magic);
      const uint32_t c = c0 + l - r * (uint32_t)nv;
      row[u] = r;
      at[u] = c * V;
      if constexpr (LOOSE) at[u] = at[u] + V > (uint32_t)D ? (uint32_t)(D - V) : at[u];
      live[u] = false;
      v[u].zero();
      if ((int)l < limit) {
        const uint32_t id = (uint32_t)id0[r];
        live[u] = id < K;
        if (live[u]) {
          uint64_t e = id;
          if (N < n) e += (uint64_t)(r < in_b0 ? b0 : b0 + 1 + (r - in_b0) / N) * K;
          const typename TI::raw* from = table + (e * (uint32_t)D + at[u]);
          if constexpr (LOOSE) v[u].load_loose(from);
          else v[u].load(from);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kVecs; ++u) {
      const int l = threadIdx.x + 256 * u;
      if (l >= limit) continue;
      float f[V];
      v[u].unpack(f);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        f[e] = live[u] ? f[e] * scale : 0.f;
        // an fp32 product for every type: without this the compiler joins it
        // with the rounding to fp16 (and only to fp16) in one instruction
        if constexpr (TO::SZ == 2) asm("" : "+v"(f[e]));
      }
      Pack<TO, V> o;
      o.pack(f);
      if constexpr (LOOSE) {
        typename TO::raw* to = dst + (row[u] * (uint32_t)D + at[u]);
        const uint32_t c = c0 + l - row[u] * (uint32_t)nv;
        if (at[u] == c * V) o.store_loose(to);
        else o.store_range(to, (int)(c * V - at[u]), V);
      } else {
        o.store_nt(dst + (int64_t)(c0 + l) * V);
      }
    }
  }
}

template <class TI, class TO, int V, bool LOOSE>
hipError_t embed_v(const void* table, const int32_t* ids, int64_t N, int K, int D, int B, float scale, void* out,
                   hipStream_t s) {
  const int64_t n = N * B;
  const int nv = (D + V - 1) / V;
  const int nslab = (nv + kTileVecs - 1) / kTileVecs;
  const int rpt = nslab == 1 ? kTileVecs / nv : 1;
  const int64_t tiles = nslab == 1 ? (n + rpt - 1) / rpt : n * nslab;
  const int64_t grid = tiles < (1 << 22) ? tiles : (1 << 22);
  const uint32_t magic = (uint32_t)((((uint64_t)1 << 32) + nv - 1) / nv);  // (nv = 1 does without)
  embed_kernel<TI, TO, V, LOOSE><<<dim3((unsigned)grid), dim3(256), 0, s>>>(
      static_cast<const typename TI::raw*>(table), ids, n, (uint32_t)N, (uint32_t)K, nv, D, magic, rpt, nslab, tiles,
      scale, static_cast<typename TO::raw*>(out));
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// backward
// ---------------------------------------------------------------------------
// How finished sums reach the gradient.
struct PutMode {
  float scale;
  bool add;   // to the old value
  bool keep;  // leave an entry without rows as it is (old values, or zeros written before)
};
// V values of an entry's sum `a` go to `at`; `any`: whether a row that counts
// was among them (an entry without one is zero or stays as it is).
template <class TO, int V>
__device__ __forceinline__ void put_grad(typename TO::raw* grad, int64_t at, const float (&a)[V], const PutMode& m,
                                         bool any) {
  if (m.keep && !any) return;
  Pack<TO, V> o;
  float r[V];
  if (m.add) {
    o.load(grad + at);
    o.unpack(r);
#pragma unroll
    for (int i = 0; i < V; ++i) r[i] = fmaf(m.scale, a[i], r[i]);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) r[i] = any ? m.scale * a[i] : 0.f;
  }
  o.pack(r);
  o.store(grad + at);
}

// Zeros into `count` entries from e0 whose bit in `absent` is set; one wave.
template <class TO, int V>
__device__ __forceinline__ void zero_entries(typename TO::raw* __restrict__ grad, int64_t e0, uint64_t absent,
                                             int nv, int lane) {
  Pack<TO, V> z;
  z.zero();
  for (; absent; absent &= absent - 1) {
    const int64_t e = e0 + __ffsll((unsigned long long)absent) - 1;
    for (int c = lane; c < nv; c += 64) z.store(grad + (e * nv + c) * V);
  }
}

// Few rows (n <= kGradDirect, 256): no sort (256 rows of 1,024 bf16 accumulated
// into 32,000 fp32: 7.4 us so, 16.3 us sorted by one workgroup; with the zeros of
// a fresh gradient, which bound it, 29 us either way at 1,024 columns in one
// buffer, and at 2,048 columns 58 us for 256 rows so, 45 us for 257 sorted).  A
// wave takes row i and a slab of 64 vectors; if no earlier row has its id, it adds every row of that id in
// order.  Further workgroups zero the entries that no row names, each
// looking for its own range of entries among the ids.
template <class TI, class TO, int V>
__global__ __launch_bounds__(256) void embed_grad_direct_kernel(const typename TI::raw* __restrict__ dout,
                                                                const int32_t* __restrict__ ids, int n, uint32_t N,
                                                                uint32_t K, int64_t entries, int nv, int nslab,
                                                                int64_t row_blocks, int64_t units, int per,
                                                                PutMode mode, typename TO::raw* __restrict__ grad) {
  __shared__ uint32_t key[kGradDirect];  // entry of every row, ~0 for none
  __shared__ unsigned long long named[4];
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  if (tid < n) {
    const uint32_t id = (uint32_t)ids[tid];
    key[tid] = id < K ? (uint32_t)tid / N * K + id : ~0u;
  }
  if (tid < 4) named[tid] = 0;
  __syncthreads();
  if ((int64_t)blockIdx.x < row_blocks) {
    const int64_t u = (int64_t)blockIdx.x * 4 + w;
    const int i = (int)(u / nslab);
    if (i >= n) return;
    const uint32_t k = key[i];
    if (k == ~0u) return;
    uint64_t same[kGradDirect / 64];
#pragma unroll
    for (int q = 0; q < kGradDirect / 64; ++q) {
      const int j = q * 64 + lane;
      same[q] = __ballot(j < n && key[j] == k);
      // an earlier row of this entry: that row's wave does the work
      const int below = i - q * 64;
      const uint64_t earlier = below <= 0 ? 0ull : below >= 64 ? ~0ull : (1ull << below) - 1;
      if (same[q] & earlier) return;
    }
    const int c = (int)(u - (int64_t)i * nslab) * 64 + lane;
    if (c >= nv) return;
    float a[V];
#pragma unroll
    for (int v = 0; v < V; ++v) a[v] = 0.f;
#pragma unroll
    for (int q = 0; q < kGradDirect / 64; ++q) {
#pragma unroll 4
      for (uint64_t m = same[q]; m; m &= m - 1) {
        const int j = q * 64 + __ffsll((unsigned long long)m) - 1;
        Pack<TI, V> p;
        float f[V];
        p.load(dout + ((int64_t)j * nv + c) * V);
        p.unpack(f);
#pragma unroll
        for (int v = 0; v < V; ++v) a[v] += f[v];
      }
    }
    put_grad<TO, V>(grad, ((int64_t)k * nv + c) * V, a, mode, true);
    return;
  }
  // zeros: a workgroup takes 4 waves of `per` (at most 64) entries at a time
  for (int64_t u = (int64_t)blockIdx.x - row_blocks; u < units; u += gridDim.x - row_blocks) {
    const int64_t e0 = (u * 4) * per, e1 = e0 + 4 * per;
    if (tid < n) {
      const uint32_t k = key[tid];
      if (k != ~0u && (int64_t)k >= e0 && (int64_t)k < e1)
        atomicOr(&named[(k - e0) / per], 1ull << ((k - e0) % per));
    }
    __syncthreads();
    const int64_t we = e0 + (int64_t)w * per;
    const int64_t left = entries - we;
    const int cnt = left <= 0 ? 0 : left < per ? (int)left : per;
    const uint64_t range = cnt <= 0 ? 0ull : cnt >= 64 ? ~0ull : (1ull << cnt) - 1;
    zero_entries<TO, V>(grad, we, ~named[w] & range, nv, lane);
    __syncthreads();
    if (tid < 4) named[tid] = 0;
    __syncthreads();
  }
}

// Joins the fragments of up to RANGE (64 at most) consecutive units of W sorted rows from
// unit u0 (of `units`), one wave, V columns a lane.  Segments that end inside
// are finished; what crosses the joined range's edges goes to its fragments
// by the same rule.
template <class TO, int V, int RANGE>
__device__ __forceinline__ void join_units(const uint2* __restrict__ kv, int64_t n, int64_t W, int64_t u0,
                                           int64_t units, const float* frag, const uint32_t* fany, int64_t fbase,
                                           int Dp, int nv, int c, bool on, const PutMode& mode,
                                           typename TO::raw* __restrict__ grad, float* ofrag, uint32_t* oany,
                                           int64_t obase, int oDp, int oc, bool flag_lane) {
  const int lane = lane_id();
  const int64_t u = u0 + lane;
  bool from_left = false, to_right = false, one = false, any0 = false, any1 = false;
  uint32_t kl = 0, kf = 0;
  if (lane < RANGE && u < units) {
    const int64_t r0 = u * W, r1 = r0 + W < n ? r0 + W : n;
    kf = kv[r0].x, kl = kv[r1 - 1].x;
    from_left = r0 > 0 && kv[r0 - 1].x == kf;
    to_right = r1 < n && kv[r1].x == kl;
    one = kf == kl;
    any0 = from_left && fany[(u - fbase) * 2];
    any1 = to_right && !(from_left && one) && fany[(u - fbase) * 2 + 1];
  }
  // unit i continues a segment from the left / starts one that goes on to the right; passes one through
  const uint64_t L = __ballot(from_left), P = __ballot(from_left && to_right && one);
  const uint64_t S = __ballot(to_right) & ~P;
  const uint64_t A0 = __ballot(any0), A1 = __ballot(any1);
  auto leave = [&](const float (&a)[V], int which, bool any) {
    if (on) {
#pragma unroll
      for (int v = 0; v < V; ++v) ofrag[(obase * 2 + which) * oDp + oc * V + v] = a[v];
    }
    if (flag_lane) oany[obase * 2 + which] = any;
  };
  float a[V];
#pragma unroll
  for (int v = 0; v < V; ++v) a[v] = 0.f;
  bool any = false, left = true, open = (L & 1) != 0;  // a piece from the left of the range is open at its start
  constexpr int kB = RANGE < 8 ? RANGE : 8;  // units whose fragments are loaded together
  for (int i0 = 0; i0 < RANGE; i0 += kB) {
    if (((L | S) >> i0 & ((1ull << kB) - 1)) == 0) continue;
    float f0[kB][V], f1[kB][V];
#pragma unroll
    for (int i = 0; i < kB; ++i) {
      const int b = i0 + i;
      const int64_t at = (u0 + b - fbase) * 2;
#pragma unroll
      for (int v = 0; v < V; ++v) f0[i][v] = f1[i][v] = 0.f;
      if ((L >> b & 1) && on) {
#pragma unroll
        for (int v = 0; v < V; ++v) f0[i][v] = frag[at * Dp + c * V + v];
      }
      if ((S >> b & 1) && on) {
#pragma unroll
        for (int v = 0; v < V; ++v) f1[i][v] = frag[(at + 1) * Dp + c * V + v];
      }
    }
#pragma unroll
    for (int i = 0; i < kB; ++i) {
      const int b = i0 + i;
      if (L >> b & 1) {
#pragma unroll
        for (int v = 0; v < V; ++v) a[v] += f0[i][v];
        any |= (A0 >> b & 1) != 0;
        if (!(P >> b & 1)) {  // the segment ends in this unit
          if (left) {
            leave(a, 0, any);
          } else if (on) {
            const uint32_t k = __builtin_amdgcn_readlane(kf, b);
            put_grad<TO, V>(grad, ((int64_t)k * nv + c) * V, a, mode, any);
          }
          open = false;
        }
      }
      if (S >> b & 1) {
#pragma unroll
        for (int v = 0; v < V; ++v) a[v] = f1[i][v];
        any = (A1 >> b & 1) != 0;
        left = false;
        open = true;
      }
    }
  }
  if (open) leave(a, left ? 0 : 1, any);  // a piece continues to the right of the range
}

// Level 1.  A group of LPR lanes, one vector each, takes a unit of U sorted
// rows and a slab of LPR vectors, and adds the rows of each segment in order,
// with 8 row loads in flight and their keys read a batch ahead of those.  A
// segment inside the unit is finished here; a piece that continues from the
// left goes to the unit's fragment 0, one that starts here and continues to
// the right to fragment 1; the workgroup joins its units' fragments in LDS
// before any reaches memory.  Rows whose word carries the mark leave nothing.
// The first workgroups zero the entries no row has (unless those keep what
// they hold), finding each by a binary search whose waits the sums fill.
// Bound by the rows' bytes: 2^23 rows of 256 bytes in 0.41 ms, 5.2 TB/s (the
// whole gradient into 65,536 x 128 fp32 0.543 ms, of it 0.104 the sort).  With
// 4 loads in flight 0.557 ms, with loads that stay in the caches 0.580 ms;
// units of at most 128 or 512 rows 0.545 and 0.550 ms.
constexpr int kAhead = 8;
template <int LPR>
constexpr int kGroups = 256 / LPR;
static_assert(3 * kAhead <= kSlack, "pairs read past the last row");
template <class TI, class TO, int V, int LPR>
__global__ __launch_bounds__(256) void embed_grad_sum_kernel(const typename TI::raw* __restrict__ dout,
                                                             const uint2* __restrict__ kv, int64_t n, uint32_t mark,
                                                             int U, int64_t units, int64_t zero_blocks, int nv,
                                                             int nslab, int64_t entries, int per, PutMode mode,
                                                             typename TO::raw* __restrict__ grad,
                                                             float* __restrict__ frag, uint32_t* __restrict__ fany,
                                                             int Dp) {
  constexpr int GPB = kGroups<LPR>;              // units per workgroup
  constexpr int VJ = V >= 4 ? 4 : 1;             // columns per lane in the join
  __shared__ __align__(16) float sfrag[GPB * 2][LPR * V];
  __shared__ uint32_t sany[GPB * 2];
  const int lane = lane_id();
  const int w = threadIdx.x >> 6;
  if ((int64_t)blockIdx.x < zero_blocks) {
    const int64_t zero_units = (entries + per - 1) / per;
    for (int64_t u = (int64_t)blockIdx.x * 4 + w; u < zero_units; u += zero_blocks * 4) {
      const int64_t e = u * per + lane;
      bool absent = false;
      if (lane < per && e < entries) {
        int64_t lo = 0, hi = n;  // first sorted position with a key of at least e
        while (lo < hi) {
          const int64_t m = (lo + hi) >> 1;
          if ((int64_t)kv[m].x < e) lo = m + 1;
          else hi = m;
        }
        absent = lo == n || (int64_t)kv[lo].x != e;
      }
      zero_entries<TO, V>(grad, u * per, __ballot(absent), nv, lane);
    }
    return;
  }
  const int64_t sb = (int64_t)blockIdx.x - zero_blocks;
  const int64_t ub = sb / nslab;  // the workgroup's units: GPB from ub * GPB
  const int slab = (int)(sb - ub * nslab);
  const int grp = threadIdx.x / LPR, gl = threadIdx.x % LPR;
  const int64_t unit = ub * GPB + grp;
  if (unit < units) {
    const int c = slab * LPR + gl;
    const bool on = c < nv;
    const int64_t j0 = unit * U, j1 = j0 + U < n ? j0 + U : n;
    uint32_t cur = kv[j0].x;
    bool left = j0 > 0 && kv[j0 - 1].x == cur;
    const bool more = j1 < n && kv[j1].x == kv[j1 - 1].x;  // the last segment continues to the right
    float a[V];
#pragma unroll
    for (int v = 0; v < V; ++v) a[v] = 0.f;
    bool any = false;
    auto to_frag = [&](int which) {
      if (on) {
        float* f = &sfrag[grp * 2 + which][gl * V];
#pragma unroll
        for (int v = 0; v < V; ++v) f[v] = a[v];
      }
      if (gl == 0) sany[grp * 2 + which] = any;
    };
    // Every row load is issued, so each ring slot keeps its registers: a marked
    // row reads row 0 and a lane past the row its last vector, both left out
    // below.
    const typename TI::raw* base = dout + (int64_t)(on ? c : nv - 1) * V;
    const int64_t pitch = (int64_t)nv * V;
    const uint32_t last = kv[j1 - 1].x;
    // The batch at j, its rows past the unit as its last key, marked.  The loads
    // are never skipped (the sorted pairs have kSlack readable ones behind them):
    // a branch here would make the first wait of every batch wait for them all.
    auto fetch = [&](uint2 (&e)[kAhead], int64_t j) {
      const uint4* p = reinterpret_cast<const uint4*>(kv + j);  // units start at multiples of 16 rows
      const int64_t have = j1 - j;
#pragma unroll
      for (int i = 0; i < kAhead / 2; ++i) {
        const uint4 t = p[i];
        e[2 * i] = 2 * i < have ? make_uint2(t.x, t.y) : make_uint2(last, mark);
        e[2 * i + 1] = 2 * i + 1 < have ? make_uint2(t.z, t.w) : make_uint2(last, mark);
      }
    };
    auto row = [&](Pack<TI, V>& p, const uint2& e) {
      p.load_nt(base + (int64_t)(e.y & mark ? 0u : e.y) * pitch);
    };
    uint2 e[kAhead], en[kAhead];
    Pack<TI, V> p[kAhead];
    auto add = [&](const Pack<TI, V>& x, const uint2& e) {
      if (e.x != cur) {
        if (left) to_frag(0);
        else if (on) put_grad<TO, V>(grad, ((int64_t)cur * nv + c) * V, a, mode, any);
        cur = e.x;
        left = any = false;
#pragma unroll
        for (int v = 0; v < V; ++v) a[v] = 0.f;
      }
      if (!(e.y & mark)) {
        float f[V];
        x.unpack(f);
#pragma unroll
        for (int v = 0; v < V; ++v) a[v] += f[v];
        any = true;
      }
    };
    fetch(e, j0);
    fetch(en, j0 + kAhead);
#pragma unroll
    for (int i = 0; i < kAhead; ++i) row(p[i], e[i]);
    int64_t j = j0;
    for (; j + kAhead < j1; j += kAhead) {
      uint2 e2[kAhead];
      fetch(e2, j + 2 * kAhead);
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        add(p[i], e[i]);
        row(p[i], en[i]);  // the same slot of the next batch
        e[i] = en[i];
        en[i] = e2[i];
      }
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) add(p[i], e[i]);
    if (left) to_frag(0);
    else if (more) to_frag(1);
    else if (on) put_grad<TO, V>(grad, ((int64_t)cur * nv + c) * V, a, mode, any);
  }
  __syncthreads();
  // the units' fragments joined: 64 lanes of VJ columns a wave
  constexpr int LJ = LPR * V / VJ;  // lanes that the slab takes
  if (w * 64 < LJ) {
    const int lj = w * 64 + lane, nj = nv * V / VJ;
    const int cj = slab * LJ + lj;
    const int64_t u0 = ub * GPB;
    join_units<TO, VJ, GPB>(kv, n, U, u0, units < u0 + GPB ? units : u0 + GPB, &sfrag[0][0] + (lj - cj) * VJ, sany, u0,
                            LPR * V, nj, cj, lj < LJ && cj < nj, mode, grad, frag, fany, ub, Dp, cj,
                            lj == 0 && slab == 0);
  }
}

constexpr int kRange = kJoin / 16;
// One workgroup joins kJoin units (16 waves of kRange, then one wave joins
// the 16) for a slab of 64 vectors of V columns.
template <class TO, int V>
__global__ __launch_bounds__(1024) void embed_grad_join_kernel(const uint2* __restrict__ kv, int64_t n, int64_t W,
                                                               int64_t units, int nslab, const float* __restrict__ frag,
                                                               const uint32_t* __restrict__ fany, int Dp, int nv,
                                                               PutMode mode, typename TO::raw* __restrict__ grad,
                                                               float* __restrict__ ofrag, uint32_t* __restrict__ oany) {
  __shared__ __align__(16) float sfrag[16 * 2][64 * V];
  __shared__ uint32_t sany[16 * 2];
  const int lane = lane_id();
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t g = blockIdx.x / nslab;
  const int slab = (int)(blockIdx.x - g * nslab);
  const int c = slab * 64 + lane;
  const bool on = c < nv;
  const int64_t u0 = g * kJoin + w * kRange;
  if (u0 < units)
    join_units<TO, V, kRange>(kv, n, W, u0, units, frag, fany, 0, Dp, nv, c, on, mode, grad, &sfrag[0][0], sany, w,
                      64 * V, lane, lane == 0);
  __syncthreads();
  if (w == 0) {
    const int64_t all = (units + kRange - 1) / kRange, s0 = g * 16;
    const int64_t s1 = s0 + 16 < all ? s0 + 16 : all;
    // the 16 joined ranges are units of kRange * W rows; their fragments are in LDS
    join_units<TO, V, kRange>(kv, n, kRange * W, s0, s1, &sfrag[0][0] + (lane - c) * V, sany, s0, 64 * V, nv, c, on,
                              mode, grad, ofrag, oany, g, Dp, c, lane == 0 && slab == 0);
  }
}

// Returns the units left to join.
template <class TI, class TO, int V, int LPR>
int64_t sum_launch(const void* dout, const uint2* kv, int64_t n, uint32_t mark, int U, int nv, int64_t entries,
                   const PutMode& mode, void* grad, float* frag, uint32_t* fany, int Dp, hipStream_t s) {
  constexpr int GPB = kGroups<LPR>;
  const int64_t units = (n + U - 1) / U, ublocks = (units + GPB - 1) / GPB;
  const int nslab = (nv + LPR - 1) / LPR;
  const int64_t sum_blocks = ublocks * nslab;
  const int per = zero_per(nv * V * TO::SZ);
  const int64_t zero_blocks = mode.keep ? 0 : zero_grid((entries + 4 * per - 1) / (4 * per));
  embed_grad_sum_kernel<TI, TO, V, LPR><<<dim3((unsigned)(sum_blocks + zero_blocks)), dim3(256), 0, s>>>(
      static_cast<const typename TI::raw*>(dout), kv, n, mark, U, units, zero_blocks, nv, nslab, entries, per, mode,
      static_cast<typename TO::raw*>(grad), frag, fany, Dp);
  return ublocks;
}

// Up to kSortOne rows, where a word holds key and row: 16,384 rows of 2,048
// bf16 into 32,000 fp32 in 75 us (86 us when each call has another buffer),
// 16,385 rows with the sort's own launches and zeros by binary search in 104 us;
// 4,099 rows of 1,024 accumulated into 131,072 in 36.5 against 52 us when the
// limit was chosen (now 32).  Against it: 16,384 rows of 16 into 1,000 take 49 us
// so, 16,385 take 42.  One workgroup argsorts the ids in LDS (stable radix passes
// of 8 or 9 bits over 32-bit words: key, out-of-range bit, row), and the other
// workgroups of the launch meanwhile zero the gradient.  Ranks as in the sort of
// many rows: digit matches inside a wave, a counter per wave and digit, waves in
// row order.
constexpr int kSortWaves = 16;
// R: rounds of 64 keys per wave (the keys stay in registers); RB: digit bits
// (9 where that saves a pass, as for keys of 17 and 18 bits: 36.5 to 33.4 us for
// the 4,099 rows above, 52.3 to 46.2 us for 15,333 rows of 16 into 92,338).
template <int R, int RB>
__global__ __launch_bounds__(1024) void embed_grad_sort_kernel(const int32_t* __restrict__ ids, int n, uint32_t N,
                                                               uint32_t K, int row_bits, int passes,
                                                               uint2* __restrict__ kv, uint8_t* __restrict__ zero,
                                                               int head, size_t words, int tail) {
  const int tid = threadIdx.x;
  if (blockIdx.x > 0) {
    // `head` bytes, `words` 16-byte words, `tail` bytes
    if (blockIdx.x == 1 && tid < 16) {
      if (tid < head) zero[tid] = 0;
      if (tid < tail) zero[head + words * 16 + tid] = 0;
    }
    uint4* body = reinterpret_cast<uint4*>(zero + head);
    const size_t step = (size_t)(gridDim.x - 1) * 1024;
    for (size_t i = (size_t)(blockIdx.x - 1) * 1024 + tid; i < words; i += step) body[i] = make_uint4(0, 0, 0, 0);
    return;
  }
  __shared__ uint32_t word[kSortWaves * 64 * R];
  constexpr uint32_t DIG = 1u << RB;
  __shared__ uint32_t cnt[kSortWaves][DIG];
  __shared__ __align__(16) uint32_t tot[DIG];
  const int lane = tid & 63, w = tid >> 6;
  const int first = w * R * 64;
  uint32_t x[R], rank[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int i = first + r * 64 + lane;
    const int at = i < n ? i : n - 1;  // (unconditional, so the words stay in separate registers)
    const uint32_t id = (uint32_t)ids[at];
    const uint32_t key = (N < (uint32_t)n ? (uint32_t)at / N * K : 0u) + (id < K ? id : K - 1);
    x[r] = (key << 1 | (id < K ? 0u : 1u)) << row_bits | (uint32_t)at;
  }
  for (int p = 0; p < passes; ++p) {
    const int shift = row_bits + 1 + RB * p;
    for (int i = tid; i < kSortWaves * (int)DIG; i += 1024) cnt[i >> RB][i & (DIG - 1)] = 0;
    __syncthreads();
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const bool valid = first + r * 64 + lane < n;
      const uint32_t d = x[r] >> shift & (DIG - 1);
      const uint64_t m = match_digit<RB>(d, valid);
      const uint32_t low = (uint32_t)__popcll(m & ((1ull << lane) - 1ull));
      const uint32_t before = cnt[w][d];
      rank[r] = before + low;
      if (valid && low == 0) cnt[w][d] = before + (uint32_t)__popcll(m);
      // one round after the other: matching 16 rounds at once would not fit the registers
      if constexpr (R > 8) __builtin_amdgcn_sched_barrier(0);
    }
    __syncthreads();
    if (tid < (int)DIG) {
      uint32_t run = 0;
#pragma unroll
      for (int q = 0; q < kSortWaves; ++q) {
        const uint32_t c = cnt[q][tid];
        cnt[q][tid] = run;
        run += c;
      }
      tot[tid] = run;
    }
    __syncthreads();
    if (w == 0) {  // exclusive scan of the digit totals, PER a lane
      constexpr int PER = (int)DIG / 64;
      uint32_t t[PER], s = 0;
#pragma unroll
      for (int q = 0; q < PER; ++q) t[q] = tot[PER * lane + q], s += t[q];
      uint32_t inc = s;
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const uint32_t v = __shfl_up(inc, o);
        if (lane >= o) inc += v;
      }
      uint32_t run = inc - s;
#pragma unroll
      for (int q = 0; q < PER; ++q) tot[PER * lane + q] = run, run += t[q];
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const uint32_t d = x[r] >> shift & (DIG - 1);
      if (first + r * 64 + lane < n) word[tot[d] + cnt[w][d] + rank[r]] = x[r];
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < R; ++r) {
      x[r] = word[first + r * 64 + lane];  // (words past n are not used)
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int i = first + r * 64 + lane;
    if (i < n)
      kv[i] = make_uint2(x[r] >> (row_bits + 1),
                         (x[r] & ((1u << row_bits) - 1)) | (x[r] >> row_bits & 1u) << 31);
  }
}

int bits_for(int64_t values) {  // bits that hold 0 .. values - 1
  int b = 1;
  while (((int64_t)1 << b) < values) ++b;
  return b;
}
bool grad_sorts_in_one(int64_t n, int64_t entries) {
  return n <= kSortOne && bits_for(entries) + 1 + bits_for(n) <= 32;
}
// Zeroes `bytes` at `zero` too, if there are any.
void sort_one_launch(const int32_t* ids, int64_t n, uint32_t N, uint32_t K, int64_t entries, uint2* kv, void* zero,
                     size_t bytes, hipStream_t s) {
  size_t head = 0, words = 0, tail = 0;
  int64_t blocks = 0;
  if (zero) {
    head = (16 - (uintptr_t)zero % 16) % 16;
    if (head > bytes) head = bytes;
    words = (bytes - head) / 16;
    tail = bytes - head - words * 16;
    blocks = (int64_t)(words / 4096) + 1;  // four words a thread
    if (blocks > 2048) blocks = 2048;
  }
  const int bits = bits_for(entries);
  const bool nine = (bits + 8) / 9 < (bits + 7) / 8;
  const int passes = nine ? (bits + 8) / 9 : (bits + 7) / 8;
  auto go = [&](auto eight_bits, auto nine_bits) {
    (nine ? nine_bits : eight_bits)<<<dim3((unsigned)(1 + blocks)), dim3(1024), 0, s>>>(
        ids, (int)n, N, K, bits_for(n), passes, kv, static_cast<uint8_t*>(zero), (int)head, words, (int)tail);
  };
  static_assert(kSortOne == kSortWaves * 64 * 16, "the longest sort's rounds");
  if (n <= 1024) go(embed_grad_sort_kernel<1, 8>, embed_grad_sort_kernel<1, 9>);
  else if (n <= 2048) go(embed_grad_sort_kernel<2, 8>, embed_grad_sort_kernel<2, 9>);
  else if (n <= 4096) go(embed_grad_sort_kernel<4, 8>, embed_grad_sort_kernel<4, 9>);
  else if (n <= 8192) go(embed_grad_sort_kernel<8, 8>, embed_grad_sort_kernel<8, 9>);
  else go(embed_grad_sort_kernel<16, 8>, embed_grad_sort_kernel<16, 9>);
}

template <class TI, class TO, int V>
hipError_t embed_grad_v(const void* dout, const int32_t* ids, int64_t N, int K, int D, int B, float scale, bool acc,
                        void* grad, GradBuffers& buf, hipStream_t s) {
  const int64_t n = N * B, entries = (int64_t)B * K;
  const int nv = D / V;
  if (n <= kGradDirect) {
    const int nslab = (nv + 63) / 64;
    const int per = zero_per(D * TO::SZ);
    const int64_t row_blocks = (n * nslab + 3) / 4;
    const int64_t units = acc ? 0 : (entries + 4 * per - 1) / (4 * per);
    const int64_t blocks = row_blocks + zero_grid(units);
    embed_grad_direct_kernel<TI, TO, V><<<dim3((unsigned)blocks), dim3(256), 0, s>>>(
        static_cast<const typename TI::raw*>(dout), ids, (int)n, (uint32_t)N, (uint32_t)K, entries, nv, nslab,
        row_blocks, units, per, PutMode{scale, acc, acc}, static_cast<typename TO::raw*>(grad));
    return hipGetLastError();
  }
  const uint2* kv = nullptr;
  uint32_t mark = 0;
  PutMode mode{scale, acc, acc};
  if (grad_sorts_in_one(n, entries)) {
    kv = buf.sort.kv[0];
    mark = 1u << 31;
    sort_one_launch(ids, n, (uint32_t)N, (uint32_t)K, entries, buf.sort.kv[0], acc ? nullptr : grad,
                    (size_t)entries * D * TO::SZ, s);
    mode.keep = true;  // what is left of the zeros it wrote stays
  } else {
    const hipError_t e = launch_argsort_marked(ids, N, B, K, buf.sort, &kv, &mark, s);
    if (e != hipSuccess) return e;
  }
  const int U = grad_unit(n, D);
  const int Dp = (D + 3) / 4 * 4;
  int64_t units = 0, W = U;
#define FKM_SUM(LPR)                                                                                                  \
  units = sum_launch<TI, TO, V, LPR>(dout, kv, n, mark, U, nv, entries, mode, grad, buf.frag[0], buf.any[0], Dp, s), \
  W *= kGroups<LPR>
  if (nv <= 4) FKM_SUM(4);
  else if (nv <= 8) FKM_SUM(8);
  else if (nv <= 16) FKM_SUM(16);
  else if (nv <= 32) FKM_SUM(32);
  else FKM_SUM(64);
#undef FKM_SUM
  constexpr int VJ = V >= 4 ? 4 : 1;
  const int nslab = (D / VJ + 63) / 64;
  for (int level = 0; units > 1; ++level) {
    const int64_t groups = (units + kJoin - 1) / kJoin;
    const int waves = units < kJoin ? (int)((units + kRange - 1) / kRange) : 16;
    embed_grad_join_kernel<TO, VJ><<<dim3((unsigned)(groups * nslab)), dim3(waves * 64), 0, s>>>(
        kv, n, W, units, nslab, buf.frag[level], buf.any[level], Dp, D / VJ, mode,
        static_cast<typename TO::raw*>(grad), buf.frag[level + 1], buf.any[level + 1]);
    W *= kJoin;
    units = groups;
  }
  return hipGetLastError();
}

}  // namespace

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
  return with_type(tdt, [&](auto ti) {
    return with_type(odt, [&](auto to) {
      using TI = decltype(ti);
      using TO = decltype(to);
      constexpr int V = 16 / TO::SZ;
      if (vec_width(D, V, table, TI::SZ, out, TO::SZ) == V)
        return embed_v<TI, TO, V, false>(table, ids, N, K, D, B, scale, out, s);
      if (D >= V) return embed_v<TI, TO, V, true>(table, ids, N, K, D, B, scale, out, s);
      return embed_v<TI, TO, 1, false>(table, ids, N, K, D, B, scale, out, s);
    });
  });
}

hipError_t launch_embed_grad(int idt, int gdt, const void* dout, const int32_t* ids, int64_t N, int K, int D, int B,
                             float scale, bool acc, void* grad, GradBuffers& buf, hipStream_t s) {
  const int w = vec_width(D, 16 / dtype_size(idt), dout, dtype_size(idt), grad, dtype_size(gdt));
  return with_type(idt, [&](auto ti) {
    return with_type(gdt, [&](auto to) {
      using TI = decltype(ti);
      using TO = decltype(to);
      if constexpr (TI::SZ == 2) {  // (four fp32 are 16 bytes)
        if (w == 8) return embed_grad_v<TI, TO, 8>(dout, ids, N, K, D, B, scale, acc, grad, buf, s);
      }
      if (w == 4) return embed_grad_v<TI, TO, 4>(dout, ids, N, K, D, B, scale, acc, grad, buf, s);
      return embed_grad_v<TI, TO, 1>(dout, ids, N, K, D, B, scale, acc, grad, buf, s);
    });
  });
}

}  // namespace fkm
