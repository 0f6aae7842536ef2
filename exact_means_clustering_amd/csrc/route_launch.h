// Which of the routing kernels a call takes (internal).
#pragma once

#include "route_rows.h"

namespace fkm {

namespace {

// Fewer choices than this in all (2,048 for each of 1,024 SIMDs) are few rows (16,384 x 128 bf16 5.9 us as few rows, 6.2
// as many; 32,768 x 128 10.0 and 7.3; 8,192 x 64 3.5 and 4.8; 16,384 x 256 fp32 in 8 groups 48 and 51).
constexpr int64_t kRouteFew = (int64_t)1 << 21;

template <class T>
__global__ __launch_bounds__(256) void route_exact_kernel(RouteArgs<T> a) {
  for (int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); row < a.n; row += (int64_t)gridDim.x * 4)
    route_row_exact(a, row);
}

template <class T, int E, int LPR, int L, RouteMode MODE>
hipError_t route_rows(const RouteArgs<T>& a, hipStream_t s) {
  constexpr int SL = 64 / LPR, V = 16 / T::SZ;
  const RouteLds o = RouteLds::of(SL, MODE == kScored ? a.K : 0, a.G, a.S, MODE == kScored);
  // waves of a workgroup share nothing: as many as leave room for several workgroups a CU
  int waves = 4;
  while (waves > 1 && waves * o.total * 4 > 40960) waves /= 2;
  const int64_t tiles = (a.n + SL - 1) / SL;
  // waves that loop where there are many rows (262,144 x 1,024 bf16, 8 a row, 201 us with 64 a CU, 216 with 24; 65,536 x
  // 256 fp32 in 8 groups with a bias 41 us with 24, 44 with 20, 49 with 16, 54 with 64)
  const int64_t want = (tiles + waves - 1) / waves, most = 256 * (MODE == kScored ? 24 : 64) / waves;
  const bool loose = a.K % V != 0 || (uintptr_t)a.logits % 16 != 0;
  route_rows_kernel<T, E, LPR, L, MODE>
      <<<dim3((unsigned)(want < most ? want : most)), dim3(64 * waves),
         waves * o.total * 4 + (MODE == kScored ? LPR * E * 4 + 16 : 0), s>>>(
          a, loose, o, ((1u << 20) + a.S - 1) / a.S, ((1u << 20) + a.G - 1) / a.G);
  return hipGetLastError();
}

template <class T, int L, RouteMode MODE>
hipError_t route_l(const RouteArgs<T>& a, hipStream_t s) {
  if (a.K <= 8) return route_rows<T, 8, 1, (L < 8 ? L : 8), MODE>(a, s);
  if (a.K <= 16) return route_rows<T, 16, 1, (L < 16 ? L : 16), MODE>(a, s);
  // few rows: four times the lanes for each, so that a wave has less to do after the other
  if constexpr (L <= 8) {
    if (a.n * a.K < kRouteFew) {
      if (a.K <= 32) return route_rows<T, 8, 4, L, MODE>(a, s);
      if (a.K <= 64) return route_rows<T, 8, 8, L, MODE>(a, s);
      if (a.K <= 128) return route_rows<T, 8, 16, L, MODE>(a, s);
      if (a.K <= 256) return route_rows<T, 8, 32, L, MODE>(a, s);
      if (a.K <= 512) return route_rows<T, 8, 64, L, MODE>(a, s);
    }
  }
  if (a.K <= 32) return route_rows<T, 32, 1, L, MODE>(a, s);
  if (a.K <= 64) return route_rows<T, 32, 2, L, MODE>(a, s);
  if (a.K <= 128) return route_rows<T, 32, 4, L, MODE>(a, s);
  if (a.K <= 256) return route_rows<T, 32, 8, L, MODE>(a, s);
  if (a.K <= 512) return route_rows<T, 32, 16, L, MODE>(a, s);
  if (a.K <= 1024) return route_rows<T, 32, 32, L, MODE>(a, s);
  return route_rows<T, 32, 64, L, MODE>(a, s);
}

template <class T>
hipError_t route_t(const RouteCall& c, hipStream_t s) {
  const RouteArgs<T> a{static_cast<const typename T::raw*>(c.logits), c.n, c.K, c.bias, c.groups, c.keep, c.best, c.S,
                       c.softmax, c.renorm, c.scale, c.valid, c.ids, c.weights, c.chosen};
  // Lists of more than 32 keys, and scores of rows longer than a wave's registers, are left to the kernel without either
  // (8,192 x 128 bf16 with 32 selections 26 us, with 33 42; 8,192 x 2,048 bf16 with a bias 80 us, x 4,096 252).
  if (a.S > 32 || (a.K > 2048 && (a.arith() || a.G > 1))) {
    const int64_t blocks = (a.n + 3) / 4;
    route_exact_kernel<T><<<dim3((unsigned)(blocks < (1 << 20) ? blocks : (1 << 20))), dim3(256), 0, s>>>(a);
    return hipGetLastError();
  }
  if (a.arith() || a.G > 1) return a.S <= 8 ? route_l<T, 8, kScored>(a, s) : route_l<T, 32, kScored>(a, s);
  if (a.K > 2048)
    return a.S <= 2   ? route_rows<T, 32, 64, 2, kWide>(a, s)
           : a.S <= 8 ? route_rows<T, 32, 64, 8, kWide>(a, s)
                      : route_rows<T, 32, 64, 32, kWide>(a, s);
  return a.S <= 2   ? route_l<T, 2, kPlain>(a, s)
         : a.S <= 8 ? route_l<T, 8, kPlain>(a, s)
                    : route_l<T, 32, kPlain>(a, s);
}

}  // namespace

}  // namespace fkm
