// Routing of rows to choices (formulas in flashkm_train.h).
#include "route.h"

namespace fkm {

namespace {

template <class T>
__global__ __launch_bounds__(256) void route_exact_kernel(RouteArgs<T> a) {
  for (int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); row < a.n; row += (int64_t)gridDim.x * 4)
    route_row_exact(a, row);
}

template <class T>
hipError_t route_t(const RouteCall& c, hipStream_t s) {
  RouteArgs<T> a{static_cast<const typename T::raw*>(c.logits), c.n, c.K, c.bias, c.groups, c.keep, c.best, c.S,
                 c.softmax, c.renorm, c.scale, c.valid, c.ids, c.weights, c.chosen};
  const int64_t blocks = (a.n + 3) / 4;
  route_exact_kernel<T><<<dim3((unsigned)(blocks < (1 << 20) ? blocks : (1 << 20))), dim3(256), 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_route(int dt, const RouteCall& c, hipStream_t s) {
  switch (dt) {
    case DT_F32: return route_t<F32>(c, s);
    case DT_F16: return route_t<F16>(c, s);
    case DT_BF16: return route_t<BF16>(c, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace fkm
