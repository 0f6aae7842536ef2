// Gradient of the routing weights with respect to the logits (formulas in flashkm_train.h).
#include "route.h"

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

// One row by one wave; lane j holds selection j.
template <class T>
__global__ __launch_bounds__(256) void route_grad_simple_kernel(GradArgs<T> a) {
  const int lane = lane_id();
  const bool dense = a.softmax && !a.renorm;
  for (int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); row < a.n; row += (int64_t)gridDim.x * 4) {
    const int64_t at = row * a.S + lane;
    const uint32_t id = lane < a.S ? (uint32_t)a.ids[at] : ~0u;
    const bool live = id < (uint32_t)a.K;
    const float g = live ? a.scale * a.dweights[at] : 0.f;
    const typename T::raw* x = dense ? a.logits + row * a.K : nullptr;
    typename T::raw* out = a.dlogits + row * a.K;
    float d = 0.f, high = -INFINITY, inv = 0.f, mean = 0.f;
    const bool any = __ballot(live) != 0;
    if (dense) {
      for (int k = lane; any && k < a.K; k += 64) high = fmaxf(high, T::to_f32(x[k]));
      high = team_max<64>(high);
      float s = 0.f;
      for (int k = lane; any && k < a.K; k += 64) s += exp_diff<F32>(T::to_f32(x[k]), high);
      inv = any ? 1.f / team_sum<64>(s) : 0.f;
      mean = team_sum<64>(live ? g * exp_diff<F32>(T::to_f32(x[id]), high) * inv : 0.f);
      d = g;
    } else {
      const float z = live ? a.chosen[at] : -INFINITY;
      if (a.renorm) {
        const float shift = share_shift(team_max<64>(z), a.softmax);
        const float t = live ? share_term(z, shift, a.softmax) : 0.f;
        const float w = t / team_sum<64>(t);
        mean = team_sum<64>(live ? w * g : 0.f);
        d = w * (g - mean);
        if (!a.softmax) d *= 1.f / (1.f + exp_to(z));
      } else {
        d = g * (1.f / (1.f + exp_to(-z))) * (1.f / (1.f + exp_to(z)));
      }
    }
    for (int64_t k0 = 0; k0 < a.K; k0 += 64) {
      const int64_t k = k0 + lane;
      float sum = 0.f;
      bool hit = dense && any;
      for (int j = 0; j < a.S; ++j) {
        const uint32_t ij = __shfl(id, j);
        const float dj = __shfl(d, j);
        if (ij < (uint32_t)a.K && ij == (uint64_t)k) sum += dj, hit = true;
      }
      if (k >= a.K) continue;
      if (dense) sum = any ? exp_diff<F32>(T::to_f32(x[k]), high) * inv * (sum - mean) : 0.f;
      if (!hit && a.accumulate) continue;
      out[k] = round_to<T>(a.accumulate ? T::to_f32(out[k]) + sum : sum);
    }
  }
}

template <class T>
hipError_t route_grad_t(const RouteGradCall& c, hipStream_t s) {
  GradArgs<T> a{static_cast<const typename T::raw*>(c.logits), c.n, c.K, c.ids, c.chosen, c.dweights, c.S, c.softmax,
                c.renorm, c.scale, c.accumulate, static_cast<typename T::raw*>(c.dlogits)};
  const int64_t blocks = (a.n + 3) / 4;
  route_grad_simple_kernel<T><<<dim3((unsigned)(blocks < (1 << 20) ? blocks : (1 << 20))), dim3(256), 0, s>>>(a);
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
