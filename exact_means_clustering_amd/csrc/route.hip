// Routing of rows to choices (formulas in flashkm_train.h).
#include "kernels.h"

namespace fkm {

hipError_t route_f32(const RouteCall& c, hipStream_t s);
hipError_t route_f16(const RouteCall& c, hipStream_t s);
hipError_t route_bf16(const RouteCall& c, hipStream_t s);

hipError_t launch_route(int dt, const RouteCall& c, hipStream_t s) {
  switch (dt) {
    case DT_F32: return route_f32(c, s);
    case DT_F16: return route_f16(c, s);
    case DT_BF16: return route_bf16(c, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace fkm
