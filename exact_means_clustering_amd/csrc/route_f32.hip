// Routing of fp32 logits (a source of its own, so that the types compile side by side).
#include "route_launch.h"

namespace fkm {

hipError_t route_f32(const RouteCall& c, hipStream_t s) { return route_t<F32>(c, s); }

}  // namespace fkm
