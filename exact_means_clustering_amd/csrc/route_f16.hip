// Routing of fp16 logits (a source of its own, so that the types compile side by side).
#include "route_launch.h"

namespace fkm {

hipError_t route_f16(const RouteCall& c, hipStream_t s) { return route_t<F16>(c, s); }

}  // namespace fkm
