// Routing of bf16 logits (a source of its own, so that the types compile side by side).
#include "route_launch.h"

namespace fkm {

hipError_t route_bf16(const RouteCall& c, hipStream_t s) { return route_t<BF16>(c, s); }

}  // namespace fkm
