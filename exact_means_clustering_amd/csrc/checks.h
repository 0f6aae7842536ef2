// Argument checks shared by the ABI entry points of the codebook and training operators (internal).
#pragma once

#include "workspace.h"

#include "flashkm.h"

namespace fkm {

inline int hip_fail(hipError_t e, const char* what) { return fail(KM_EHIP, "%s: %s", what, hipGetErrorString(e)); }

#define KM_HIP(expr, what)                           \
  do {                                               \
    hipError_t e_ = (expr);                          \
    if (e_ != hipSuccess) return hip_fail(e_, what); \
  } while (0)

constexpr int64_t kMax31 = (int64_t)1 << 31;

inline bool known_type(int dt) { return dt == KM_F32 || dt == KM_F16 || dt == KM_BF16; }

inline int check_type(int dt, const char* name) {
  if (!known_type(dt)) return fail(KM_EUNSUPPORTED, "unsupported %s %d", name, dt);
  return KM_OK;
}

// One array of a call: its name, address, bytes and element size.
struct Arr {
  const char* name;
  const void* p;
  uint64_t bytes;
  unsigned align;
  bool out;
};

// Present and aligned where it has elements; no output overlaps another array.
template <int M>
int check_arrays(const Arr (&a)[M]) {
  for (const Arr& x : a) {
    if (x.bytes && !x.p) return fail(KM_EINVAL, "%s must be non-null", x.name);
    if ((uintptr_t)x.p % x.align) return fail(KM_EINVAL, "misaligned pointer: %s needs %u bytes", x.name, x.align);
  }
  for (int i = 0; i < M; ++i)
    for (int j = 0; j < M; ++j) {
      if (i == j || !a[i].out || !a[i].bytes || !a[j].bytes) continue;
      const uint64_t p = (uintptr_t)a[i].p, q = (uintptr_t)a[j].p;
      if (p < q + a[j].bytes && q < p + a[i].bytes) return fail(KM_EINVAL, "%s overlaps %s", a[i].name, a[j].name);
    }
  return KM_OK;
}

}  // namespace fkm
