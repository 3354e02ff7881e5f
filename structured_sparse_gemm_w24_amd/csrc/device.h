// Host helpers shared by the files that export device entry points.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace ssg {

// SSG_OK if a gfx950 device is current; SSG_ENODEV / SSG_EARCH / SSG_EHIP otherwise.
int check_device();

// SSG_OK and a cleared message after a good launch, else SSG_EHIP naming it.
int launched(hipError_t e, const char *what);

inline bool fits_int(int64_t v) { return v >= 0 && v < (int64_t(1) << 31); }

}  // namespace ssg
