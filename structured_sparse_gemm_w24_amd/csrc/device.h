// Host helpers shared by the files that export device entry points.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace ssg {

// SSG_OK if a gfx950 device is current; SSG_ENODEV / SSG_EARCH / SSG_EHIP otherwise.
int check_device();

// SSG_OK and a cleared message after a good launch, else SSG_EHIP naming it.
int launched(hipError_t e, const char *what);

// Shape and pointer checks of the row-major GEMMs: SSG_OK (also for M = 0) or
// SSG_EINVAL with a message that names fn.
int check_gemm(const char *fn, const void *A, const void *W, const void *C, int64_t M, int64_t N, int64_t K,
               int k_mult, int n_mult);

inline bool fits_int(int64_t v) { return v >= 0 && v < (int64_t(1) << 31); }

}  // namespace ssg
