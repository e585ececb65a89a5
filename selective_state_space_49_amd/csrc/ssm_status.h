// ssm_status.h -- what the C entry points share: statuses with a detail string, and the
// checks of pointers.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "ssm_scan.h"

namespace ssm {

// Sets this thread's detail string and returns s.
__attribute__((format(printf, 2, 3))) ssm_status fail(ssm_status s, const char *fmt, ...);
// Clears it.
ssm_status ok();

inline bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }

inline bool overlaps(const void *a, size_t na, const void *b, size_t nb) {
    if (!a || !b || na == 0 || nb == 0) return false;
    const uintptr_t pa = (uintptr_t)a, pb = (uintptr_t)b;
    return pa < pb + nb && pb < pa + na;
}

inline ssm_status launch_status(hipError_t e, const char *what) {
    if (e != hipSuccess) return fail(SSM_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
    return ok();
}

}  // namespace ssm
