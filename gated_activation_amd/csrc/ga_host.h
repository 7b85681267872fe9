// Host-side helpers shared by the C-ABI's source files (defined in api.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/ga.h"

namespace ga {

// Records the message ga_last_error returns on this thread and passes `st` on.
ga_status fail(ga_status st, const char *fmt, ...) __attribute__((format(printf, 2, 3)));
const char *last_error();
// GA_OK, or GA_EHIP with the launch's error.
ga_status launched(const char *op, hipError_t e);
// Bytes of an element, 0 for an unknown dtype.
size_t elem_size(int32_t dtype);
bool overlaps(const void *a, size_t abytes, const void *b, size_t bbytes);
// Compute units of the current device.
ga_status current_cus(int *cus);

}  // namespace ga
