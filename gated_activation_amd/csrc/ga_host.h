// Host-side helpers shared by the C-ABI's source files (defined in api.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/ga.h"
#include "ga_internal.h"

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

// One array of a call, for the checks that all share.
struct Region {
    const char *name;
    const void *at;
    size_t bytes;
    size_t align;
    bool written;
    bool optional;
};

// Null, misaligned and overlapping arrays.  Arrays without a byte may be null;
// one that is written overlaps no other.
template <int N>
inline ga_status check_regions(const char *op, const Region (&r)[N]) {
    for (int i = 0; i < N; ++i) {
        if (r[i].at == nullptr) {
            if (r[i].optional || r[i].bytes == 0) continue;
            return fail(GA_EINVAL, "%s: null %s", op, r[i].name);
        }
        if ((uintptr_t)r[i].at % r[i].align != 0)
            return fail(GA_EINVAL, "%s: %s is not aligned to %zu bytes", op, r[i].name, r[i].align);
        for (int j = 0; j < i; ++j) {
            if (r[j].at == nullptr || !(r[i].written || r[j].written) || r[i].bytes == 0 || r[j].bytes == 0) continue;
            if (overlaps(r[i].at, r[i].bytes, r[j].at, r[j].bytes))
                return fail(GA_EINVAL, "%s: %s and %s overlap", op, r[j].name, r[i].name);
        }
    }
    return GA_OK;
}

inline ga_status check_sizes(const char *op, int64_t rows, int64_t d, int64_t most_d, int32_t dtype) {
    if (rows < 0 || rows > INT32_MAX)
        return fail(GA_EINVAL, "%s: row count %lld out of [0, 2^31)", op, (long long)rows);
    if (d < 1) return fail(GA_EINVAL, "%s: d = %lld must be >= 1", op, (long long)d);
    if (elem_size(dtype) == 0) return fail(GA_EINVAL, "%s: unknown dtype %d", op, (int)dtype);
    if (d > most_d) return fail(GA_EUNSUPPORTED, "%s: d = %lld above %lld", op, (long long)d, (long long)most_d);
    return GA_OK;
}

inline int64_t blocks_of(int64_t d) { return (d + GA_CHECKPOINT_BLOCK - 1) / GA_CHECKPOINT_BLOCK; }

// Elementwise kernels number the blocks of 128 values in 31 bits; the launches
// of kernels that give a row `lanes` work-items have fewer than 2^32.
inline ga_status check_blocks(const char *op, int64_t blocks) {
    if (blocks > INT32_MAX)
        return fail(GA_EUNSUPPORTED, "%s: %lld blocks of 128 values in one call (2^31 or more)", op, (long long)blocks);
    return GA_OK;
}

inline ga_status check_items(const char *op, int64_t rows, int64_t lanes) {
    if (rows * lanes + 1024 > (int64_t)UINT32_MAX)
        return fail(GA_EUNSUPPORTED, "%s: %lld rows of %lld lanes in one launch (2^32 work-items or more)", op,
                    (long long)rows, (long long)lanes);
    return GA_OK;
}

inline int op_of(int32_t activation) {
    switch (activation) {
    case GA_ACT_SILU: return OP_SILU_MUL;
    case GA_ACT_GELU_TANH: return OP_GELU_TANH_MUL;
    case GA_ACT_GELU_ERF: return OP_GELU_ERF_MUL;
    case GA_ACT_SQUARED_RELU: return OP_SQUARED_RELU;
    default: return -1;
    }
}

}  // namespace ga
