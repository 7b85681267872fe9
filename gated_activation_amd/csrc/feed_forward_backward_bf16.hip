// The feed-forward layer's backward pass in bf16 (ga_feed_forward.h).
#include "ga_feed_forward.h"

namespace ga {

hipError_t launch_feed_forward_backward_bf16(int op, const void *dy, const void *x, const void *kept, const void *w_in,
                                             const void *w_down, void *dx, void *dw_in, void *dw_down, int32_t rows,
                                             int32_t H, int32_t d, const int32_t *live, uint8_t *workspace,
                                             hipStream_t stream) {
    return op == OP_SQUARED_RELU
               ? backward_as<DT_BF16, false>(op, dy, x, kept, w_in, w_down, dx, dw_in, dw_down, rows, H, d, live, workspace, stream)
               : backward_as<DT_BF16, true>(op, dy, x, kept, w_in, w_down, dx, dw_in, dw_down, rows, H, d, live, workspace, stream);
}

}  // namespace ga
