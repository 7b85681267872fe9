// The feed-forward layer's forward pass in bf16 (ga_feed_forward.h).
#include "ga_feed_forward.h"

namespace ga {

hipError_t launch_feed_forward_bf16(int op, const void *x, const void *w_in, const void *w_down, void *y, void *kept,
                                    int32_t rows, int32_t H, int32_t d, const int32_t *live, uint8_t *workspace,
                                    hipStream_t stream) {
    return op == OP_SQUARED_RELU ? forward_as<DT_BF16, false>(op, x, w_in, w_down, y, kept, rows, H, d, live, workspace, stream)
                                 : forward_as<DT_BF16, true>(op, x, w_in, w_down, y, kept, rows, H, d, live, workspace, stream);
}

}  // namespace ga
