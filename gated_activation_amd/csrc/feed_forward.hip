// The feed-forward layer on the host: how a product runs, workspaces, and the
// choice of the element type's kernels.
#include "ga_device.h"
#include "ga_internal.h"

namespace ga {

namespace {

constexpr size_t align256(size_t n) { return (n + 255) / 256 * 256; }

}  // namespace

// Which tiles, by how many workgroups they make for the 256 compute units.
//   256 x 256, one workgroup a unit, where their last round is at least 0.76 full:
//     128 x 128, two a unit, run at 0.75 to 0.78 of their rate (bf16 8192 x 4096 x
//     16384 1284 and 974 TFLOP/s; 4-bit 4096 x 4096 x 16384 4370 and 3410), and at
//     288 and 384 large tiles (bf16 12288 x 2 * 768 x 2048 and 12288 x 2048 x 768)
//     take 86 us against 96 and 43 against 45.
//   128 x 128 with two stages, two a unit, where there are more than 256 of them
//     (bf16 4112 x 1032 x 1001 20.4 us; four stages, one a unit, 26.9).
//   128 x 64 or else 128 x 128 with four stages, one a unit, where 256 or fewer are
//     there and the loads' latency counts (bf16 1001 x 1032 x 4112 27.2 us, 128 x
//     128 37.4, with two stages 49.4; 1032 x 2056 x 1001 128 x 128 13.9, 128 x 64,
//     289 of them, 19.8).
//   64 x 64 for up to 64 tokens, where 256 or fewer are there: the weights are all
//     the bytes there are, and more units bring them (bf16 64 x 4096 by 2 * 8192,
//     256 of them, 36.4 us; 128 x 64, 128 of them, 43.4).
// k is cut where part of the card would idle, into slices of at least eight steps
// that fill it (bf16 64 x 8192 by 4096, weights from HBM: 128 x 64 in two slices
// 36.3 us, four 23.1, eight 19.3, sixteen, 512 workgroups, 25.7).
ProductPlan plan_product(int64_t F, int64_t T, int64_t K, bool halves, bool contiguous, int step) {
    constexpr int64_t CUS = 256, LEAST_STEPS = 8, MOST_SLICES = 64;
    const int64_t steps = K > 0 ? (K + step - 1) / step : 1;
    const auto tiles = [&](int64_t features, int64_t tokens) {
        const int64_t fw = halves ? features / 2 : features;
        return ((F + fw - 1) / fw) * ((T + tokens - 1) / tokens);
    };
    const int64_t big = tiles(256, 256), mid = tiles(128, 128), slim = tiles(128, 64),
                  thin = tiles(64, 64);
    int64_t splits = 1;
    ProductPlan p{};
    if (contiguous && T <= PRODUCT_FEW_TOKENS) {
        p.tile = PRODUCT_FEW;
        p.workgroups = (F + 7) / 8;  // at most
    } else if (100 * big >= 76 * CUS * ((big + CUS - 1) / CUS)) {
        p.tile = PRODUCT_BIG;
        p.workgroups = big;
    } else if (mid > CUS) {
        p.tile = PRODUCT_MID;
        p.workgroups = mid;
    } else if (slim > CUS) {
        p.tile = PRODUCT_DEEP;
        p.workgroups = mid;
    } else {
        p.tile = T <= 64 && thin <= CUS ? PRODUCT_THIN : PRODUCT_SLIM;
        p.workgroups = p.tile == PRODUCT_THIN ? thin : slim;
        splits = p.workgroups > 0 ? CUS / p.workgroups : 1;
        splits = splits < steps / LEAST_STEPS ? splits : steps / LEAST_STEPS;
        splits = splits < 1 ? 1 : splits > MOST_SLICES ? MOST_SLICES : splits;
    }
    const int64_t per = (steps + splits - 1) / splits;
    p.splits = (int)((steps + per - 1) / per);
    p.k_split = (int32_t)(p.splits == 1 ? INT32_MAX : per * step);
    p.workgroups *= p.splits;
    p.partial_bytes = p.splits == 1 ? 0 : (size_t)p.splits * T * F * (halves ? 8 : 4);
    return p;
}

FeedForwardSpace feed_forward_space(int64_t rows, int64_t H, int64_t d, int halves) {
    FeedForwardSpace s{};
    s.partial = align256((size_t)rows * d * 2);
    const size_t a = plan_product(d, rows, H, halves == 2, true, 64).partial_bytes, b = plan_product(H, rows, d, false, true, 64).partial_bytes;
    s.total = s.partial + align256(a > b ? a : b);
    return s;
}

FeedForwardSpace feed_forward_backward_space(int64_t rows, int64_t H, int64_t d, int halves) {
    FeedForwardSpace s{};
    s.gradient = align256((size_t)rows * d * 2);
    s.partial = s.gradient + align256((size_t)rows * halves * d * 2);
    const size_t parts[4] = {plan_product(d, rows, H, false, false, 64).partial_bytes,
                             plan_product(H, rows, halves * d, false, false, 64).partial_bytes,
                             plan_product(H, halves * d, rows, false, false, 64).partial_bytes,
                             plan_product(d, H, rows, false, false, 64).partial_bytes};
    size_t most = 0;
    for (size_t b : parts) most = b > most ? b : most;
    s.total = s.partial + align256(most);
    return s;
}

hipError_t launch_feed_forward(int dtype, int op, const void *x, const void *w_in, const void *w_down, void *y, void *kept,
                               int32_t rows, int32_t H, int32_t d, const int32_t *live, uint8_t *workspace,
                               hipStream_t stream) {
    switch (dtype) {
    case DT_F16: return launch_feed_forward_f16(op, x, w_in, w_down, y, kept, rows, H, d, live, workspace, stream);
    case DT_BF16: return launch_feed_forward_bf16(op, x, w_in, w_down, y, kept, rows, H, d, live, workspace, stream);
    default: return hipErrorInvalidValue;
    }
}

hipError_t launch_feed_forward_backward(int dtype, int op, const void *dy, const void *x, const void *kept,
                                        const void *w_in, const void *w_down, void *dx, void *dw_in, void *dw_down,
                                        int32_t rows, int32_t H, int32_t d, const int32_t *live, uint8_t *workspace,
                                        hipStream_t stream) {
    switch (dtype) {
    case DT_F16:
        return launch_feed_forward_backward_f16(op, dy, x, kept, w_in, w_down, dx, dw_in, dw_down, rows, H, d, live, workspace, stream);
    case DT_BF16:
        return launch_feed_forward_backward_bf16(op, dy, x, kept, w_in, w_down, dx, dw_in, dw_down, rows, H, d, live, workspace, stream);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace ga
