// The feed-forward layer on the host: how a product runs, workspaces, and the
// choice of the element type's kernels.
#include "ga_device.h"
#include "ga_internal.h"

namespace ga {

namespace {

constexpr size_t align256(size_t n) { return (n + 255) / 256 * 256; }

constexpr int64_t CUS = 256;

// A plan of p.workgroups tiles with k in `splits` slices.
void cut(ProductPlan &p, int64_t F, int64_t T, int64_t steps, int64_t splits, bool halves, int step) {
    const int64_t per = (steps + splits - 1) / splits;
    p.splits = (int)((steps + per - 1) / per);
    p.k_split = (int32_t)(p.splits == 1 ? INT32_MAX : per * step);
    p.workgroups *= p.splits;
    p.partial_bytes = p.splits == 1 ? 0 : (size_t)p.splits * T * F * (halves ? 8 : 4);
}

int64_t steps_of(int64_t K, int step) { return K > 0 ? (K + step - 1) / step : 1; }

// How many slices of at least eight steps bring `tiles` to `slots`.
int64_t slices(int64_t tiles, int64_t steps, int64_t slots) {
    constexpr int64_t LEAST_STEPS = 8, MOST_SLICES = 64;
    int64_t n = tiles > 0 ? slots / tiles : 1;
    n = n < steps / LEAST_STEPS ? n : steps / LEAST_STEPS;
    return n < 1 ? 1 : n > MOST_SLICES ? MOST_SLICES : n;
}

}  // namespace

// Which tiles: those whose rounds on the 256 compute units take the least.  A
// round is a tile on every unit, or two on every unit, and takes as long as it was
// measured to, relative to the largest tile's (bf16, k of 2048); where two are on a
// unit, later rounds follow one another tile by tile, and a little over one round
// takes as long as 1.55 (128 x 192: 512 tiles 54 us, 704 87, 768 78, 896 98, 1408
// 152; 128 x 128: 512 41, 768 69, 1280 105):
//   256 x 256, one a unit                    100  (62 us), 88 with fewer of them
//   128 x 192, two a unit                     87  (54 us), 60 where one is there
//   128 x 128, two stages, two a unit         66  (41 us), 55
//   128 x 128, four stages, one a unit        42  (26 us)
//   128 x 64, four stages, one a unit         30
// So the large tiles are taken where they fill their rounds (bf16 8192 x 4096 x
// 16384 1284 TFLOP/s, 128 x 192 1109, 128 x 128 1102; 4-bit 4096 x 4096 x 16384
// 4370, 128 x 128 3410), 128 x 192 where they don't (12288 x 2 * 768 x 2048 78 us,
// 256 x 256 98, 128 x 128 94; 2560 x 2 * 4096 x 2048 98, 102, 105), 128 x 128 for a
// round of it (1024 x 2 * 4096 x 2048 41 us, 128 x 192 49, 256 x 256 55), and four
// stages, which cover more of the loads' latency, where one tile a unit is all
// there is (2048 x 2048 x 4096 40 us, two stages 58; 1001 x 1032 x 4112 128 x 64 28
// us, 128 x 128 39).  128 x 192 is for 16 bits and contiguous operands: two of them
// with scales do not fit a unit, a row of 192 strided tokens does not divide a load,
// and with A strided the compiler moves its sums about while products are pending.
// For up to 64 tokens the weights are all the bytes there are, and more units bring
// them: 64 x 64 where 256 or fewer are there (bf16 64 x 4096 by 2 * 8192, 256 of
// them, 36.4 us; 128 x 64, 128 of them, 43.4).
// k is cut where part of the card would idle, into slices of at least eight steps
// that fill it (bf16 64 x 8192 by 4096, weights from HBM: 128 x 64 in two slices
// 36.3 us, four 23.1, eight 19.3, sixteen, 512 workgroups, 25.7).
ProductPlan plan_product(int64_t F, int64_t T, int64_t K, bool halves, int strided, int step) {
    const auto tiles = [&](int64_t features, int64_t tokens) {
        const int64_t fw = halves ? features / 2 : features;
        return ((F + fw - 1) / fw) * ((T + tokens - 1) / tokens);
    };
    ProductPlan p{};
    if (strided == 0 && T <= PRODUCT_FEW_TOKENS) {
        p.tile = PRODUCT_FEW;
        p.threads = 512;
        // as launch_stream_tokens has it, with two halves at most (a quarter from nine tokens on)
        p.workgroups = halves || F < PRODUCT_FEW_WIDE ? (F + 7) / 8 : (F + 15) / 16;
        p.splits = 1;
        p.k_split = INT32_MAX;
        return p;
    }
    // a_unit: tiles of it at a time; part: a round of at most one a unit
    const struct {
        int tile, threads;
        int64_t features, tokens, a_unit, round, part;
        bool there;
    } choices[] = {{PRODUCT_BIG, 512, 256, 256, 1, 100, 88, true},
                   {PRODUCT_WIDE, 256, 128, 192, 2, 87, 60, strided == 0 && step == 64},
                   {PRODUCT_MID, 256, 128, 128, 2, 66, 55, true},
                   {PRODUCT_DEEP, 256, 128, 128, 1, 42, 42, true},
                   {PRODUCT_SLIM, 256, 128, 64, 1, 30, 30, true}};
    int64_t least = INT64_MAX;
    for (const auto &c : choices) {
        const int64_t n = tiles(c.features, c.tokens), slots = c.a_unit * CUS, last = n % slots;
        const int64_t cost = c.a_unit == 1 ? n / slots * c.round + (last == 0 ? 0 : c.part)
                             : n <= CUS    ? c.part
                             : n <= slots  ? c.round
                                           : (100 * n > 155 * slots ? 100 * n : 155 * slots) * c.round / (100 * slots);
        if (!c.there || cost >= least) continue;
        least = cost;
        p.tile = c.tile;
        p.threads = c.threads;
        p.workgroups = n;
    }
    if (p.tile == PRODUCT_SLIM && T <= 64 && tiles(64, 64) <= CUS) {
        p.tile = PRODUCT_THIN;
        p.workgroups = tiles(64, 64);
    }
    const int64_t steps = steps_of(K, step);
    cut(p, F, T, steps, p.tile == PRODUCT_SLIM || p.tile == PRODUCT_THIN ? slices(p.workgroups, steps, CUS) : 1, halves, step);
    return p;
}

// Together where the card has room for them, which one of them alone would leave
// idle at its ends, the weights' gradients cut into slices that fill it twice and all
// slices added by one launch (bf16, all four products, rows x H by d: 128 x 512 by
// 1024 30.6 -> 18.8 us, 1024 x 512 by 2048 53.5 -> 39.0, 2048 x 256 by 256 35 -> 23,
// 4096 x 256 by 512 49 -> 33, 1024 x 2048 by 2048, with 512 and 768 tiles, 93.7 ->
// 88.8, 4096 x 1280 by 512, with 1280 and 120, 88.6 -> 74.5; but 1024 x 4096 by 1024,
// with 1024 and 768, 88 -> 92, and 2048 x 2048 by 1024, with 1024 and 384, 86.5 ->
// 88.0).
ThreePlan plan_three(int64_t rows, int64_t H, int64_t d, int64_t zd) {
    const auto tiles = [](int64_t F, int64_t T, int64_t side) { return ((F + side - 1) / side) * ((T + side - 1) / side); };
    ThreePlan p{};
    p.x.tile = PRODUCT_THIN;
    p.in.tile = p.down.tile = PRODUCT_MID;
    p.x.threads = p.in.threads = p.down.threads = 256;
    p.x.workgroups = tiles(H, rows, 64);
    p.in.workgroups = tiles(H, zd, 128);
    p.down.workgroups = tiles(d, H, 128);
    const int64_t w = p.in.workgroups + p.down.workgroups, steps = steps_of(rows, 64);
    const int64_t splits = slices(w, steps, 2 * CUS);
    p.together = rows > 0 && ((p.x.workgroups <= 2 * CUS && w <= 3 * CUS) || (p.x.workgroups <= 5 * CUS && w <= CUS));
    cut(p.x, H, rows, steps_of(zd, 64), slices(p.x.workgroups, steps_of(zd, 64), CUS), false, 64);
    cut(p.in, H, zd, steps, splits, false, 64);
    cut(p.down, d, H, steps, splits, false, 64);
    p.cut_w = p.in.splits > 1;
    return p;
}

FeedForwardSpace feed_forward_space(int64_t rows, int64_t H, int64_t d, int halves) {
    FeedForwardSpace s{};
    s.partial = align256((size_t)rows * d * 2);
    const size_t a = plan_product(d, rows, H, halves == 2, 0, 64).partial_bytes, b = plan_product(H, rows, d, false, 0, 64).partial_bytes;
    s.total = s.partial + align256(a > b ? a : b);
    return s;
}

FeedForwardSpace feed_forward_backward_space(int64_t rows, int64_t H, int64_t d, int halves) {
    FeedForwardSpace s{};
    s.gradient = align256((size_t)rows * d * 2);
    s.partial = s.gradient + align256((size_t)rows * halves * d * 2);
    const size_t parts[4] = {plan_product(d, rows, H, false, 1, 64).partial_bytes,
                             plan_product(H, rows, halves * d, false, 1, 64).partial_bytes,
                             plan_product(H, halves * d, rows, false, 2, 64).partial_bytes,
                             plan_product(d, H, rows, false, 2, 64).partial_bytes};
    const ThreePlan three = plan_three(rows, H, d, halves * d);
    size_t most = three.together ? three.x.partial_bytes + three.in.partial_bytes + three.down.partial_bytes : 0;
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
