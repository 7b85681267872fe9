// The gated feed-forward layer in 16 bits, gfx950: forward and backward.
//
//   z = x w_in^T = gate | up        w_in [2d, H] (gate rows, up rows; squared ReLU [d, H])
//   h = act(gate) up                rounded to the type
//   y = h w_down^T                  w_down [H, d]
//
// Forward, two products: the first forms gate and up of the same features in one
// tile and activates them in its epilogue, so z goes to memory only where it is
// kept; the second is plain.  Backward, from dy, x and the kept z, four:
//
//   dh = dy w_down, whose epilogue reads z and leaves dz and h (dh itself is
//        never stored)
//   dx = dz w_in,  dw_in = dz^T x,  dw_down = dy^T h
//
// h and dz are rounded to the type, as the matrix cores take them; dh, the
// activation and its slope stay in fp32.
#include "ga_stream.h"

namespace ga {

namespace {

constexpr size_t align256(size_t n) { return (n + 255) / 256 * 256; }

constexpr bool KC = false, KS = true;  // k contiguous, strided
template <int DT, bool A, bool B> using Big = Tile<DT, A, B, 2, 4, 8, 4>;
template <int DT, bool A, bool B> using Mid = Tile<DT, A, B, 2, 2, 4, 4>;

template <int DT, bool A, bool B, int EPI, int ACT>
hipError_t product(const TileArgs &p, bool halves, float *partial, hipStream_t stream) {
    const ProductPlan plan = plan_product(p.F, p.T, p.K, halves, !A && !B, KPerStep<DT>::value);
    return launch_product<Big<DT, A, B>, Mid<DT, A, B>, EPI, ACT, DT>(p, plan, halves, partial, stream);
}

template <int DT, int ACT>
hipError_t forward_as(const void *x, const void *w_in, const void *w_down, void *y, void *kept, int32_t rows, int32_t H,
                      int32_t d, const int32_t *live, uint8_t *workspace, hipStream_t stream) {
    constexpr bool GATED = act_gated<ACT>();
    const FeedForwardSpace at = feed_forward_space(rows, H, d, GATED ? 2 : 1);
    void *h = workspace + at.hidden;
    float *partial = (float *)(workspace + at.partial);
    TileArgs p{};
    p.a = w_in, p.a_row = 2 * (int64_t)H, p.b = x, p.b_row = 2 * (int64_t)H;
    p.F = d, p.T = rows, p.K = H, p.live = live, p.out = h, p.out2 = kept;
    hipError_t e = product<DT, KC, KC, EPI_GATED, ACT>(p, GATED, partial, stream);
    if (e != hipSuccess) return e;
    p = TileArgs{};
    p.a = w_down, p.a_row = 2 * (int64_t)d, p.b = h, p.b_row = 2 * (int64_t)d;
    p.F = H, p.T = rows, p.K = d, p.live = live, p.out = y;
    return product<DT, KC, KC, EPI_STORE, OP_SQUARED_RELU>(p, false, partial, stream);
}

template <int DT, int ACT>
hipError_t backward_as(const void *dy, const void *x, const void *kept, const void *w_in, const void *w_down, void *dx,
                       void *dw_in, void *dw_down, int32_t rows, int32_t H, int32_t d, const int32_t *live,
                       uint8_t *workspace, hipStream_t stream) {
    const int32_t zd = act_gated<ACT>() ? 2 * d : d;
    const FeedForwardSpace at = feed_forward_backward_space(rows, H, d, zd / d);
    void *h = workspace + at.hidden, *dz = workspace + at.gradient;
    float *partial = (float *)(workspace + at.partial);
    hipError_t e = hipSuccess;
    TileArgs p{};
    if (rows > 0) {
        p.a = w_down, p.a_row = 2 * (int64_t)d, p.b = dy, p.b_row = 2 * (int64_t)H;
        p.F = d, p.T = rows, p.K = H, p.live = live, p.out = dz, p.out2 = h, p.z = kept;
        e = product<DT, KS, KC, EPI_BACKWARD, ACT>(p, false, partial, stream);
        if (e != hipSuccess) return e;
        p = TileArgs{};
        p.a = w_in, p.a_row = 2 * (int64_t)H, p.b = dz, p.b_row = 2 * (int64_t)zd;
        p.F = H, p.T = rows, p.K = zd, p.live = live, p.out = dx;
        e = product<DT, KS, KC, EPI_STORE, OP_SQUARED_RELU>(p, false, partial, stream);
        if (e != hipSuccess) return e;
    }
    p = TileArgs{};
    p.a = x, p.a_row = 2 * (int64_t)H, p.b = dz, p.b_row = 2 * (int64_t)zd;
    p.F = H, p.T = zd, p.K = rows, p.live = live, p.out = dw_in;
    e = product<DT, KS, KS, EPI_STORE, OP_SQUARED_RELU>(p, false, partial, stream);
    if (e != hipSuccess) return e;
    p = TileArgs{};
    p.a = h, p.a_row = 2 * (int64_t)d, p.b = dy, p.b_row = 2 * (int64_t)H;
    p.F = d, p.T = H, p.K = rows, p.live = live, p.out = dw_down;
    return product<DT, KS, KS, EPI_STORE, OP_SQUARED_RELU>(p, false, partial, stream);
}

template <int DT>
hipError_t forward_op(int op, const void *x, const void *w_in, const void *w_down, void *y, void *kept, int32_t rows,
                      int32_t H, int32_t d, const int32_t *live, uint8_t *workspace, hipStream_t stream) {
    switch (op) {
    case OP_SILU_MUL: return forward_as<DT, OP_SILU_MUL>(x, w_in, w_down, y, kept, rows, H, d, live, workspace, stream);
    case OP_GELU_TANH_MUL:
        return forward_as<DT, OP_GELU_TANH_MUL>(x, w_in, w_down, y, kept, rows, H, d, live, workspace, stream);
    case OP_GELU_ERF_MUL:
        return forward_as<DT, OP_GELU_ERF_MUL>(x, w_in, w_down, y, kept, rows, H, d, live, workspace, stream);
    case OP_SQUARED_RELU:
        return forward_as<DT, OP_SQUARED_RELU>(x, w_in, w_down, y, kept, rows, H, d, live, workspace, stream);
    default: return hipErrorInvalidValue;
    }
}

template <int DT>
hipError_t backward_op(int op, const void *dy, const void *x, const void *kept, const void *w_in, const void *w_down,
                       void *dx, void *dw_in, void *dw_down, int32_t rows, int32_t H, int32_t d, const int32_t *live,
                       uint8_t *workspace, hipStream_t stream) {
    switch (op) {
    case OP_SILU_MUL:
        return backward_as<DT, OP_SILU_MUL>(dy, x, kept, w_in, w_down, dx, dw_in, dw_down, rows, H, d, live, workspace, stream);
    case OP_GELU_TANH_MUL:
        return backward_as<DT, OP_GELU_TANH_MUL>(dy, x, kept, w_in, w_down, dx, dw_in, dw_down, rows, H, d, live, workspace,
                                                 stream);
    case OP_GELU_ERF_MUL:
        return backward_as<DT, OP_GELU_ERF_MUL>(dy, x, kept, w_in, w_down, dx, dw_in, dw_down, rows, H, d, live, workspace,
                                                stream);
    case OP_SQUARED_RELU:
        return backward_as<DT, OP_SQUARED_RELU>(dy, x, kept, w_in, w_down, dx, dw_in, dw_down, rows, H, d, live, workspace,
                                                stream);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace

// Tiles of 256 x 256 where they fill the card, else of 128 x 128 with k in
// slices until two workgroups a compute unit are there or a slice is short.
ProductPlan plan_product(int64_t F, int64_t T, int64_t K, bool halves, bool contiguous, int step) {
    constexpr int64_t CUS = 256, LEAST_STEPS = 8;
    const auto tiles = [&](int64_t side) {
        const int64_t fw = halves ? side / 2 : side;
        return ((F + fw - 1) / fw) * ((T + side - 1) / side);
    };
    ProductPlan p{PRODUCT_BIG, 1, 0, tiles(256), 0};
    const int64_t steps = K > 0 ? (K + step - 1) / step : 1;
    int64_t splits = 1;
    if (contiguous && T <= PRODUCT_FEW_TOKENS) {
        p.tile = PRODUCT_FEW;
        p.workgroups = (F + 7) / 8;  // at most
    } else if (p.workgroups < CUS * 3 / 4) {
        p.tile = PRODUCT_MID;
        p.workgroups = tiles(128);
        splits = 2 * CUS / (p.workgroups > 0 ? p.workgroups : 1);
        splits = splits < steps / LEAST_STEPS ? splits : steps / LEAST_STEPS;
        splits = splits < 1 ? 1 : splits > 64 ? 64 : splits;
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
    case DT_F16: return forward_op<DT_F16>(op, x, w_in, w_down, y, kept, rows, H, d, live, workspace, stream);
    case DT_BF16: return forward_op<DT_BF16>(op, x, w_in, w_down, y, kept, rows, H, d, live, workspace, stream);
    default: return hipErrorInvalidValue;
    }
}

hipError_t launch_feed_forward_backward(int dtype, int op, const void *dy, const void *x, const void *kept,
                                        const void *w_in, const void *w_down, void *dx, void *dw_in, void *dw_down,
                                        int32_t rows, int32_t H, int32_t d, const int32_t *live, uint8_t *workspace,
                                        hipStream_t stream) {
    switch (dtype) {
    case DT_F16:
        return backward_op<DT_F16>(op, dy, x, kept, w_in, w_down, dx, dw_in, dw_down, rows, H, d, live, workspace, stream);
    case DT_BF16:
        return backward_op<DT_BF16>(op, dy, x, kept, w_in, w_down, dx, dw_in, dw_down, rows, H, d, live, workspace, stream);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace ga
