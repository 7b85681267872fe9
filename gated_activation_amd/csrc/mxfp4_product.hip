// Products of microscaled 4-bit arrays, gfx950, and the feed-forward layer on
// them.
//
//   out[t, f] = sum over k of a[t, k] w[f, k]    of the values that codes and
//                                                scales stand for, fp32 sums
//   layer: x is quantised, z = q(x) w_in^T = gate | up stays in fp32, the first
//          product's epilogue activates and quantises h = act(gate) up, and
//          y = q(h) w_down^T
#include "ga_stream.h"

namespace ga {

namespace {

constexpr size_t align256(size_t n) { return (n + 255) / 256 * 256; }
constexpr int64_t blocks_of(int64_t d) { return (d + MX_BLOCK - 1) / MX_BLOCK; }

using Big = Tile<DT_MX4, false, false, 2, 4, 8, 4>;
using Mid = Tile<DT_MX4, false, false, 2, 2, 4, 4>;
constexpr int STEP = KPerStep<DT_MX4>::value;

template <int EPI, int ACT, int OUT>
hipError_t product(const void *a, const uint8_t *a_scales, const void *w, const uint8_t *w_scales, void *out, void *out2,
                   int32_t rows, int32_t n, int32_t k, bool halves, const int32_t *live, float *partial,
                   hipStream_t stream) {
    TileArgs p{};
    p.a = w, p.a_scales = w_scales, p.b = a, p.b_scales = a_scales;
    p.blocks = (int32_t)blocks_of(k), p.a_row = p.b_row = 16 * (int64_t)p.blocks;
    p.F = n, p.T = rows, p.K = p.blocks * MX_BLOCK, p.live = live, p.out = out, p.out2 = out2;
    return launch_product<Big, Mid, EPI, ACT, OUT>(p, plan_product(n, rows, k, halves, true, STEP), halves, partial, stream);
}

template <int OUT>
hipError_t plain(const void *a, const uint8_t *a_scales, const void *w, const uint8_t *w_scales, void *out, int32_t rows,
                 int32_t n, int32_t k, const int32_t *live, uint8_t *workspace, hipStream_t stream) {
    return product<EPI_STORE, OP_SQUARED_RELU, OUT>(a, a_scales, w, w_scales, out, nullptr, rows, n, k, false, live,
                                                    (float *)workspace, stream);
}

template <int OUT, int ACT>
hipError_t layer_as(const void *x, const void *w_in, const uint8_t *w_in_scales, const void *w_down,
                    const uint8_t *w_down_scales, void *y, int32_t rows, int32_t H, int32_t d, const int32_t *live,
                    uint8_t *workspace, hipStream_t stream) {
    constexpr bool GATED = act_gated<ACT>();
    const FeedForward4Space at = feed_forward_mxfp4_space(rows, H, d, GATED ? 2 : 1);
    uint8_t *xc = workspace + at.x_codes, *xs = workspace + at.x_scales;
    uint8_t *hc = workspace + at.h_codes, *hs = workspace + at.h_scales;
    hipError_t e = launch_mxfp4_quantize(OUT, -1, x, xc, xs, rows, (uint32_t)H, live, stream);
    if (e != hipSuccess) return e;
    e = product<EPI_QUANTIZE, ACT, OUT>(xc, xs, w_in, w_in_scales, hc, hs, rows, d, H, GATED, live,
                                        (float *)(workspace + at.partial), stream);
    if (e != hipSuccess) return e;
    return plain<OUT>(hc, hs, w_down, w_down_scales, y, rows, H, d, live, workspace + at.partial, stream);
}

template <int OUT>
hipError_t layer_op(int op, const void *x, const void *w_in, const uint8_t *w_in_scales, const void *w_down,
                    const uint8_t *w_down_scales, void *y, int32_t rows, int32_t H, int32_t d, const int32_t *live,
                    uint8_t *ws, hipStream_t stream) {
    switch (op) {
    case OP_SILU_MUL:
        return layer_as<OUT, OP_SILU_MUL>(x, w_in, w_in_scales, w_down, w_down_scales, y, rows, H, d, live, ws, stream);
    case OP_GELU_TANH_MUL:
        return layer_as<OUT, OP_GELU_TANH_MUL>(x, w_in, w_in_scales, w_down, w_down_scales, y, rows, H, d, live, ws, stream);
    case OP_GELU_ERF_MUL:
        return layer_as<OUT, OP_GELU_ERF_MUL>(x, w_in, w_in_scales, w_down, w_down_scales, y, rows, H, d, live, ws, stream);
    case OP_SQUARED_RELU:
        return layer_as<OUT, OP_SQUARED_RELU>(x, w_in, w_in_scales, w_down, w_down_scales, y, rows, H, d, live, ws, stream);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace

size_t mxfp4_product_space(int64_t rows, int64_t n, int64_t k) {
    return align256(plan_product(n, rows, k, false, true, STEP).partial_bytes);
}

hipError_t launch_mxfp4_product(int dtype, const void *a, const uint8_t *a_scales, const void *w, const uint8_t *w_scales,
                                void *out, int32_t rows, int32_t n, int32_t k, const int32_t *live, uint8_t *workspace,
                                hipStream_t stream) {
    switch (dtype) {
    case DT_F32: return plain<DT_F32>(a, a_scales, w, w_scales, out, rows, n, k, live, workspace, stream);
    case DT_F16: return plain<DT_F16>(a, a_scales, w, w_scales, out, rows, n, k, live, workspace, stream);
    case DT_BF16: return plain<DT_BF16>(a, a_scales, w, w_scales, out, rows, n, k, live, workspace, stream);
    default: return hipErrorInvalidValue;
    }
}

FeedForward4Space feed_forward_mxfp4_space(int64_t rows, int64_t H, int64_t d, int halves) {
    FeedForward4Space s{};
    s.x_scales = align256((size_t)rows * blocks_of(H) * 16);
    s.h_codes = s.x_scales + align256((size_t)rows * blocks_of(H));
    s.h_scales = s.h_codes + align256((size_t)rows * blocks_of(d) * 16);
    s.partial = s.h_scales + align256((size_t)rows * blocks_of(d));
    const size_t a = plan_product(d, rows, H, halves == 2, true, STEP).partial_bytes, b = plan_product(H, rows, d, false, true, STEP).partial_bytes;
    s.total = s.partial + align256(a > b ? a : b);
    return s;
}

hipError_t launch_feed_forward_mxfp4(int dtype, int op, const void *x, const void *w_in, const uint8_t *w_in_scales,
                                     const void *w_down, const uint8_t *w_down_scales, void *y, int32_t rows, int32_t H,
                                     int32_t d, const int32_t *live, uint8_t *workspace, hipStream_t stream) {
    switch (dtype) {
    case DT_F16:
        return layer_op<DT_F16>(op, x, w_in, w_in_scales, w_down, w_down_scales, y, rows, H, d, live, workspace, stream);
    case DT_BF16:
        return layer_op<DT_BF16>(op, x, w_in, w_in_scales, w_down, w_down_scales, y, rows, H, d, live, workspace, stream);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace ga
