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

constexpr int STEP = KPerStep<DT_MX4>::value;

template <int EPI, bool PAIR, int OUT>
hipError_t product(int act, const void *a, const uint8_t *a_scales, const void *w, const uint8_t *w_scales, void *out,
                   void *out2, int32_t rows, int32_t n, int32_t k, const int32_t *live, uint8_t *partial,
                   hipStream_t stream) {
    TileArgs p{};
    p.a = w, p.a_scales = w_scales, p.b = a, p.b_scales = a_scales;
    p.blocks = (int32_t)blocks_of(k), p.a_row = p.b_row = 16 * (int64_t)p.blocks;
    p.F = n, p.T = rows, p.K = p.blocks * MX_BLOCK, p.act = act, p.live = live, p.out = out, p.out2 = out2;
    return launch_product<DT_MX4, false, false, EPI, PAIR, OUT>(p, PAIR, (float *)partial, stream);
}

template <int OUT>
hipError_t plain(const void *a, const uint8_t *a_scales, const void *w, const uint8_t *w_scales, void *out, int32_t rows,
                 int32_t n, int32_t k, const int32_t *live, uint8_t *workspace, hipStream_t stream) {
    return product<EPI_STORE, false, OUT>(0, a, a_scales, w, w_scales, out, nullptr, rows, n, k, live, workspace, stream);
}

template <int OUT>
hipError_t layer_as(int op, const void *x, const void *w_in, const uint8_t *w_in_scales, const void *w_down,
                    const uint8_t *w_down_scales, void *y, int32_t rows, int32_t H, int32_t d, const int32_t *live,
                    uint8_t *workspace, hipStream_t stream) {
    const bool pair = op != OP_SQUARED_RELU;
    const FeedForward4Space at = feed_forward_mxfp4_space(rows, H, d, pair ? 2 : 1);
    uint8_t *xc = workspace + at.x_codes, *xs = workspace + at.x_scales;
    uint8_t *hc = workspace + at.h_codes, *hs = workspace + at.h_scales;
    hipError_t e = launch_mxfp4_quantize(OUT, -1, x, xc, xs, rows, (uint32_t)H, live, stream);
    if (e != hipSuccess) return e;
    // (the epilogue's results have no type)
    e = pair ? product<EPI_QUANTIZE, true, DT_F32>(op, xc, xs, w_in, w_in_scales, hc, hs, rows, d, H, live,
                                                   workspace + at.partial, stream)
             : product<EPI_QUANTIZE, false, DT_F32>(op, xc, xs, w_in, w_in_scales, hc, hs, rows, d, H, live,
                                                    workspace + at.partial, stream);
    if (e != hipSuccess) return e;
    return plain<OUT>(hc, hs, w_down, w_down_scales, y, rows, H, d, live, workspace + at.partial, stream);
}

}  // namespace

size_t mxfp4_product_space(int64_t rows, int64_t n, int64_t k) {
    return align256(plan_product(n, rows, k, false, 0, STEP).partial_bytes);
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
    const size_t a = plan_product(d, rows, H, halves == 2, 0, STEP).partial_bytes, b = plan_product(H, rows, d, false, 0, STEP).partial_bytes;
    s.total = s.partial + align256(a > b ? a : b);
    return s;
}

hipError_t launch_feed_forward_mxfp4(int dtype, int op, const void *x, const void *w_in, const uint8_t *w_in_scales,
                                     const void *w_down, const uint8_t *w_down_scales, void *y, int32_t rows, int32_t H,
                                     int32_t d, const int32_t *live, uint8_t *workspace, hipStream_t stream) {
    switch (dtype) {
    case DT_F16:
        return layer_as<DT_F16>(op, x, w_in, w_in_scales, w_down, w_down_scales, y, rows, H, d, live, workspace, stream);
    case DT_BF16:
        return layer_as<DT_BF16>(op, x, w_in, w_in_scales, w_down, w_down_scales, y, rows, H, d, live, workspace, stream);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace ga
