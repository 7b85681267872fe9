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
//
// Templates of one element type; each type's forward and backward pass is a
// translation unit of its own.
#pragma once

#include "ga_stream.h"

namespace ga {

namespace {

constexpr bool KC = false, KS = true;  // k contiguous, strided

template <int DT, bool A, bool B, int EPI, bool PAIR>
hipError_t product(const TileArgs &p, bool halves, float *partial, hipStream_t stream) {
    return launch_product<DT, A, B, EPI, PAIR, DT>(p, halves, partial, stream);
}

template <int DT, bool PAIR>
hipError_t forward_as(int act, const void *x, const void *w_in, const void *w_down, void *y, void *kept, int32_t rows,
                      int32_t H, int32_t d, const int32_t *live, uint8_t *workspace, hipStream_t stream) {
    const FeedForwardSpace at = feed_forward_space(rows, H, d, PAIR ? 2 : 1);
    void *h = workspace + at.hidden;
    float *partial = (float *)(workspace + at.partial);
    TileArgs p{};
    p.a = w_in, p.a_row = 2 * (int64_t)H, p.b = x, p.b_row = 2 * (int64_t)H;
    p.F = d, p.T = rows, p.K = H, p.act = act, p.live = live, p.out = h, p.out2 = kept;
    hipError_t e = product<DT, KC, KC, EPI_GATED, PAIR>(p, PAIR, partial, stream);
    if (e != hipSuccess) return e;
    p = TileArgs{};
    p.a = w_down, p.a_row = 2 * (int64_t)d, p.b = h, p.b_row = 2 * (int64_t)d;
    p.F = H, p.T = rows, p.K = d, p.live = live, p.out = y;
    return product<DT, KC, KC, EPI_STORE, false>(p, false, partial, stream);
}

template <int DT, bool PAIR>
hipError_t backward_as(int act, const void *dy, const void *x, const void *kept, const void *w_in, const void *w_down,
                       void *dx, void *dw_in, void *dw_down, int32_t rows, int32_t H, int32_t d, const int32_t *live,
                       uint8_t *workspace, hipStream_t stream) {
    const int32_t zd = PAIR ? 2 * d : d;
    const FeedForwardSpace at = feed_forward_backward_space(rows, H, d, PAIR ? 2 : 1);
    void *h = workspace + at.hidden, *dz = workspace + at.gradient;
    float *partial = (float *)(workspace + at.partial);
    TileArgs p{};
    if (rows > 0) {
        p.a = w_down, p.a_row = 2 * (int64_t)d, p.b = dy, p.b_row = 2 * (int64_t)H;
        p.F = d, p.T = rows, p.K = H, p.act = act, p.live = live, p.out = dz, p.out2 = h, p.z = kept;
        const hipError_t e = product<DT, KS, KC, EPI_BACKWARD, PAIR>(p, false, partial, stream);
        if (e != hipSuccess) return e;
    }
    TileArgs px{}, pi{}, pd{};
    px.a = w_in, px.a_row = 2 * (int64_t)H, px.b = dz, px.b_row = 2 * (int64_t)zd;
    px.F = H, px.T = rows, px.K = zd, px.live = live, px.out = dx;
    pi.a = x, pi.a_row = 2 * (int64_t)H, pi.b = dz, pi.b_row = 2 * (int64_t)zd;
    pi.F = H, pi.T = zd, pi.K = rows, pi.live = live, pi.out = dw_in;
    pd.a = h, pd.a_row = 2 * (int64_t)d, pd.b = dy, pd.b_row = 2 * (int64_t)H;
    pd.F = d, pd.T = H, pd.K = rows, pd.live = live, pd.out = dw_down;
    const ThreePlan three = plan_three(rows, H, d, zd);
    if (three.together) return launch_three<DT>(px, pi, pd, three, partial, stream);
    hipError_t e = rows > 0 ? product<DT, KS, KC, EPI_STORE, false>(px, false, partial, stream) : hipSuccess;
    if (e == hipSuccess) e = product<DT, KS, KS, EPI_STORE, false>(pi, false, partial, stream);
    return e != hipSuccess ? e : product<DT, KS, KS, EPI_STORE, false>(pd, false, partial, stream);
}

}  // namespace

}  // namespace ga
