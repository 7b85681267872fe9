// Activation checkpoints in 8 bits and the elementwise activations' training
// pair, gfx950.
//
//   store    x [rows, d] -> codes, scales (block_encode in ga_train.h)
//   restore  codes, scales -> x [rows, d]
//   forward  the gated activation of x [rows, 2d] (squared ReLU: x [rows, d])
//            with the codes of x written in the same pass over it
//   backward the gradient of x from dout and x, or from dout and the codes:
//            dgate = dout up f'(gate), dup = dout f(gate)
//
// All four are bound by HBM: every input byte is read once and every output
// byte written once.  Work is numbered in blocks of 128 values of one row's
// half; 16 consecutive lanes hold a block, eight values each, so its maximum
// is four DPP steps.  A lane holds the octets of both halves at the same
// column.  The live count is read on the device and the grid comes from the
// capacity alone, as in the forward-only kernels.
//
// Measured (medians of a kernel trace, bf16 unless said): silu forward with codes,
// 12288 live rows of 768 (76 MB) 16.6 us, 4.6 TB/s, its backward from codes
// 14.8 us, 5.1 TB/s; forward and backward of 8192 x 4096 (271 MB each) gelu, erf
// 46.2 and 43.4 us, tanh 45.8 and 43.7 us (5.9 and 6.2 TB/s), squared ReLU (169 MB)
// 30.8 and 27.6 us, 5.5 and 6.1 TB/s, in fp32 (472 MB) silu 88.8 and 87.0 us, gelu
// (erf) 89.8 and 88.2 us, 5.3 TB/s; store 4096 x 16384 (203 MB) 34.0 us, 6.0 TB/s,
// restore 34.6 us, 5.9 TB/s; gelu backward from x, 1023 x 4099 fp16 (42 MB, rows off
// 16-byte alignment) 10.4 us, 4.0 TB/s.
#include "ga_internal.h"
#include "ga_train.h"

namespace ga {

namespace {

constexpr int FLAT_BLOCK = 256;
constexpr uint32_t FLAT_GROUPS = FLAT_BLOCK / 16;
constexpr int OP_NONE = -1;

// Blocks a 16-lane group has in flight.  Two where a block is one 16-byte load
// a lane (4096 rows of 16384, bf16, fastest of a trace: store 31.8 us, 36.3 with
// one, 32.4 with four); one where it is more (gelu forward, 8192 rows of 4096,
// bf16: 44.0 us, 47.2 with two).
template <int DT> constexpr int unroll_of(int halves) { return DT != DT_F32 && halves == 1 ? 2 : 1; }

template <int ACT>
__device__ __forceinline__ float act_value(float x) {
    if constexpr (ACT == OP_SILU_MUL) return silu(x);
    else if constexpr (ACT == OP_GELU_TANH_MUL) return gelu_tanh(x);
    else if constexpr (ACT == OP_GELU_ERF_MUL) return gelu_erf(x);
    else {
        const float r = __builtin_fmaxf(x, 0.0f);
        return r * r;
    }
}

template <int ACT>
__device__ __forceinline__ void act_slope(float x, float &f, float &df) {
    if constexpr (ACT == OP_SILU_MUL) silu_slope(x, f, df);
    else if constexpr (ACT == OP_GELU_TANH_MUL) gelu_tanh_slope(x, f, df);
    else gelu_erf_slope(x, f, df);
}

// One half's block: codes and, from the block's first lane, its scale.
template <int DT>
__device__ __forceinline__ void keep_block(const float (&x)[8], uint8_t *codes, float *scale_at, int n, bool first) {
    float scale;
    const uint2 c = block_encode<code_of<DT>(), false>(x, scale);
    codes_store(codes, c, n);
    if (first) *scale_at = scale;
}

// forward with checkpoint (ACT >= 0) and plain store (OP_NONE: no out, one half)
template <int DT, int ACT, bool TINY>
__global__ __launch_bounds__(FLAT_BLOCK) void store_kernel(
    const typename Elem<DT>::storage *__restrict__ in, typename Elem<DT>::storage *__restrict__ out,
    uint8_t *__restrict__ codes, float *__restrict__ scales, int32_t rows_cap, uint32_t d, uint32_t nb, FastDiv by_nb,
    const int32_t *__restrict__ live) {
    constexpr bool GATED = ACT >= 0 && ACT != OP_SQUARED_RELU;
    constexpr int H = GATED ? 2 : 1, UNROLL = unroll_of<DT>(H);
    const uint32_t rows = live != nullptr ? (uint32_t)clamp_live(live, rows_cap) : (uint32_t)rows_cap;
    const uint32_t total = rows * nb;
    const uint32_t step = gridDim.x * FLAT_GROUPS * UNROLL;
    const uint32_t l8 = (threadIdx.x & 15) * 8;
    // a block's row and this lane's column; past the last block that one, unused
    auto place = [&](uint32_t b, uint32_t &row, uint32_t &col, int &n) {
        b = b < total ? b : total - 1;
        row = by_nb(b);
        col = (b - row * nb) * BLOCK8 + l8;
        n = (int)d - (int)col;
    };
    for (uint32_t base = blockIdx.x * FLAT_GROUPS * UNROLL + (threadIdx.x >> 4); base < total; base += step) {
        Oct<DT> g[UNROLL], u[UNROLL];
        uint32_t row[UNROLL], col[UNROLL];
        int n[UNROLL];
#pragma unroll
        for (int k = 0; k < UNROLL; ++k) {
            const uint32_t b = base + k * FLAT_GROUPS;
            place(b, row[k], col[k], n[k]);
            const typename Elem<DT>::storage *x = in + (size_t)row[k] * (H * d);
            oct_fetch<DT, TINY>(g[k], x, (int)col[k], (int)d);
            if constexpr (GATED) oct_fetch<DT, TINY>(u[k], x + d, (int)col[k], (int)d);
        }
#pragma unroll
        for (int k = 0; k < UNROLL; ++k) {
            const uint32_t b = base + k * FLAT_GROUPS;
            if (b >= total) continue;
            float x[8], y[8];
            oct_trim<DT, TINY>(g[k], (int)col[k], (int)d);
            oct_unpack<DT>(g[k], x);
            const size_t at = (size_t)row[k] * (H * d) + col[k];
            const size_t block = (size_t)row[k] * (H * nb) + (b - row[k] * nb);
            keep_block<DT>(x, codes + at, scales + block, n[k], l8 == 0);
            if constexpr (ACT >= 0) {
#pragma unroll
                for (int e = 0; e < 8; ++e) y[e] = act_value<ACT>(x[e]);
                if constexpr (GATED) {
                    float up[8];
                    oct_trim<DT, TINY>(u[k], (int)col[k], (int)d);
                    oct_unpack<DT>(u[k], up);
                    keep_block<DT>(up, codes + at + d, scales + block + nb, n[k], l8 == 0);
#pragma unroll
                    for (int e = 0; e < 8; ++e) y[e] *= up[e];
                }
                oct_store<DT>(out + (size_t)row[k] * d + col[k], y, n[k]);
            }
        }
    }
}

// codes * scale; `stats` (nullable): two floats for every `halves` rows, the
// first of which is added to the first half (what the codes are relative to).
template <int DT, bool TINY>
__global__ __launch_bounds__(FLAT_BLOCK) void restore_kernel(
    const uint8_t *__restrict__ codes, const float *__restrict__ scales, const float *__restrict__ stats,
    typename Elem<DT>::storage *__restrict__ out, int32_t rows_cap, uint32_t d, uint32_t nb, FastDiv by_nb,
    int32_t halves, const int32_t *__restrict__ live) {
    constexpr int UNROLL = unroll_of<DT>(1);
    const uint32_t rows = (live != nullptr ? (uint32_t)clamp_live(live, rows_cap) : (uint32_t)rows_cap) * halves;
    const uint32_t total = rows * nb;
    const uint32_t step = gridDim.x * FLAT_GROUPS * UNROLL;
    const uint32_t l8 = (threadIdx.x & 15) * 8;
    // a block's row and this lane's column; past the last block that one, unused
    auto place = [&](uint32_t b, uint32_t &row, uint32_t &col, int &n) {
        b = b < total ? b : total - 1;
        row = by_nb(b);
        col = (b - row * nb) * BLOCK8 + l8;
        n = (int)d - (int)col;
    };
    for (uint32_t base = blockIdx.x * FLAT_GROUPS * UNROLL + (threadIdx.x >> 4); base < total; base += step) {
        uint2 c[UNROLL];
        float scale[UNROLL], shift[UNROLL];
        uint32_t row[UNROLL], col[UNROLL];
        int n[UNROLL];
#pragma unroll
        for (int k = 0; k < UNROLL; ++k) {
            const uint32_t b = base + k * FLAT_GROUPS;
            place(b, row[k], col[k], n[k]);
            scale[k] = scales[b < total ? b : total - 1];
            c[k] = codes_fetch<TINY>(codes + (size_t)row[k] * d, (int)col[k], (int)d);
            shift[k] = 0.0f;
            if (stats != nullptr && (halves == 1 || (row[k] & 1) == 0))
                shift[k] = stats[2 * (size_t)(halves == 1 ? row[k] : row[k] >> 1)];
        }
#pragma unroll
        for (int k = 0; k < UNROLL; ++k) {
            if (base + k * FLAT_GROUPS >= total) continue;
            float x[8];
            codes_trim<TINY>(c[k], (int)col[k], (int)d);
            block_decode(c[k], scale[k], x);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] += shift[k];
            oct_store<DT>(out + (size_t)row[k] * d + col[k], x, n[k]);
        }
    }
}

// KEPT: gate (and up) restored from the codes; else read from x.
template <int DT, int ACT, bool KEPT, bool TINY>
__global__ __launch_bounds__(FLAT_BLOCK) void backward_kernel(
    const typename Elem<DT>::storage *__restrict__ dout, const typename Elem<DT>::storage *__restrict__ in,
    const uint8_t *__restrict__ codes, const float *__restrict__ scales, typename Elem<DT>::storage *__restrict__ dx,
    int32_t rows_cap, uint32_t d, uint32_t nb, FastDiv by_nb, const int32_t *__restrict__ live) {
    constexpr bool GATED = ACT != OP_SQUARED_RELU;
    constexpr int H = GATED ? 2 : 1, UNROLL = unroll_of<DT>(H);
    const uint32_t rows = live != nullptr ? (uint32_t)clamp_live(live, rows_cap) : (uint32_t)rows_cap;
    const uint32_t total = rows * nb;
    const uint32_t step = gridDim.x * FLAT_GROUPS * UNROLL;
    const uint32_t l8 = (threadIdx.x & 15) * 8;
    // a block's row and this lane's column; past the last block that one, unused
    auto place = [&](uint32_t b, uint32_t &row, uint32_t &col, int &n) {
        b = b < total ? b : total - 1;
        row = by_nb(b);
        col = (b - row * nb) * BLOCK8 + l8;
        n = (int)d - (int)col;
    };
    for (uint32_t base = blockIdx.x * FLAT_GROUPS * UNROLL + (threadIdx.x >> 4); base < total; base += step) {
        Oct<DT> dy[UNROLL], g[UNROLL], u[UNROLL];
        uint2 cg[UNROLL], cu[UNROLL];
        float sg[UNROLL], su[UNROLL];
        uint32_t row[UNROLL], col[UNROLL];
        int n[UNROLL];
#pragma unroll
        for (int k = 0; k < UNROLL; ++k) {
            const uint32_t b = base + k * FLAT_GROUPS;
            place(b, row[k], col[k], n[k]);
            oct_fetch<DT, TINY>(dy[k], dout + (size_t)row[k] * d, (int)col[k], (int)d);
            const size_t at = (size_t)row[k] * (H * d);
            if constexpr (KEPT) {
                const size_t block = (size_t)row[k] * (H * nb) + col[k] / BLOCK8;
                cg[k] = codes_fetch<TINY>(codes + at, (int)col[k], (int)d);
                sg[k] = scales[block];
                if constexpr (GATED) {
                    cu[k] = codes_fetch<TINY>(codes + at + d, (int)col[k], (int)d);
                    su[k] = scales[block + nb];
                }
            } else {
                oct_fetch<DT, TINY>(g[k], in + at, (int)col[k], (int)d);
                if constexpr (GATED) oct_fetch<DT, TINY>(u[k], in + at + d, (int)col[k], (int)d);
            }
        }
#pragma unroll
        for (int k = 0; k < UNROLL; ++k) {
            if (base + k * FLAT_GROUPS >= total) continue;
            float x[8], t[8], a[8], v[8];
            oct_trim<DT, TINY>(dy[k], (int)col[k], (int)d);
            oct_unpack<DT>(dy[k], t);
            if constexpr (KEPT) {
                codes_trim<TINY>(cg[k], (int)col[k], (int)d);
                if constexpr (GATED) codes_trim<TINY>(cu[k], (int)col[k], (int)d);
                block_decode(cg[k], sg[k], x);
            } else {
                oct_trim<DT, TINY>(g[k], (int)col[k], (int)d);
                if constexpr (GATED) oct_trim<DT, TINY>(u[k], (int)col[k], (int)d);
                oct_unpack<DT>(g[k], x);
            }
            const size_t at = (size_t)row[k] * (H * d) + col[k];
            if constexpr (GATED) {
                float up[8];
                if constexpr (KEPT) block_decode(cu[k], su[k], up);
                else oct_unpack<DT>(u[k], up);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    float f, df;
                    act_slope<ACT>(x[e], f, df);
                    a[e] = t[e] * up[e] * df;
                    v[e] = t[e] * f;
                }
                oct_store<DT>(dx + at, a, n[k]);
                oct_store<DT>(dx + at + d, v, n[k]);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) a[e] = 2.0f * above_zero<KEPT>(x[e]) * t[e];
                oct_store<DT>(dx + at, a, n[k]);
            }
        }
    }
}

// One workgroup per FLAT_GROUPS * unroll blocks; past GRID_MOST workgroups
// the grid strides.
constexpr int64_t GRID_MOST = 1 << 22;

template <int DT>
dim3 flat_grid(int64_t blocks, int halves) {
    const int64_t per = FLAT_GROUPS * unroll_of<DT>(halves);
    const int64_t g = (blocks + per - 1) / per;
    return dim3((uint32_t)(g < GRID_MOST ? g : GRID_MOST));
}

template <int DT, int ACT>
hipError_t store_as(const void *in, void *out, void *codes, float *scales, int32_t rows, uint32_t d,
                    const int32_t *live, hipStream_t stream) {
    using S = typename Elem<DT>::storage;
    const uint32_t nb = (d + BLOCK8 - 1) / BLOCK8;
    const dim3 grid = flat_grid<DT>((int64_t)rows * nb, ACT == OP_NONE || ACT == OP_SQUARED_RELU ? 1 : 2);
    const auto kernel = d < 8 ? store_kernel<DT, ACT, true> : store_kernel<DT, ACT, false>;
    return launch_kernel(kernel, grid, FLAT_BLOCK, stream, (const S *)in, (S *)out, (uint8_t *)codes, scales, rows, d, nb,
                         FastDiv(nb), live);
}

template <int DT>
hipError_t store_op(int op, const void *in, void *out, void *codes, float *scales, int32_t rows, uint32_t d,
                    const int32_t *live, hipStream_t stream) {
    switch (op) {
    case OP_NONE: return store_as<DT, OP_NONE>(in, out, codes, scales, rows, d, live, stream);
    case OP_SILU_MUL: return store_as<DT, OP_SILU_MUL>(in, out, codes, scales, rows, d, live, stream);
    case OP_GELU_TANH_MUL: return store_as<DT, OP_GELU_TANH_MUL>(in, out, codes, scales, rows, d, live, stream);
    case OP_GELU_ERF_MUL: return store_as<DT, OP_GELU_ERF_MUL>(in, out, codes, scales, rows, d, live, stream);
    case OP_SQUARED_RELU: return store_as<DT, OP_SQUARED_RELU>(in, out, codes, scales, rows, d, live, stream);
    default: return hipErrorInvalidValue;
    }
}

template <int DT>
hipError_t restore_as(const void *codes, const float *scales, const float *stats, void *out, int32_t rows, uint32_t d,
                      int32_t halves, const int32_t *live, hipStream_t stream) {
    const uint32_t nb = (d + BLOCK8 - 1) / BLOCK8;
    const auto kernel = d < 8 ? restore_kernel<DT, true> : restore_kernel<DT, false>;
    return launch_kernel(kernel, flat_grid<DT>((int64_t)rows * halves * nb, 1), FLAT_BLOCK, stream,
                         (const uint8_t *)codes, scales, stats, (typename Elem<DT>::storage *)out, rows, d, nb,
                         FastDiv(nb), halves, live);
}

template <int DT, int ACT>
hipError_t backward_as(const void *dout, const void *in, const void *codes, const float *scales, void *dx,
                       int32_t rows, uint32_t d, const int32_t *live, hipStream_t stream) {
    using S = typename Elem<DT>::storage;
    const uint32_t nb = (d + BLOCK8 - 1) / BLOCK8;
    const dim3 grid = flat_grid<DT>((int64_t)rows * nb, ACT == OP_SQUARED_RELU ? 1 : 2);
    const auto kernel = in == nullptr ? (d < 8 ? backward_kernel<DT, ACT, true, true> : backward_kernel<DT, ACT, true, false>)
                                      : (d < 8 ? backward_kernel<DT, ACT, false, true> : backward_kernel<DT, ACT, false, false>);
    return launch_kernel(kernel, grid, FLAT_BLOCK, stream, (const S *)dout, (const S *)in, (const uint8_t *)codes, scales,
                         (S *)dx, rows, d, nb, FastDiv(nb), live);
}

template <int DT>
hipError_t backward_op(int op, const void *dout, const void *in, const void *codes, const float *scales, void *dx,
                       int32_t rows, uint32_t d, const int32_t *live, hipStream_t stream) {
    switch (op) {
    case OP_SILU_MUL: return backward_as<DT, OP_SILU_MUL>(dout, in, codes, scales, dx, rows, d, live, stream);
    case OP_GELU_TANH_MUL: return backward_as<DT, OP_GELU_TANH_MUL>(dout, in, codes, scales, dx, rows, d, live, stream);
    case OP_GELU_ERF_MUL: return backward_as<DT, OP_GELU_ERF_MUL>(dout, in, codes, scales, dx, rows, d, live, stream);
    case OP_SQUARED_RELU: return backward_as<DT, OP_SQUARED_RELU>(dout, in, codes, scales, dx, rows, d, live, stream);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace

hipError_t launch_checkpoint_store(int dtype, int op, const void *in, void *out, void *codes, float *scales,
                                   int32_t rows, uint32_t d, const int32_t *live, hipStream_t stream) {
    switch (dtype) {
    case DT_F32: return store_op<DT_F32>(op, in, out, codes, scales, rows, d, live, stream);
    case DT_F16: return store_op<DT_F16>(op, in, out, codes, scales, rows, d, live, stream);
    case DT_BF16: return store_op<DT_BF16>(op, in, out, codes, scales, rows, d, live, stream);
    default: return hipErrorInvalidValue;
    }
}

hipError_t launch_checkpoint_restore(int dtype, const void *codes, const float *scales, const float *stats, void *out,
                                     int32_t rows, uint32_t d, int32_t halves, const int32_t *live,
                                     hipStream_t stream) {
    switch (dtype) {
    case DT_F32: return restore_as<DT_F32>(codes, scales, stats, out, rows, d, halves, live, stream);
    case DT_F16: return restore_as<DT_F16>(codes, scales, stats, out, rows, d, halves, live, stream);
    case DT_BF16: return restore_as<DT_BF16>(codes, scales, stats, out, rows, d, halves, live, stream);
    default: return hipErrorInvalidValue;
    }
}

hipError_t launch_act_backward(int dtype, int op, const void *dout, const void *in, const void *codes,
                               const float *scales, void *dx, int32_t rows, uint32_t d, const int32_t *live,
                               hipStream_t stream) {
    switch (dtype) {
    case DT_F32: return backward_op<DT_F32>(op, dout, in, codes, scales, dx, rows, d, live, stream);
    case DT_F16: return backward_op<DT_F16>(op, dout, in, codes, scales, dx, rows, d, live, stream);
    case DT_BF16: return backward_op<DT_BF16>(op, dout, in, codes, scales, dx, rows, d, live, stream);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace ga
