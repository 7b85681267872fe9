// Microscaled 4-bit arrays, gfx950:
//   quantize    x [rows, d] -> codes, scales (ga_mx.h)
//   activation  a gated activation of x [rows, 2d] (squared ReLU: x [rows, d]),
//               rounded to x's type, -> codes, scales
//   dequantize  codes, scales -> x [rows, d]
//
// All three are bound by HBM: every input byte is read once and every output
// byte written once.  As in checkpoint.hip work is numbered in groups of 128
// values of a row, eight to each of 16 lanes; a block of 32 is a quad of lanes,
// so its maximum is two DPP steps.  Measured, bf16 4096 x 16384: quantise 31 us,
// dequantise 30 us (5.5 and 5.7 TB/s), silu straight to 4 bits 48 us (6.3 TB/s).
#include "ga_internal.h"
#include "ga_mx.h"
#include "ga_train.h"

namespace ga {

namespace {

constexpr int FLAT_BLOCK = 256;
constexpr uint32_t FLAT_GROUPS = FLAT_BLOCK / 16;
constexpr int OP_NONE = -1;

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

// nb: blocks a row, ng: groups of 128 values a row
template <int DT, int ACT, bool TINY>
__global__ __launch_bounds__(FLAT_BLOCK) void quantize_kernel(const typename Elem<DT>::storage *__restrict__ in,
                                                              uint32_t *__restrict__ codes, uint8_t *__restrict__ scales,
                                                              int32_t rows_cap, uint32_t d, uint32_t nb, uint32_t ng,
                                                              FastDiv by_ng, const int32_t *__restrict__ live) {
    constexpr bool GATED = ACT >= 0 && ACT != OP_SQUARED_RELU;
    constexpr int H = GATED ? 2 : 1, UNROLL = unroll_of<DT>(H);
    const uint32_t rows = live != nullptr ? (uint32_t)clamp_live(live, rows_cap) : (uint32_t)rows_cap;
    const uint32_t total = rows * ng;
    const uint32_t step = gridDim.x * FLAT_GROUPS * UNROLL;
    const uint32_t l16 = threadIdx.x & 15;
    for (uint32_t base = blockIdx.x * FLAT_GROUPS * UNROLL + (threadIdx.x >> 4); base < total; base += step) {
        Oct<DT> g[UNROLL], u[UNROLL];
        uint32_t row[UNROLL], col[UNROLL];
#pragma unroll
        for (int k = 0; k < UNROLL; ++k) {
            uint32_t b = base + k * FLAT_GROUPS;
            b = b < total ? b : total - 1;
            row[k] = by_ng(b);
            col[k] = (b - row[k] * ng) * 128 + l16 * 8;
            const typename Elem<DT>::storage *x = in + (size_t)row[k] * (H * d);
            oct_fetch<DT, TINY>(g[k], x, (int)col[k], (int)d);
            if constexpr (GATED) oct_fetch<DT, TINY>(u[k], x + d, (int)col[k], (int)d);
        }
#pragma unroll
        for (int k = 0; k < UNROLL; ++k) {
            if (base + k * FLAT_GROUPS >= total) continue;
            float x[8];
            oct_trim<DT, TINY>(g[k], (int)col[k], (int)d);
            oct_unpack<DT>(g[k], x);
            if constexpr (ACT >= 0) {
                float up[8];
                if constexpr (GATED) {
                    oct_trim<DT, TINY>(u[k], (int)col[k], (int)d);
                    oct_unpack<DT>(u[k], up);
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = Elem<DT>::round(GATED ? act_value<ACT>(x[e]) * up[e] : act_value<ACT>(x[e]));
            }
            uint32_t top = magnitude(x[0]);
#pragma unroll
            for (int e = 1; e < 8; ++e) top = max(top, magnitude(x[e]));
            top = dpp_umax<0xB1>(top);
            top = dpp_umax<0x4E>(top);
            const uint32_t s = mx_scale_byte(top), block = col[k] / MX_BLOCK;
            if (block < nb) {
                const size_t at = (size_t)row[k] * nb + block;
                __builtin_nontemporal_store(mx_codes8(x, s), codes + at * 4 + (l16 & 3));
                if ((l16 & 3) == 0) scales[at] = (uint8_t)s;
            }
        }
    }
}

template <int DT>
__global__ __launch_bounds__(FLAT_BLOCK) void dequantize_kernel(const uint32_t *__restrict__ codes,
                                                                const uint8_t *__restrict__ scales,
                                                                typename Elem<DT>::storage *__restrict__ out,
                                                                int32_t rows_cap, uint32_t d, uint32_t nb, uint32_t ng,
                                                                FastDiv by_ng, const int32_t *__restrict__ live) {
    constexpr int UNROLL = unroll_of<DT>(1);
    const uint32_t rows = live != nullptr ? (uint32_t)clamp_live(live, rows_cap) : (uint32_t)rows_cap;
    const uint32_t total = rows * ng;
    const uint32_t step = gridDim.x * FLAT_GROUPS * UNROLL;
    const uint32_t l16 = threadIdx.x & 15;
    for (uint32_t base = blockIdx.x * FLAT_GROUPS * UNROLL + (threadIdx.x >> 4); base < total; base += step) {
        uint32_t c[UNROLL], s[UNROLL], row[UNROLL], col[UNROLL];
#pragma unroll
        for (int k = 0; k < UNROLL; ++k) {
            uint32_t b = base + k * FLAT_GROUPS;
            b = b < total ? b : total - 1;
            row[k] = by_ng(b);
            col[k] = (b - row[k] * ng) * 128 + l16 * 8;
            const uint32_t block = col[k] / MX_BLOCK;
            const size_t at = (size_t)row[k] * nb + (block < nb ? block : nb - 1);
            c[k] = __builtin_nontemporal_load(codes + at * 4 + (l16 & 3));
            s[k] = scales[at];
        }
#pragma unroll
        for (int k = 0; k < UNROLL; ++k) {
            if (base + k * FLAT_GROUPS >= total || col[k] >= d) continue;
            float x[8];
            mx_values8(c[k], s[k], x);
            oct_store<DT>(out + (size_t)row[k] * d + col[k], x, (int)(d - col[k]));
        }
    }
}

// One workgroup per FLAT_GROUPS * unroll groups; past GRID_MOST workgroups the
// grid strides.
constexpr int64_t GRID_MOST = 1 << 22;

template <int DT>
dim3 flat_grid(int64_t groups, int halves) {
    const int64_t per = FLAT_GROUPS * unroll_of<DT>(halves);
    const int64_t g = (groups + per - 1) / per;
    return dim3((uint32_t)(g < GRID_MOST ? g : GRID_MOST));
}

template <int DT, int ACT>
hipError_t quantize_as(const void *in, void *codes, uint8_t *scales, int32_t rows, uint32_t d, const int32_t *live,
                       hipStream_t stream) {
    const uint32_t nb = (d + MX_BLOCK - 1) / MX_BLOCK, ng = (d + 127) / 128;
    const auto kernel = d < 8 ? quantize_kernel<DT, ACT, true> : quantize_kernel<DT, ACT, false>;
    const dim3 grid = flat_grid<DT>((int64_t)rows * ng, ACT >= 0 && ACT != OP_SQUARED_RELU ? 2 : 1);
    return launch_kernel(kernel, grid, FLAT_BLOCK, stream, (const typename Elem<DT>::storage *)in, (uint32_t *)codes,
                         scales, rows, d, nb, ng, FastDiv(ng), live);
}

template <int DT>
hipError_t quantize_op(int op, const void *in, void *codes, uint8_t *scales, int32_t rows, uint32_t d,
                       const int32_t *live, hipStream_t stream) {
    switch (op) {
    case OP_NONE: return quantize_as<DT, OP_NONE>(in, codes, scales, rows, d, live, stream);
    case OP_SILU_MUL: return quantize_as<DT, OP_SILU_MUL>(in, codes, scales, rows, d, live, stream);
    case OP_GELU_TANH_MUL: return quantize_as<DT, OP_GELU_TANH_MUL>(in, codes, scales, rows, d, live, stream);
    case OP_GELU_ERF_MUL: return quantize_as<DT, OP_GELU_ERF_MUL>(in, codes, scales, rows, d, live, stream);
    case OP_SQUARED_RELU: return quantize_as<DT, OP_SQUARED_RELU>(in, codes, scales, rows, d, live, stream);
    default: return hipErrorInvalidValue;
    }
}

template <int DT>
hipError_t dequantize_as(const void *codes, const uint8_t *scales, void *out, int32_t rows, uint32_t d,
                         const int32_t *live, hipStream_t stream) {
    const uint32_t nb = (d + MX_BLOCK - 1) / MX_BLOCK, ng = (d + 127) / 128;
    return launch_kernel(dequantize_kernel<DT>, flat_grid<DT>((int64_t)rows * ng, 1), FLAT_BLOCK, stream,
                         (const uint32_t *)codes, scales, (typename Elem<DT>::storage *)out, rows, d, nb, ng, FastDiv(ng),
                         live);
}

}  // namespace

hipError_t launch_mxfp4_quantize(int dtype, int op, const void *in, void *codes, uint8_t *scales, int32_t rows,
                                 uint32_t d, const int32_t *live, hipStream_t stream) {
    switch (dtype) {
    case DT_F32: return quantize_op<DT_F32>(op, in, codes, scales, rows, d, live, stream);
    case DT_F16: return quantize_op<DT_F16>(op, in, codes, scales, rows, d, live, stream);
    case DT_BF16: return quantize_op<DT_BF16>(op, in, codes, scales, rows, d, live, stream);
    default: return hipErrorInvalidValue;
    }
}

hipError_t launch_mxfp4_dequantize(int dtype, const void *codes, const uint8_t *scales, void *out, int32_t rows,
                                   uint32_t d, const int32_t *live, hipStream_t stream) {
    switch (dtype) {
    case DT_F32: return dequantize_as<DT_F32>(codes, scales, out, rows, d, live, stream);
    case DT_F16: return dequantize_as<DT_F16>(codes, scales, out, rows, d, live, stream);
    case DT_BF16: return dequantize_as<DT_BF16>(codes, scales, out, rows, d, live, stream);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace ga
