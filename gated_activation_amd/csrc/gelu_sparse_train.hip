// The sparse GELU's training pair, gfx950: the forward pass that keeps its
// input in 8 bits, and the backward pass from those codes or from the input.
//
// Per row of x = [gate | up] (d values each), with mean m and population
// std s of the gate and the cutoff c = m + z s:
//     t = fp32(gate - c), out = gelu_tanh(max(t, 0)) up
//     q_i  = dout_i up_i gelu_tanh'(t_i) where t_i > 0, else 0;  G = sum q
//     dgate_i = q_i - (G / d) (1 + z (gate_i - m) / s)
//     dup_i   = dout_i gelu_tanh(max(t_i, 0))
// (the second term of the bracket is the derivative of s; a row without spread
// has s = 0 and the term is taken as 0).  gate - m is t + z s, so
// dgate_i = q_i - A - B t_i with two numbers A, B a row.
//
// gelu_tanh'(0) is 1/2, so the gradient jumps where the gate passes the
// cutoff: the side is decided in fp64 (statistics and difference), which runs
// at fp32's rate here.  The kept codes are those of t, with t > 0 never below
// code 1: an 8-bit gate would change sides within half a step of the cutoff.
// What the codes are relative to is kept as two floats a row, (c, s).
//
// A team of W wavefronts holds the row in registers, V octets a lane, so every
// byte is read once: one reduction for the statistics (a shifted sum and sum
// of squares, see shifted_moments), one for G.  dup goes out as soon as it is
// formed; only q and t stay for the second half.
#include "ga_internal.h"
#include "ga_train.h"

namespace ga {

namespace {

template <int W> constexpr int team_rows() { return W == 1 ? 4 : 1; }   // rows of a workgroup
template <int W> constexpr int team_block() { return W == 1 ? 256 : 64 * W; }

struct RowAt {
    uint32_t row, lane;  // the row and this lane's place in its team
};

template <int W>
__device__ __forceinline__ RowAt row_of_team() {
    if constexpr (W == 1) return {blockIdx.x * 4 + (threadIdx.x >> 6), threadIdx.x & 63};
    else return {blockIdx.x, threadIdx.x};
}

// Statistics of the row's gate octets; every lane of the team gets the same.
template <int DT, int W, int V>
__device__ __forceinline__ void gate_moments(const Oct<DT> (&g)[V], uint32_t lane, int d, float first, double *slots,
                                             double &mean, double &var) {
    double s1 = 0.0, s2 = 0.0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int n = d - (int)(v * 64 * W + lane) * 8;
        float x[8];
        oct_unpack<DT>(g[v], x);
        if (n < 8) {
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = e < n ? x[e] : first;
        }
        add_shifted<DT>(x, first, s1, s2);
    }
    team_sum2<64 * W>(s1, s2, slots);
    shifted_moments(s1, s2, (double)first, (double)d, mean, var);
}

// fp32(gate - cutoff) of an octet; 0 past the row's end.
template <int DT>
__device__ __forceinline__ void over_cutoff(const Oct<DT> &g, const RowOrigin<DT> &cutoff, int n, float (&t)[8]) {
    oct_unpack<DT>(g, t);
#pragma unroll
    for (int e = 0; e < 8; ++e) t[e] = cutoff.from(t[e]);
    if (n < 8) {
#pragma unroll
        for (int e = 0; e < 8; ++e) t[e] = e < n ? t[e] : 0.0f;
    }
}

// Waves a SIMD holds at least: 16-wave workgroups of two octets a lane pair up
// on a compute unit within 64 registers (a third register pair halves that).
template <int DT, int W, int V> constexpr int sparse_waves() { return DT != DT_F32 && W == 16 && V == 2 ? 8 : 4; }

template <int DT, int W, int V>
__global__ __launch_bounds__(team_block<W>(), (sparse_waves<DT, W, V>())) void sparse_store_kernel(
    const typename Elem<DT>::storage *__restrict__ in, typename Elem<DT>::storage *__restrict__ out,
    uint8_t *__restrict__ codes, float *__restrict__ scales, float *__restrict__ stats, int32_t rows, int32_t d,
    uint32_t nb, float z, const int32_t *__restrict__ live) {
    __shared__ double slots[2 * W];
    const RowAt at = row_of_team<W>();
    const uint32_t live_rows = live != nullptr ? (uint32_t)clamp_live(live, rows) : (uint32_t)rows;
    if (at.row >= live_rows) return;
    const typename Elem<DT>::storage *x = in + (size_t)at.row * 2 * d;
    Oct<DT> g[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int c = (int)(v * 64 * W + at.lane) * 8;
        oct_load<DT>(g[v], x + c, d - c);
    }
    Oct<DT> u[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int c = (int)(v * 64 * W + at.lane) * 8;
        oct_load<DT>(u[v], x + d + c, d - c);
    }
    const float first = Elem<DT>::to_f32(x[0]);
    double mean, var;
    gate_moments<DT, W, V>(g, at.lane, d, first, slots, mean, var);
    const double std = __builtin_sqrt(var);
    const RowOrigin<DT> cutoff(__builtin_fma((double)z, std, mean));
    if (at.lane == 0) {
        stats[2 * (size_t)at.row] = cutoff.hi;
        stats[2 * (size_t)at.row + 1] = (float)std;
    }
    uint8_t *row_codes = codes + (size_t)at.row * 2 * d;
    float *row_scales = scales + (size_t)at.row * 2 * nb;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int c = (int)(v * 64 * W + at.lane) * 8;
        const int n = d - c;
        const uint32_t block = (uint32_t)c / BLOCK8;
        if (block >= nb) continue;  // the same for the 16 lanes of a block
        float t[8], up[8], scale;
        over_cutoff<DT>(g[v], cutoff, n, t);
        const uint2 ct = block_encode<difference_of<DT>(), true>(t, scale);
        codes_store(row_codes + c, ct, n);
        if ((at.lane & 15) == 0) row_scales[block] = scale;
        oct_unpack<DT>(u[v], up);
        const uint2 cu = block_encode<code_of<DT>(), false>(up, scale);
        codes_store(row_codes + d + c, cu, n);
        if ((at.lane & 15) == 0) row_scales[nb + block] = scale;
#pragma unroll
        for (int e = 0; e < 8; ++e) t[e] = gelu_tanh(__builtin_fmaxf(t[e], 0.0f)) * up[e];
        oct_store<DT>(out + (size_t)at.row * d + c, t, n);
    }
}

// KEPT: t and up restored from the codes, s from stats; else from x.
template <int DT, int W, int V, bool KEPT>
__global__ __launch_bounds__(team_block<W>()) void sparse_backward_kernel(
    const typename Elem<DT>::storage *__restrict__ dout, const typename Elem<DT>::storage *__restrict__ in,
    const uint8_t *__restrict__ codes, const float *__restrict__ scales, const float *__restrict__ stats,
    typename Elem<DT>::storage *__restrict__ dx, int32_t rows, int32_t d, uint32_t nb, float z,
    const int32_t *__restrict__ live) {
    __shared__ double slots[2 * W];
    __shared__ float sums[2 * W];
    const RowAt at = row_of_team<W>();
    const uint32_t live_rows = live != nullptr ? (uint32_t)clamp_live(live, rows) : (uint32_t)rows;
    if (at.row >= live_rows) return;
    const size_t row2 = (size_t)at.row * 2 * d;
    const typename Elem<DT>::storage *dy = dout + (size_t)at.row * d;
    Oct<DT> g[KEPT ? 1 : V];
    uint2 ct[KEPT ? V : 1];
    float st[KEPT ? V : 1];
    RowOrigin<DT> cutoff(0.0);
    float s;
    if constexpr (KEPT) {
        s = stats[2 * (size_t)at.row + 1];
    } else {
        const typename Elem<DT>::storage *x = in + row2;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = (int)(v * 64 * W + at.lane) * 8;
            oct_load<DT>(g[v], x + c, d - c);
        }
        const float first = Elem<DT>::to_f32(x[0]);
        double mean, var;
        gate_moments<DT, W, V>(g, at.lane, d, first, slots, mean, var);
        const double std = __builtin_sqrt(var);
        cutoff = RowOrigin<DT>(__builtin_fma((double)z, std, mean));
        s = (float)std;
    }
    float q[V][8], total = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int c = (int)(v * 64 * W + at.lane) * 8;
        const int n = d - c;
        if (n <= 0) {
#pragma unroll
            for (int e = 0; e < 8; ++e) q[v][e] = 0.0f;
            continue;
        }
        Oct<DT> o;
        float t[8], up[8], dv[8], du[8];
        oct_load<DT>(o, dy + c, n);
        if constexpr (KEPT) {
            const float *row_scales = scales + (size_t)at.row * 2 * nb + (uint32_t)c / BLOCK8;
            ct[v] = codes_load(codes + row2 + c, n);
            st[v] = row_scales[0];
            block_decode(ct[v], st[v], t);
            block_decode(codes_load(codes + row2 + d + c, n), row_scales[nb], up);
        } else {
            Oct<DT> u;
            oct_load<DT>(u, in + row2 + d + c, n);
            over_cutoff<DT>(g[v], cutoff, n, t);
            oct_unpack<DT>(u, up);
        }
        oct_unpack<DT>(o, dv);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float f, df;
            gelu_tanh_slope(__builtin_fmaxf(t[e], 0.0f), f, df);
            q[v][e] = t[e] > 0.0f ? dv[e] * up[e] * df : 0.0f;
            du[e] = dv[e] * f;
            total += q[v][e];
        }
        oct_store<DT>(dx + row2 + d + c, du, n);
    }
    float unused = 0.0f;
    team_sum2<64 * W>(total, unused, sums);
    const float share = total / (float)d;
    const float b = s == 0.0f ? 0.0f : share * z / s;
    const float a = s == 0.0f ? share : __builtin_fmaf(share, z * z, share);
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int c = (int)(v * 64 * W + at.lane) * 8;
        const int n = d - c;
        if (n <= 0) continue;
        float t[8];
        if constexpr (KEPT) block_decode(ct[v], st[v], t);
        else over_cutoff<DT>(g[v], cutoff, n, t);
#pragma unroll
        for (int e = 0; e < 8; ++e) t[e] = q[v][e] - __builtin_fmaf(b, t[e], a);
        oct_store<DT>(dx + row2 + c, t, n);
    }
}

struct Args {
    const void *dout, *in;
    void *out;
    void *codes;
    float *scales, *stats;
    int32_t rows, d;
    float z;
    const int32_t *live;
    hipStream_t stream;
};

enum Pass { STORE, BACKWARD, BACKWARD_KEPT };

template <int DT, int W, int V>
hipError_t launch_as(Pass pass, const Args &a) {
    using S = typename Elem<DT>::storage;
    const uint32_t nb = ((uint32_t)a.d + BLOCK8 - 1) / BLOCK8;
    const dim3 grid((uint32_t)(((int64_t)a.rows + team_rows<W>() - 1) / team_rows<W>()));
    const dim3 block(team_block<W>());
    if (pass == STORE)
        sparse_store_kernel<DT, W, V><<<grid, block, 0, a.stream>>>((const S *)a.in, (S *)a.out, (uint8_t *)a.codes,
                                                                    a.scales, a.stats, a.rows, a.d, nb, a.z, a.live);
    else if (pass == BACKWARD)
        sparse_backward_kernel<DT, W, V, false><<<grid, block, 0, a.stream>>>(
            (const S *)a.dout, (const S *)a.in, nullptr, nullptr, nullptr, (S *)a.out, a.rows, a.d, nb, a.z, a.live);
    else
        sparse_backward_kernel<DT, W, V, true><<<grid, block, 0, a.stream>>>(
            (const S *)a.dout, nullptr, (const uint8_t *)a.codes, a.scales, a.stats, (S *)a.out, a.rows, a.d, nb, a.z,
            a.live);
    return hipGetLastError();
}

template <int DT>
hipError_t launch_dt(Pass pass, const Args &a) {
    const int waves = sparse_train_waves(a.d);
    const int64_t octets = ((int64_t)a.d + 7) / 8;
    const int64_t v = (octets + 64 * waves - 1) / (64 * waves);
    switch (waves) {
    case 1: return v <= 1 ? launch_as<DT, 1, 1>(pass, a) : launch_as<DT, 1, 2>(pass, a);
    case 2: return launch_as<DT, 2, 2>(pass, a);
    case 4: return launch_as<DT, 4, 2>(pass, a);
    case 8: return launch_as<DT, 8, 2>(pass, a);
    default:
        return v <= 2 ? launch_as<DT, 16, 2>(pass, a) : v <= 4 ? launch_as<DT, 16, 4>(pass, a)
                                                               : launch_as<DT, 16, 8>(pass, a);
    }
}

hipError_t launch_any(int dtype, Pass pass, const Args &a) {
    switch (dtype) {
    case DT_F32: return launch_dt<DT_F32>(pass, a);
    case DT_F16: return launch_dt<DT_F16>(pass, a);
    case DT_BF16: return launch_dt<DT_BF16>(pass, a);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace

// Two octets a lane where the row allows it: 64 W lanes of 16 values.
int sparse_train_waves(int64_t d) {
    int w = 1;
    while (w < 16 && (int64_t)w * 1024 < d) w *= 2;
    return w;
}

hipError_t launch_sparse_store(int dtype, const void *in, void *out, void *codes, float *scales, float *stats,
                               int32_t rows, int32_t d, float z, const int32_t *live, hipStream_t stream) {
    return launch_any(dtype, STORE, Args{nullptr, in, out, codes, scales, stats, rows, d, z, live, stream});
}

hipError_t launch_sparse_backward(int dtype, const void *dout, const void *in, const void *codes, const float *scales,
                                  const float *stats, void *dx, int32_t rows, int32_t d, float z, const int32_t *live,
                                  hipStream_t stream) {
    return launch_any(dtype, in != nullptr ? BACKWARD : BACKWARD_KEPT,
                      Args{dout, in, dx, const_cast<void *>(codes), const_cast<float *>(scales),
                           const_cast<float *>(stats), rows, d, z, live, stream});
}

}  // namespace ga
