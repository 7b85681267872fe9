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
// has s = 0 and the term is taken as 0).  From x that is q_i - A - B (gate_i - m)
// with A = G / d and B = A z / s, two numbers a row.  From codes gate - m is
// t + z s, and with A = (1 + z^2) G / d it is q_i - A - B t_i; from x that form
// would lose z^2 roundings of t for nothing.  B (gate - m) is formed with both
// scaled by the power of two of 1 / s: z / s alone passes fp32's range where a
// row has next to no spread.
//
// gelu_tanh'(0) is 1/2, so the gradient jumps where the gate passes the
// cutoff: the side is decided from sums in fp64, which runs at fp32's rate here
// (34 T lane operations a second either way), of differences in fp64.  The kept codes are those of t, with t > 0 never below
// code 1: an 8-bit gate would change sides within half a step of the cutoff.
// What the codes are relative to is kept as two floats a row, (c, s).
//
// A team of W wavefronts holds the row in registers, V octets a lane, so every
// byte is read once: one reduction for the statistics (a shifted sum and sum
// of squares, see shifted_moments), one for G.  dup goes out as soon as it is
// formed; only q and t stay for the second half.
//
// Measured (medians of a kernel trace, bf16): forward 2048 x 16384 (271 MB)
// 52 - 55 us, 4.9 - 5.2 TB/s, its vector units busy 74 % of the time (about 44
// instructions a value, half of them for the two codes); backward from codes
// 51.4 us, 5.3 TB/s; backward from x 2048 x 8192 (168 MB) 32.0 us, 5.2 TB/s,
// 2048 x 16384 (336 MB) 61.7 us, 5.4 TB/s; forward 16384 x 2048 48.2 us, 5.6 TB/s,
// backward from codes 45.1 us, 6.0 TB/s; 512 x 65536 forward 57.9 us, backward from
// codes 52.6 us, from x 75.4 us, where eight octets a lane spill (in both backward
// forms, and in fp32's forward).
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
    if constexpr (W == 1) return {team_row<64>(blockIdx.x * 4 + (threadIdx.x >> 6)), threadIdx.x & 63};
    else return {blockIdx.x, threadIdx.x};
}

// Statistics of the row's gate octets; every lane of the team gets the same.
template <int DT, int W, int V>
__device__ __forceinline__ void gate_moments(const Oct<DT> (&g)[V], uint32_t lane, int d, double inv_d, float first,
                                             double *slots, double &mean, double &var) {
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
        add_shifted(x, first, s1, s2);
    }
    team_sum2<64 * W>(s1, s2, slots);
    shifted_moments(s1, s2, (double)first, inv_d, mean, var);
}

template <int DT, int W, int V, bool TINY>
__device__ __forceinline__ void trim_all(Oct<DT> (&o)[V], uint32_t lane, int d) {
#pragma unroll
    for (int v = 0; v < V; ++v) oct_trim<DT, TINY>(o[v], (int)(v * 64 * W + lane) * 8, d);
}

// fp32(gate - at) of an octet, at the cutoff or the mean; 0 past the row's end.
template <int DT>
__device__ __forceinline__ void less(const Oct<DT> &g, const RowOrigin<DT> &at, int n, float (&t)[8]) {
    oct_unpack<DT>(g, t);
#pragma unroll
    for (int e = 0; e < 8; ++e) t[e] = at.from(t[e]);
    if (n < 8) {
#pragma unroll
        for (int e = 0; e < 8; ++e) t[e] = e < n ? t[e] : 0.0f;
    }
}

// Waves a SIMD holds at least.  16-wave workgroups pair up on a compute unit
// within 64 registers, which two octets a lane of 16-bit values fit.
template <int DT, int W, int V> constexpr int sparse_waves() { return DT == DT_F32 || V > 2 ? 4 : W == 16 ? 8 : 6; }

// TINY: rows of fewer than eight values.
template <int DT, int W, int V, bool TINY>
__global__ __launch_bounds__(team_block<W>(), (sparse_waves<DT, W, V>())) void sparse_store_kernel(
    const typename Elem<DT>::storage *__restrict__ in, typename Elem<DT>::storage *__restrict__ out,
    uint8_t *__restrict__ codes, float *__restrict__ scales, float *__restrict__ stats, int32_t rows, int32_t d,
    uint32_t nb, float z, double inv_d, const int32_t *__restrict__ live) {
    __shared__ double slots[2 * W];
    const RowAt at = row_of_team<W>();
    const uint32_t live_rows = live != nullptr ? (uint32_t)clamp_live(live, rows) : (uint32_t)rows;
    if (at.row >= live_rows) return;
    const typename Elem<DT>::storage *x = in + (size_t)at.row * 2 * d;
    Oct<DT> g[V], u[V];
#pragma unroll
    for (int v = 0; v < V; ++v) oct_fetch<DT, TINY>(g[v], x, (int)(v * 64 * W + at.lane) * 8, d);
    constexpr bool EARLY = V <= 4;  // up with the gate, while registers last
    if constexpr (EARLY) {
#pragma unroll
        for (int v = 0; v < V; ++v) oct_fetch<DT, TINY>(u[v], x + d, (int)(v * 64 * W + at.lane) * 8, d);
    }
    const float first = row_pivot<DT>(x, d);
    double mean, var;
    trim_all<DT, W, V, TINY>(g, at.lane, d);
    gate_moments<DT, W, V>(g, at.lane, d, inv_d, first, slots, mean, var);
#pragma unroll
    for (int v = 0; v < V; ++v) stay_raw(g[v]);
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
        uint32_t lane = at.lane;
        // columns formed again: kept from the gate's loads, eight of them spill, and a load of up then waits for
        // its address behind the stores of the octet before
        if constexpr (!EARLY) asm volatile("" : "+v"(lane));
        const int c = (int)(v * 64 * W + lane) * 8;
        const int n = d - c;
        const uint32_t block = (uint32_t)c / BLOCK8;
        if constexpr (!EARLY) {
            __builtin_amdgcn_sched_barrier(0);
            oct_fetch<DT, TINY>(u[v], x + d, c, d);
        }
        if (block >= nb) continue;  // the same for the 16 lanes of a block
        float t[8], up[8], scale;
        less<DT>(g[v], cutoff, n, t);
        const uint2 ct = block_encode<difference_of<DT>(), true>(t, scale);
        codes_store(row_codes + (uint32_t)c, ct, n);
        if ((at.lane & 15) == 0) row_scales[block] = scale;
        oct_trim<DT, TINY>(u[v], c, d);
        oct_unpack<DT>(u[v], up);
        const uint2 cu = block_encode<code_of<DT>(), false>(up, scale);
        codes_store(row_codes + (uint32_t)(d + c), cu, n);
        if ((at.lane & 15) == 0) row_scales[nb + block] = scale;
#pragma unroll
        for (int e = 0; e < 8; ++e) t[e] = gelu_tanh(__builtin_fmaxf(t[e], 0.0f)) * up[e];
        oct_store<DT>(out + (size_t)at.row * d + (uint32_t)c, t, n);
    }
}

// KEPT: t and up restored from the codes, s from stats; else from x.
template <int DT, int W, int V, bool TINY, bool KEPT>
__global__ __launch_bounds__(team_block<W>(), (sparse_waves<DT, W, V>())) void sparse_backward_kernel(
    const typename Elem<DT>::storage *__restrict__ dout, const typename Elem<DT>::storage *__restrict__ in,
    const uint8_t *__restrict__ codes, const float *__restrict__ scales, const float *__restrict__ stats,
    typename Elem<DT>::storage *__restrict__ dx, int32_t rows, int32_t d, uint32_t nb, float z,
    double inv_d, const int32_t *__restrict__ live) {
    __shared__ double slots[2 * W];
    __shared__ float sums[2 * W];
    const RowAt at = row_of_team<W>();
    const uint32_t live_rows = live != nullptr ? (uint32_t)clamp_live(live, rows) : (uint32_t)rows;
    if (at.row >= live_rows) return;
    const size_t row2 = (size_t)at.row * 2 * d;
    const typename Elem<DT>::storage *dy = dout + (size_t)at.row * d;
    // all of the row's loads at once with up to two octets a lane
    constexpr bool EARLY = V <= 2;
    Oct<DT> g[KEPT ? 1 : V], o[V], u[KEPT ? 1 : V];
    uint2 ct[KEPT ? V : 1], cu[KEPT ? V : 1];
    float st[KEPT ? V : 1], su[KEPT ? V : 1];
    auto load = [&](int v) {
        const int c = (int)(v * 64 * W + at.lane) * 8;
        oct_fetch<DT, TINY>(o[v], dy, c, d);
        if constexpr (KEPT) {
            const uint32_t block = (uint32_t)c / BLOCK8 < nb ? (uint32_t)c / BLOCK8 : nb - 1;
            const float *row_scales = scales + (size_t)at.row * 2 * nb + block;
            ct[v] = codes_fetch<TINY>(codes + row2, c, d);
            cu[v] = codes_fetch<TINY>(codes + row2 + d, c, d);
            st[v] = row_scales[0];
            su[v] = row_scales[nb];
        } else {
            oct_fetch<DT, TINY>(u[v], in + row2 + d, c, d);
        }
    };
    RowOrigin<DT> cutoff(0.0), middle(0.0);
    double std;
    if constexpr (KEPT) {
        if constexpr (EARLY) {
#pragma unroll
            for (int v = 0; v < V; ++v) load(v);
        }
        std = stats[2 * (size_t)at.row + 1];
    } else {
        const typename Elem<DT>::storage *x = in + row2;
#pragma unroll
        for (int v = 0; v < V; ++v) oct_fetch<DT, TINY>(g[v], x, (int)(v * 64 * W + at.lane) * 8, d);
        const float first = row_pivot<DT>(x, d);
        if constexpr (EARLY) {
#pragma unroll
            for (int v = 0; v < V; ++v) load(v);
        }
        double mean, var;
        trim_all<DT, W, V, TINY>(g, at.lane, d);
        gate_moments<DT, W, V>(g, at.lane, d, inv_d, first, slots, mean, var);
#pragma unroll
        for (int v = 0; v < V; ++v) stay_raw(g[v]);
        std = __builtin_sqrt(var);
        cutoff = RowOrigin<DT>(__builtin_fma((double)z, std, mean));
        middle = RowOrigin<DT>(mean);
    }
    float q[V][8], total = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int c = (int)(v * 64 * W + at.lane) * 8;
        const int n = d - c;
        float t[8], up[8], dv[8], du[8];
        if constexpr (V > 2) __builtin_amdgcn_sched_barrier(0);  // one octet at a time: interleaved they spill
        if constexpr (!EARLY) load(v);
        oct_trim<DT, TINY>(o[v], c, d);
        if constexpr (KEPT) {
            codes_trim<TINY>(ct[v], c, d);
            codes_trim<TINY>(cu[v], c, d);
            block_decode(ct[v], st[v], t);
            block_decode(cu[v], su[v], up);
        } else {
            oct_trim<DT, TINY>(u[v], c, d);
            less<DT>(g[v], cutoff, n, t);
            oct_unpack<DT>(u[v], up);
        }
        oct_unpack<DT>(o[v], dv);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float f, df;
            gelu_tanh_slope(above_zero<KEPT>(t[e]), f, df);
            // a restored NaN stands for a value whose side is lost: it goes into the row's sum
            const bool on = KEPT ? !(t[e] <= 0.0f) : t[e] > 0.0f;
            q[v][e] = on ? dv[e] * up[e] * df : 0.0f;
            asm volatile("" : "+v"(q[v][e]));  // else its factors are kept for a later fma: twice the registers
            du[e] = dv[e] * f;
            total += q[v][e];
        }
        oct_store<DT>(dx + row2 + (uint32_t)(d + c), du, n);
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
        if constexpr (KEPT) stay_raw(ct[v]);
        else stay_raw(g[v]);
    }
    float unused = 0.0f;
    team_sum2<64 * W>(total, unused, sums);
    const float share = total * (float)inv_d;
    // unit = 2^-e for std in [2^e, 2^(e+1)), e within fp32's normal exponents
    int e2 = (int)(__builtin_bit_cast(uint64_t, std) >> 52) - 1023;
    e2 = e2 < -126 ? -126 : e2 > 126 ? 126 : e2;
    const float unit = __builtin_bit_cast(float, (uint32_t)(127 - e2) << 23);
    // (no gradient, no share of it: z * z may be past fp32's range)
    const bool alone = std == 0.0 || share == 0.0f;
    const float b = alone ? 0.0f : share * z * (float)(1.0 / (std * (double)unit));
    const float a = !KEPT || alone ? share : __builtin_fmaf(share, z * z, share);
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int c = (int)(v * 64 * W + at.lane) * 8;
        const int n = d - c;
        if constexpr (V > 2) __builtin_amdgcn_sched_barrier(0);
        if (n <= 0) continue;
        float t[8];
        if constexpr (KEPT) block_decode(ct[v], st[v], t);
        else less<DT>(g[v], middle, n, t);
#pragma unroll
        for (int e = 0; e < 8; ++e) t[e] = q[v][e] - __builtin_fmaf(b, t[e] * unit, a);
        oct_store<DT>(dx + row2 + (uint32_t)c, t, n);
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

template <Pass P, int DT, int W, int V, bool TINY = false>
hipError_t launch_as(const Args &a) {
    using S = typename Elem<DT>::storage;
    const uint32_t nb = ((uint32_t)a.d + BLOCK8 - 1) / BLOCK8;
    const dim3 grid((uint32_t)(((int64_t)a.rows + team_rows<W>() - 1) / team_rows<W>()));
    const dim3 block(team_block<W>());
    const double inv_d = 1.0 / a.d;
    if constexpr (P == STORE)
        return launch_kernel(sparse_store_kernel<DT, W, V, TINY>, grid, block, a.stream, (const S *)a.in, (S *)a.out,
                             (uint8_t *)a.codes, a.scales, a.stats, a.rows, a.d, nb, a.z, inv_d, a.live);
    else
        return launch_kernel(sparse_backward_kernel<DT, W, V, TINY, P == BACKWARD_KEPT>, grid, block, a.stream,
                             (const S *)a.dout, (const S *)a.in, (const uint8_t *)a.codes, a.scales, a.stats,
                             (S *)a.out, a.rows, a.d, nb, a.z, inv_d, a.live);
}

template <Pass P, int DT>
hipError_t launch_dt(const Args &a) {
    if (a.d < 8) return launch_as<P, DT, 1, 1, true>(a);
    if (a.d <= 512) return launch_as<P, DT, 1, 1>(a);
    switch (sparse_train_waves(a.d)) {
    case 1: return launch_as<P, DT, 1, 2>(a);
    case 2: return launch_as<P, DT, 2, 2>(a);
    case 4: return launch_as<P, DT, 4, 2>(a);
    case 8: return launch_as<P, DT, 8, 2>(a);
    default: break;
    }
    // From x at 16 waves of two octets the backward needs more than the 64
    // registers that let two workgroups share a compute unit: 2048 rows of
    // 16384, bf16, 69 us, against 59 us for eight waves of four (fastest of a trace).
    constexpr int W = P == BACKWARD ? 8 : 16;
    if (a.d <= 16384) return launch_as<P, DT, W, 32 / W>(a);
    if (a.d <= 32768) return launch_as<P, DT, 16, 4>(a);
    return launch_as<P, DT, 16, 8>(a);
}

template <Pass P>
hipError_t launch_pass(int dtype, const Args &a) {
    switch (dtype) {
    case DT_F32: return launch_dt<P, DT_F32>(a);
    case DT_F16: return launch_dt<P, DT_F16>(a);
    case DT_BF16: return launch_dt<P, DT_BF16>(a);
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
    return launch_pass<STORE>(dtype, Args{nullptr, in, out, codes, scales, stats, rows, d, z, live, stream});
}

hipError_t launch_sparse_backward(int dtype, const void *dout, const void *in, const void *codes, const float *scales,
                                  const float *stats, void *dx, int32_t rows, int32_t d, float z, const int32_t *live,
                                  hipStream_t stream) {
    const Args a{dout, in, dx, const_cast<void *>(codes), const_cast<float *>(scales), const_cast<float *>(stats),
                 rows, d, z, live, stream};
    return in != nullptr ? launch_pass<BACKWARD>(dtype, a) : launch_pass<BACKWARD_KEPT>(dtype, a);
}

}  // namespace ga
