// Layer norm with its backward pass, gfx950.
//
// forward, per row of x [rows, d] with mean m and population variance v:
//     r = 1 / sqrt(v + eps), n_i = (x_i - m) r, y_i = n_i w_i + b_i
// keeping (m, r) as two floats and, where asked, fp32(x - m) in 8-bit blocks
// (block_encode in ga_train.h).
// backward, with v_i = dy_i w_i:
//     dx_i = r (v_i - mean(v) - n_i mean(v n)),
//     dw_i = sum over rows of dy_i n_i, db_i = sum over rows of dy_i
// with n from x and (m, r), or r times the value its code stands for.
//
// Both are bound by HBM.  A team of lanes (a 16-lane DPP row, a wavefront, or
// a workgroup) holds a row in registers, V octets a lane, so a row is read
// once.  The statistics are fp64 (shifted_moments): one reduction, exact for a
// constant row, no loss where the mean is large against the spread.
//
// The backward's weight gradient is a sum over all rows, column by column: a
// lane owns the same columns in every row its team takes, so it adds them in
// registers (fp32), 16 V accumulators.  At the end a workgroup's teams are
// added through LDS in a fixed order and leave one partial row; a second
// launch adds the workgroups' partials, again in a fixed order, so the result
// does not depend on scheduling.  One workgroup per compute unit keeps those
// partials at 8 d bytes times 256.
#include "ga_internal.h"
#include "ga_train.h"

namespace ga {

namespace {

// fp32 weights where WIDE, else the rows' type.
template <int DT, bool WIDE> constexpr int weight_type() { return WIDE ? DT_F32 : DT; }

// The team of a row by its width: LANES lanes of V octets.  Two octets a lane
// halve what the row's reductions cost a value; a row of up to 1024 values is
// a wavefront's own and needs no barrier.
template <int LANES_, int V_> struct Team {
    static constexpr int LANES = LANES_, V = V_;
};

template <typename F>
auto by_width(int64_t d, F &&f) {
    if (d <= 128) return f(Team<16, 1>());
    if (d <= 512) return f(Team<64, 1>());
    if (d <= 1024) return f(Team<64, 2>());
    if (d <= 2048) return f(Team<128, 2>());
    if (d <= 4096) return f(Team<256, 2>());
    if (d <= 8192) return f(Team<512, 2>());
    if (d <= 16384) return f(Team<1024, 2>());
    return f(Team<1024, 4>());
}

constexpr int FORWARD_BLOCK = 256;  // workgroups of several teams; a larger team is one by itself
template <int LANES> constexpr int forward_block() { return LANES > FORWARD_BLOCK ? LANES : FORWARD_BLOCK; }

// One row of a team, and the rows its workgroup's teams take in turn.
template <int DT, bool WIDE, int LANES, int V, bool KEEP>
__global__ __launch_bounds__(forward_block<LANES>(), 4) void forward_kernel(
    const typename Elem<DT>::storage *__restrict__ in,
    const typename Elem<weight_type<DT, WIDE>()>::storage *__restrict__ weight,
    const typename Elem<weight_type<DT, WIDE>()>::storage *__restrict__ bias, typename Elem<DT>::storage *__restrict__ out,
    uint8_t *__restrict__ codes, float *__restrict__ scales, float *__restrict__ stats, int32_t rows, int32_t d,
    float eps, const int32_t *__restrict__ live) {
    constexpr int WT = weight_type<DT, WIDE>();
    constexpr int TEAMS = forward_block<LANES>() / LANES, WAVES = LANES > 64 ? LANES / 64 : 1;
    __shared__ double slots[2][TEAMS][2 * WAVES];
    const uint32_t lane = threadIdx.x % LANES, team = threadIdx.x / LANES;
    const uint32_t live_rows = live != nullptr ? (uint32_t)clamp_live(live, rows) : (uint32_t)rows;
    const uint32_t step = gridDim.x * TEAMS;
    const uint32_t nb = ((uint32_t)d + BLOCK8 - 1) / BLOCK8;
    Oct<WT> w[V], b[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int c = (int)(v * LANES + lane) * 8;
        oct_load<WT, false>(w[v], weight + c, d - c);
        if (bias != nullptr) oct_load<WT, false>(b[v], bias + c, d - c);
        else oct_zero(b[v]);
    }
    Oct<DT> next[V];
    float next_first = 0.0f;
    auto load = [&](uint32_t row) {
        if (row >= live_rows) return;
        const typename Elem<DT>::storage *x = in + (size_t)row * d;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = (int)(v * LANES + lane) * 8;
            oct_load<DT>(next[v], x + c, d - c);
        }
        next_first = Elem<DT>::to_f32(x[0]);
    };
    load(blockIdx.x * TEAMS + team);
    int turn = 0;
    for (uint32_t base = blockIdx.x * TEAMS; base < live_rows; base += step) {  // the same for the workgroup
        const uint32_t row = base + team;
        Oct<DT> o[V];
#pragma unroll
        for (int v = 0; v < V; ++v) o[v] = next[v];
        const float first = next_first;
        load(row + step);
        double s1 = 0.0, s2 = 0.0;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int n = d - (int)(v * LANES + lane) * 8;
            float f[8];
            oct_unpack<DT>(o[v], f);
            if (n < 8) {
#pragma unroll
                for (int e = 0; e < 8; ++e) f[e] = e < n ? f[e] : first;
            }
            add_shifted<DT>(f, first, s1, s2);
        }
        team_sum2<LANES>(s1, s2, slots[turn][team]);
        turn ^= 1;
        if (row >= live_rows) continue;
        double m, var;
        shifted_moments(s1, s2, (double)first, (double)d, m, var);
        const RowOrigin<DT> mean(m);
        const float rstd = (float)(1.0 / __builtin_sqrt(var + (double)eps));
        if (lane == 0) {
            stats[2 * (size_t)row] = mean.hi;
            stats[2 * (size_t)row + 1] = rstd;
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = (int)(v * LANES + lane) * 8;
            const int n = d - c;
            const uint32_t block = (uint32_t)c / BLOCK8;
            if (block >= nb) continue;  // the same for the 16 lanes of a block
            float f[8], wf[8], bf[8];
            oct_unpack<DT>(o[v], f);
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = mean.from(f[e]);
            if constexpr (KEEP) {
                if (n < 8) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) f[e] = e < n ? f[e] : 0.0f;
                }
                float scale;
                const uint2 k = block_encode<difference_of<DT>(), false>(f, scale);
                codes_store(codes + (size_t)row * d + c, k, n);
                if ((lane & 15) == 0) scales[(size_t)row * nb + block] = scale;
            }
            oct_unpack<WT>(w[v], wf);
            oct_unpack<WT>(b[v], bf);
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = __builtin_fmaf(f[e] * rstd, wf[e], bf[e]);
            oct_store<DT>(out + (size_t)row * d + c, f, n);
        }
    }
}

// A workgroup of the backward: 16 wavefronts, one to a compute unit.
constexpr int BACK_BLOCK = 1024;

// What a team reads of a row, loaded one row ahead.
template <int DT, int V, bool KEPT> struct RowIn {
    Oct<DT> dy[V], x[KEPT ? 1 : V];
    uint2 k[KEPT ? V : 1];
    float scale[KEPT ? V : 1];
    float mean, rstd;
};

template <int DT, bool WIDE, int LANES, int V, bool KEPT>
__global__ __launch_bounds__(BACK_BLOCK) void backward_kernel(
    const typename Elem<DT>::storage *__restrict__ dout, const typename Elem<DT>::storage *__restrict__ in,
    const uint8_t *__restrict__ codes, const float *__restrict__ scales, const float *__restrict__ stats,
    const typename Elem<weight_type<DT, WIDE>()>::storage *__restrict__ weight, typename Elem<DT>::storage *__restrict__ dx,
    typename Elem<weight_type<DT, WIDE>()>::storage *__restrict__ dweight,
    typename Elem<weight_type<DT, WIDE>()>::storage *__restrict__ dbias, float *__restrict__ partial, int32_t rows,
    int32_t d, const int32_t *__restrict__ live) {
    constexpr int WT = weight_type<DT, WIDE>();
    constexpr int TEAMS = BACK_BLOCK / LANES, WAVES = BACK_BLOCK / 64;
    constexpr int TEAM_WAVES = LANES > 64 ? LANES / 64 : 1;
    constexpr int COLS = LANES > 64 ? 64 : LANES;  // lanes of a wave that own different columns
    // rows loaded one ahead where the registers allow it (128 a lane)
    constexpr bool AHEAD = V * (DT == DT_F32 ? 2 : 1) <= 2;
    __shared__ float slots[2][TEAMS][2 * TEAM_WAVES];
    __shared__ float parts[TEAMS > 1 ? WAVES * 16 * (COLS + 1) : 1];
    const uint32_t lane = threadIdx.x % LANES, team = threadIdx.x / LANES;
    const uint32_t live_rows = live != nullptr ? (uint32_t)clamp_live(live, rows) : (uint32_t)rows;
    const uint32_t step = gridDim.x * TEAMS;
    const uint32_t nb = ((uint32_t)d + BLOCK8 - 1) / BLOCK8;
    const float inv_d = 1.0f / (float)d;
    Oct<WT> w[V];
    float aw[V][8], ab[V][8];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int c = (int)(v * LANES + lane) * 8;
        oct_load<WT, false>(w[v], weight + c, d - c);
#pragma unroll
        for (int e = 0; e < 8; ++e) aw[v][e] = ab[v][e] = 0.0f;
    }
    auto load = [&](RowIn<DT, V, KEPT> &r, uint32_t row) {
        if (row >= live_rows) return;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = (int)(v * LANES + lane) * 8;
            const int n = d - c;
            oct_load<DT>(r.dy[v], dout + (size_t)row * d + c, n);
            if constexpr (KEPT) {
                r.k[v] = codes_load(codes + (size_t)row * d + c, n);
                r.scale[v] = n > 0 ? scales[(size_t)row * nb + (uint32_t)c / BLOCK8] : 0.0f;
            } else {
                oct_load<DT>(r.x[v], in + (size_t)row * d + c, n);
            }
        }
        r.mean = stats[2 * (size_t)row];
        r.rstd = stats[2 * (size_t)row + 1];
    };
    // dy and t (n = rstd t) of an octet; past the row's end dy is 0
    auto octet = [&](const RowIn<DT, V, KEPT> &r, int v, float (&dy)[8], float (&t)[8]) {
        oct_unpack<DT>(r.dy[v], dy);
        if constexpr (KEPT) {
            block_decode(r.k[v], r.scale[v], t);
        } else {
            oct_unpack<DT>(r.x[v], t);
#pragma unroll
            for (int e = 0; e < 8; ++e) t[e] -= r.mean;
        }
    };
    RowIn<DT, V, KEPT> r, next;
    if constexpr (AHEAD) load(next, blockIdx.x * TEAMS + team);
    int turn = 0;
    for (uint32_t base = blockIdx.x * TEAMS; base < live_rows; base += step) {  // the same for the workgroup
        const uint32_t row = base + team;
        if constexpr (AHEAD) {
            r = next;
            load(next, row + step);
        } else {
            load(r, row);
        }
        float s1 = 0.0f, s2 = 0.0f;
        if (row < live_rows) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float dy[8], t[8], wf[8];
                octet(r, v, dy, t);
                oct_unpack<WT>(w[v], wf);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float n = t[e] * r.rstd, dv = dy[e] * wf[e];
                    s1 += dv;
                    s2 = __builtin_fmaf(dv, n, s2);
                    ab[v][e] += dy[e];
                    aw[v][e] = __builtin_fmaf(dy[e], n, aw[v][e]);
                }
            }
        }
        team_sum2<LANES>(s1, s2, slots[turn][team]);
        turn ^= 1;
        if (row >= live_rows) continue;
        const float m1 = s1 * inv_d, m2 = s2 * inv_d * r.rstd;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = (int)(v * LANES + lane) * 8;
            float dy[8], t[8], wf[8];
            octet(r, v, dy, t);
            oct_unpack<WT>(w[v], wf);
#pragma unroll
            for (int e = 0; e < 8; ++e) dy[e] = r.rstd * (dy[e] * wf[e] - __builtin_fmaf(t[e], m2, m1));
            if (c < d) oct_store<DT>(dx + (size_t)row * d + c, dy, d - c);
        }
    }
    // one workgroup in all: its sums are the gradients
    const bool last = gridDim.x == 1;
    float *pw = partial + (size_t)blockIdx.x * 2 * d, *pb = pw + d;
    auto put = [&](int which, int col, float v) {
        if (last) {
            if (which == 0) dweight[col] = Elem<WT>::from_f32(v);
            else if (dbias != nullptr) dbias[col] = Elem<WT>::from_f32(v);
        } else {
            (which == 0 ? pw : pb)[col] = v;
        }
    };
    if constexpr (TEAMS == 1) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = (int)(v * LANES + lane) * 8;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if (c + e < d) {
                    put(0, c + e, aw[v][e]);
                    put(1, c + e, ab[v][e]);
                }
            }
        }
    } else {
        // the teams' sums, wave by wave (a 16-lane team's wave adds its four first)
        const uint32_t wave = threadIdx.x / 64, wl = threadIdx.x & 63;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            __syncthreads();
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float a = aw[v][e], b = ab[v][e];
                if constexpr (LANES == 16) {
                    a += __shfl_xor(a, 16);
                    b += __shfl_xor(b, 16);
                    a += __shfl_xor(a, 32);
                    b += __shfl_xor(b, 32);
                }
                if (wl < COLS) {
                    parts[(wave * 16 + e) * (COLS + 1) + wl] = a;
                    parts[(wave * 16 + 8 + e) * (COLS + 1) + wl] = b;
                }
            }
            __syncthreads();
            // WAVES / TEAM_WAVES waves hold each of the team's 64 TEAM_WAVES lanes
            constexpr uint32_t WIDTH = TEAM_WAVES * COLS * 8;
            for (uint32_t i = threadIdx.x; i < 2 * WIDTH; i += BACK_BLOCK) {
                const uint32_t which = i / WIDTH, at = i % WIDTH;
                const uint32_t e = at % 8, cl = at / 8;  // element, lane of the team
                float t = 0.0f;
#pragma unroll
                for (int g = 0; g < WAVES / TEAM_WAVES; ++g)
                    t += parts[((g * TEAM_WAVES + cl / COLS) * 16 + which * 8 + e) * (COLS + 1) + cl % COLS];
                const int col = (int)(v * LANES + cl) * 8 + (int)e;
                if (col < d) put((int)which, col, t);
            }
        }
    }
}

// Columns of [groups, 2 d] partials, 32 to a workgroup, 16 slices of the
// groups each, added slice by slice in order.
constexpr int REDUCE_COLS = 32, REDUCE_SLICES = 16;

template <int WT>
__global__ __launch_bounds__(REDUCE_COLS *REDUCE_SLICES) void reduce_kernel(
    const float *__restrict__ partial, typename Elem<WT>::storage *__restrict__ dweight,
    typename Elem<WT>::storage *__restrict__ dbias, int32_t groups, int32_t d) {
    __shared__ float sums[REDUCE_SLICES][REDUCE_COLS];
    const int col = (int)blockIdx.x * REDUCE_COLS + (int)(threadIdx.x % REDUCE_COLS);
    const int slice = threadIdx.x / REDUCE_COLS;
    const int width = 2 * d;
    float t = 0.0f;
    if (col < width) {
#pragma unroll 8
        for (int g = slice; g < groups; g += REDUCE_SLICES) t += partial[(size_t)g * width + col];
    }
    sums[slice][threadIdx.x % REDUCE_COLS] = t;
    __syncthreads();
    if (slice != 0 || col >= width) return;
#pragma unroll
    for (int s = 1; s < REDUCE_SLICES; ++s) t += sums[s][threadIdx.x];
    if (col < d) dweight[col] = Elem<WT>::from_f32(t);
    else if (dbias != nullptr) dbias[col - d] = Elem<WT>::from_f32(t);
}

struct Forward {
    const void *in, *weight, *bias;
    void *out, *codes;
    float *scales, *stats;
    int32_t rows, d;
    float eps;
    const int32_t *live;
    int cus;
    hipStream_t stream;
};

constexpr int FORWARD_HELD = 1024;  // threads of a compute unit

template <int DT, bool WIDE, int LANES, int V>
hipError_t forward_as(const Forward &a) {
    using S = typename Elem<DT>::storage;
    using WS = typename Elem<weight_type<DT, WIDE>()>::storage;
    constexpr int BLOCK = forward_block<LANES>(), TEAMS = BLOCK / LANES;
    // as many workgroups as the device holds at four wavefronts a SIMD
    const int64_t need = ((int64_t)a.rows + TEAMS - 1) / TEAMS, most = (int64_t)a.cus * (FORWARD_HELD / BLOCK);
    const dim3 grid((uint32_t)(need < most ? need : most)), block(BLOCK);
    if (a.codes != nullptr)
        forward_kernel<DT, WIDE, LANES, V, true><<<grid, block, 0, a.stream>>>(
            (const S *)a.in, (const WS *)a.weight, (const WS *)a.bias, (S *)a.out, (uint8_t *)a.codes, a.scales,
            a.stats, a.rows, a.d, a.eps, a.live);
    else
        forward_kernel<DT, WIDE, LANES, V, false><<<grid, block, 0, a.stream>>>(
            (const S *)a.in, (const WS *)a.weight, (const WS *)a.bias, (S *)a.out, nullptr, nullptr, a.stats, a.rows,
            a.d, a.eps, a.live);
    return hipGetLastError();
}

template <int DT, bool WIDE>
hipError_t forward_dt(const Forward &a) {
    return by_width(a.d, [&](auto t) { return forward_as<DT, WIDE, decltype(t)::LANES, decltype(t)::V>(a); });
}

struct Backward {
    const void *dout, *in, *codes;
    const float *scales, *stats;
    const void *weight;
    void *dx, *dweight, *dbias;
    bool kept;
    int32_t rows, d;
    const int32_t *live;
    int groups;
    float *workspace;
    hipStream_t stream;
};

template <int DT, bool WIDE, int LANES, int V>
hipError_t backward_as(const Backward &a) {
    using S = typename Elem<DT>::storage;
    constexpr int WT = weight_type<DT, WIDE>();
    using WS = typename Elem<WT>::storage;
    const dim3 grid((uint32_t)a.groups), block(BACK_BLOCK);
    if (!a.kept)
        backward_kernel<DT, WIDE, LANES, V, false><<<grid, block, 0, a.stream>>>(
            (const S *)a.dout, (const S *)a.in, nullptr, nullptr, a.stats, (const WS *)a.weight, (S *)a.dx,
            (WS *)a.dweight, (WS *)a.dbias, a.workspace, a.rows, a.d, a.live);
    else
        backward_kernel<DT, WIDE, LANES, V, true><<<grid, block, 0, a.stream>>>(
            (const S *)a.dout, nullptr, (const uint8_t *)a.codes, a.scales, a.stats, (const WS *)a.weight, (S *)a.dx,
            (WS *)a.dweight, (WS *)a.dbias, a.workspace, a.rows, a.d, a.live);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.groups == 1) return e;
    reduce_kernel<WT><<<dim3((uint32_t)((2 * a.d + REDUCE_COLS - 1) / REDUCE_COLS)),
                        dim3(REDUCE_COLS * REDUCE_SLICES), 0, a.stream>>>(a.workspace, (WS *)a.dweight, (WS *)a.dbias,
                                                                          a.groups, a.d);
    return hipGetLastError();
}

template <int DT, bool WIDE>
hipError_t backward_dt(const Backward &a) {
    return by_width(a.d, [&](auto t) { return backward_as<DT, WIDE, decltype(t)::LANES, decltype(t)::V>(a); });
}

}  // namespace

int layer_norm_groups(int64_t rows, int64_t d, int cus) {
    const int64_t teams = by_width(d, [](auto t) { return (int64_t)(BACK_BLOCK / decltype(t)::LANES); });
    const int64_t need = (rows + teams - 1) / teams;
    return (int)(need < 1 ? 1 : need < cus ? need : cus);
}

hipError_t launch_layer_norm(int dtype, bool wide, const void *in, const void *weight, const void *bias, void *out,
                             void *codes, float *scales, float *stats, int32_t rows, int32_t d, float eps,
                             const int32_t *live, int cus, hipStream_t stream) {
    const Forward a{in, weight, bias, out, codes, scales, stats, rows, d, eps, live, cus, stream};
    switch (dtype) {
    case DT_F32: return forward_dt<DT_F32, true>(a);
    case DT_F16: return wide ? forward_dt<DT_F16, true>(a) : forward_dt<DT_F16, false>(a);
    case DT_BF16: return wide ? forward_dt<DT_BF16, true>(a) : forward_dt<DT_BF16, false>(a);
    default: return hipErrorInvalidValue;
    }
}

hipError_t launch_layer_norm_backward(int dtype, bool wide, const void *dout, const void *in, const void *codes,
                                      const float *scales, const float *stats, const void *weight, void *dx,
                                      void *dweight, void *dbias, bool kept, int32_t rows, int32_t d,
                                      const int32_t *live, int groups, float *workspace, hipStream_t stream) {
    const Backward a{dout, in, codes, scales, stats, weight, dx, dweight, dbias, kept, rows, d, live, groups,
                     workspace, stream};
    switch (dtype) {
    case DT_F32: return backward_dt<DT_F32, true>(a);
    case DT_F16: return wide ? backward_dt<DT_F16, true>(a) : backward_dt<DT_F16, false>(a);
    case DT_BF16: return wide ? backward_dt<DT_BF16, true>(a) : backward_dt<DT_BF16, false>(a);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace ga
