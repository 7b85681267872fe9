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
// m comes as an fp32 number.  Where the mean is far above the spread its
// rounding would be in every n of a row (3.75e-3 at mean 65536.3 and spread 1),
// so the backward from x also sums x - m over the row and takes the mean of that
// off again (off_centre).
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
// partials at 8 d bytes times 256 (two per compute unit: 8192 x 4096 from codes
// 39.9 us, 33.6 us with one, fastest of a trace).
//
// Measured (medians of a kernel trace): forward 16384 x 2048 bf16 (134 MB) 25.1 us,
// 5.4 TB/s; with codes 8192 x 4096 (169 MB) 35.4 us, 4.8 TB/s; backward from codes
// 33.9 us and 4.6 us for the sums (169 MB, 4.4 TB/s); backward from x, 4096 x 4096
// fp32 (201 MB) 42.4 us and 4.7 us, 4.3 TB/s; 4001 x 1027 fp32 (49 MB) 16.3 us and
// 4.0 us: 1027 columns are 129 octets on a team of 256 lanes, the lanes past them
// load and store the row's last octet again, and the sums' launch is latency.
#include <type_traits>

#include "ga_internal.h"
#include "ga_train.h"

namespace ga {

namespace {

// fp32 weights where WIDE, else the rows' type.
template <int DT, bool WIDE> constexpr int weight_type() { return WIDE ? DT_F32 : DT; }

// The team of a row by its width: LANES lanes of V octets.  Two octets a lane
// halve what the row's reductions cost a value; a row of up to 1024 values is
// a wavefront's own and needs no barrier.  Four octets a lane for the forward
// took 34.7 us for 38.2 at 4096 x 8192 bf16 with codes, but 35.4 for 34.3 at
// 4096 columns, 33.6 for 32.9 at 2048, and 3.0 for 2.4 for a single row (medians).
template <int LANES_, int V_, bool TINY_ = false> struct Team {
    static constexpr int LANES = LANES_, V = V_;
    static constexpr bool TINY = TINY_;  // rows of fewer than eight values
};

template <typename F>
auto by_width(int64_t d, F &&f) {
    if (d < 8) return f(Team<16, 1, true>());
    if (d <= 128) return f(Team<16, 1>());
    if (d <= 512) return f(Team<64, 1>());
    if (d <= 1024) return f(Team<64, 2>());
    if (d <= 2048) return f(Team<128, 2>());
    if (d <= 4096) return f(Team<256, 2>());
    if (d <= 8192) return f(Team<512, 2>());
    if (d <= 16384) return f(Team<1024, 2>());
    return f(Team<1024, 4>());
}

constexpr int FORWARD_BLOCK = 128;  // workgroups of several teams; a larger team is one by itself
template <int LANES> constexpr int forward_block() { return LANES > FORWARD_BLOCK ? LANES : FORWARD_BLOCK; }

// One row to a team.  Rows come and go with the workgroups, so a wavefront's
// stores never hold up a load; all of a row's loads are issued at once.
template <int DT, bool WIDE, typename T, bool KEEP>
__global__ __launch_bounds__(forward_block<T::LANES>()) void forward_kernel(
    const typename Elem<DT>::storage *__restrict__ in,
    const typename Elem<weight_type<DT, WIDE>()>::storage *__restrict__ weight,
    const typename Elem<weight_type<DT, WIDE>()>::storage *__restrict__ bias, typename Elem<DT>::storage *__restrict__ out,
    uint8_t *__restrict__ codes, float *__restrict__ scales, float *__restrict__ stats, int32_t rows, int32_t d,
    float eps, double inv_d, const int32_t *__restrict__ live) {
    constexpr int WT = weight_type<DT, WIDE>();
    constexpr int LANES = T::LANES, V = T::V;
    constexpr bool TINY = T::TINY;
    constexpr int TEAMS = forward_block<LANES>() / LANES, WAVES = LANES > 64 ? LANES / 64 : 1;
    __shared__ double slots[TEAMS][2 * WAVES];
    const uint32_t lane = threadIdx.x % LANES, team = threadIdx.x / LANES;
    const uint32_t live_rows = live != nullptr ? (uint32_t)clamp_live(live, rows) : (uint32_t)rows;
    const uint32_t nb = ((uint32_t)d + BLOCK8 - 1) / BLOCK8;
    if (blockIdx.x * TEAMS >= live_rows) return;
    const bool mine = blockIdx.x * TEAMS + team < live_rows;  // a team without a row follows the last one
    const uint32_t row = team_row<LANES>(mine ? blockIdx.x * TEAMS + team : live_rows - 1);
    const typename Elem<DT>::storage *x = in + (size_t)row * d;
    Oct<DT> o[V];
    Oct<WT> w[V], b[V];
#pragma unroll
    for (int v = 0; v < V; ++v) oct_fetch<DT, TINY>(o[v], x, (int)(v * LANES + lane) * 8, d);
    const float first = row_pivot<DT>(x, d);
#pragma unroll
    for (int v = 0; v < V; ++v) {
        oct_fetch<WT, TINY, false>(w[v], weight, (int)(v * LANES + lane) * 8, d);
        oct_fetch<WT, TINY, false>(b[v], bias != nullptr ? bias : weight, (int)(v * LANES + lane) * 8, d);
    }
    double s1 = 0.0, s2 = 0.0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int c = (int)(v * LANES + lane) * 8;
        const int n = d - c;
        float f[8];
        oct_trim<DT, TINY>(o[v], c, d);
        oct_unpack<DT>(o[v], f);
        if (n < 8) {
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = e < n ? f[e] : first;
        }
        add_shifted(f, first, s1, s2);
    }
    team_sum2<LANES>(s1, s2, slots[team]);
    if (!mine) return;
    double m, var;
    shifted_moments(s1, s2, (double)first, inv_d, m, var);
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
            codes_store(codes + (size_t)row * d + (uint32_t)c, k, n);
            if ((lane & 15) == 0) scales[(size_t)row * nb + block] = scale;
        }
        oct_trim<WT, TINY>(w[v], c, d);
        oct_unpack<WT>(w[v], wf);
        if (bias != nullptr) {
            oct_trim<WT, TINY>(b[v], c, d);
            oct_unpack<WT>(b[v], bf);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) bf[e] = 0.0f;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = __builtin_fmaf(f[e] * rstd, wf[e], bf[e]);
        oct_store<DT>(out + (size_t)row * d + (uint32_t)c, f, n);
    }
}

// A workgroup of the backward: eight wavefronts of up to 256 registers, one
// workgroup to a compute unit.
constexpr int BACK_BLOCK = 512;

// fp32 rows up to 4096 values: one octet a lane, which leaves the registers to
// load a row ahead (4001 rows of 1027, fastest of a trace: 15.3 us, 17.8 us with two
// octets and none ahead).
template <bool F32, typename F>
auto by_width_backward(int64_t d, F &&f) {
    constexpr int V = F32 ? 1 : 2;
    if (d < 8) return f(Team<16, 1, true>());
    if (d <= 128) return f(Team<16, 1>());
    if (d <= 512) return f(Team<64, 1>());
    if (d <= 1024) return f(Team<128 / V, V>());
    if (d <= 2048) return f(Team<256 / V, V>());
    if (d <= 4096) return f(Team<512 / V, V>());
    return f(Team<512, 2>());
}

// Rows wider than a workgroup's 512 lanes of two octets are cut into strips and
// read twice.  SUMS leaves each 8192-column strip's part of a row's sums in
// the workspace; APPLY adds a row's parts and does the rest for strips of 1024
// columns, a wavefront to a row, so that a workgroup adds up eight rows and few
// partials are left.  (Fastest of a trace: four and eight octets a lane, one pass,
// spilled: 2048 rows of 16384, bf16 from codes, took 80 us, 1024 rows of 32768 414 us, against
// 52 us either way; APPLY in strips of 8192 columns took 33 us for 311 rows of
// 20897, from x, against 23 us.)
enum Stage { WHOLE, SUMS, APPLY };
using SumsTeam = Team<512, 2>;
using ApplyTeam = Team<64, 2>;
template <typename T> constexpr int64_t strips_of(int64_t d) {
    return (d + T::LANES * T::V * 8 - 1) / (T::LANES * T::V * 8);
}
constexpr int ROW_SUMS = 3;  // floats of a row and strip, at most
inline bool in_strips(int64_t d) { return strips_of<SumsTeam>(d) > 1; }

// Rows a team has in flight beside the one it works on, as the registers allow.
template <int DT, int V> constexpr int rows_ahead() { return V * (DT == DT_F32 ? 2 : 1) <= 2 ? 1 : 0; }

// The row's mean less the fp32 m it came as, from the sum of x - m.  Taken where
// |m| r > 4, with n off by at most 2^-22 otherwise, of the order of the other
// roundings of n; a sum of more than m's rounding can leave (and a few roundings
// of a mean that was itself summed in fp32) means that m is not meant to be the
// row's mean, and m is used as it is.
__device__ __forceinline__ float off_centre(float sum, float inv_d, float m, float r) {
    const float off = sum * inv_d, size = __builtin_fabsf(m);
    return size * r > 4.0f && __builtin_fabsf(off) <= 0x1p-22f * size ? off : 0.0f;
}

// What a team reads of a row.
template <int DT, int V, bool KEPT> struct RowIn {
    Oct<DT> dy[V], x[KEPT ? 1 : V];
    uint2 k[KEPT ? V : 1];
    float scale[KEPT ? V : 1], before[KEPT ? V : 1];  // of the octet's block, and of its first element's
    float mean, rstd;
};

// The loop over rows has no branch around a load or a store: such a branch
// makes the compiler wait for all of them wherever its paths meet, the stores
// of the row before among them.  A lane whose octet passes the row's end works
// on the row's last eight values instead: those of them that other lanes own
// are left out of the sums, and stored with the very bits their owners store.
// A team past the last row does that row again, out of the columns' sums.
template <int DT, bool WIDE, typename T, bool KEPT, Stage STAGE>
__global__ __launch_bounds__(BACK_BLOCK, 2) void backward_kernel(
    const typename Elem<DT>::storage *__restrict__ dout, const typename Elem<DT>::storage *__restrict__ in,
    const uint8_t *__restrict__ codes, const float *__restrict__ scales, const float *__restrict__ stats,
    const typename Elem<weight_type<DT, WIDE>()>::storage *__restrict__ weight, typename Elem<DT>::storage *__restrict__ dx,
    typename Elem<weight_type<DT, WIDE>()>::storage *__restrict__ dweight,
    typename Elem<weight_type<DT, WIDE>()>::storage *__restrict__ dbias, float *__restrict__ partial,
    float *__restrict__ row_sums, int32_t rows, int32_t d, const int32_t *__restrict__ live) {
    constexpr int WT = weight_type<DT, WIDE>();
    constexpr int LANES = T::LANES, V = T::V;
    constexpr bool TINY = T::TINY;
    constexpr int TEAMS = BACK_BLOCK / LANES, WAVES = BACK_BLOCK / 64;
    constexpr int TEAM_WAVES = LANES > 64 ? LANES / 64 : 1;
    constexpr int COLS = LANES > 64 ? 64 : LANES;  // lanes of a wave that own different columns
    constexpr int AHEAD = rows_ahead<DT, V>();
    constexpr int SUMMED = KEPT ? 2 : 3;
    __shared__ float slots[2][TEAMS][SUMMED * TEAM_WAVES];
    __shared__ float parts[TEAMS > 1 ? WAVES * 16 * (COLS + 1) : 1];
    const uint32_t lane = threadIdx.x % LANES, team = threadIdx.x / LANES;
    const uint32_t live_rows = live != nullptr ? (uint32_t)clamp_live(live, rows) : (uint32_t)rows;
    // workgroups are numbered by group and strip
    const uint32_t strips = STAGE == WHOLE ? 1 : (uint32_t)strips_of<T>(d);
    const uint32_t strip = STAGE == WHOLE ? 0 : blockIdx.x % strips;
    const uint32_t group = STAGE == WHOLE ? blockIdx.x : blockIdx.x / strips;
    const uint32_t groups = STAGE == WHOLE ? gridDim.x : gridDim.x / strips;
    const int left = STAGE == WHOLE ? 0 : (int)strip * (LANES * V * 8);  // the strip's first column
    auto column = [&](int v) { return left + (int)(v * LANES + lane) * 8; };
    const uint32_t step = groups * TEAMS;
    const uint32_t nb = ((uint32_t)d + BLOCK8 - 1) / BLOCK8;
    const float inv_d = 1.0f / (float)d;
    Oct<WT> w[V];
    float aw[V][8], ab[V][8];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int c = column(v);
        oct_fetch<WT, TINY, false>(w[v], weight, c, d);
#pragma unroll
        for (int e = 0; e < 8; ++e) aw[v][e] = ab[v][e] = 0.0f;
    }
    auto load = [&](RowIn<DT, V, KEPT> &r, uint32_t row) {
        row = team_row<LANES>(row < live_rows ? row : live_rows - 1);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = column(v);
            oct_fetch<DT, TINY>(r.dy[v], dout + (size_t)row * d, c, d);
            if constexpr (KEPT) {
                const uint32_t at = (uint32_t)(TINY || c < d - 8 ? c : d - 8), last = nb - 1;
                const uint32_t block = (uint32_t)c / BLOCK8 < last ? (uint32_t)c / BLOCK8 : last;
                r.k[v] = codes_fetch<TINY>(codes + (size_t)row * d, c, d);
                r.scale[v] = scales[(size_t)row * nb + block];
                r.before[v] = TINY ? 0.0f : scales[(size_t)row * nb + at / BLOCK8];
            } else {
                oct_fetch<DT, TINY>(r.x[v], in + (size_t)row * d, c, d);
            }
        }
        r.mean = stats[2 * (size_t)row];
        r.rstd = stats[2 * (size_t)row + 1];
    };
    // dy and t (n = rstd t) of an octet
    auto octet = [&](const RowIn<DT, V, KEPT> &r, int v, float (&dy)[8], float (&t)[8]) {
        oct_unpack<DT>(r.dy[v], dy);
        if constexpr (KEPT) {
            block_decode(r.k[v], r.scale[v], t);
            // a last eight that begin in the block before the row's last
            const int c = column(v), edge = (int)(nb - 1) * BLOCK8 - (d - 8);
            if (!TINY && edge > 0 && c > d - 8) {
                float u[8];
                block_decode(r.k[v], r.before[v], u);
#pragma unroll
                for (int e = 0; e < 8; ++e) t[e] = e < edge ? u[e] : t[e];
            }
        } else {
            oct_unpack<DT>(r.x[v], t);
#pragma unroll
            for (int e = 0; e < 8; ++e) t[e] -= r.mean;
        }
    };
    auto dropped = [&](int v) {
        const int s = column(v) - (d - 8);
        return TINY || s < 0 ? 0 : s < 8 ? s : 8;
    };
    RowIn<DT, V, KEPT> r, next[AHEAD > 0 ? AHEAD : 1];
    if (live_rows > 0) {
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) load(next[i], (group + i * groups) * TEAMS + team);
    }
    int turn = 0;
    for (uint32_t base = group * TEAMS; base < live_rows; base += step) {  // the same for the workgroup
        const bool mine = base + team < live_rows;
        const uint32_t row = team_row<LANES>(mine ? base + team : live_rows - 1);
        if constexpr (AHEAD > 0) {
            r = next[0];
#pragma unroll
            for (int i = 1; i < AHEAD; ++i) next[i - 1] = next[i];
            load(next[AHEAD - 1], base + team + AHEAD * step);
        } else {
            load(r, row);
        }
        float s[SUMMED] = {};  // of dy w, of dy w n and, from x, of x - m
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int drop = dropped(v);  // elements that are other lanes'
            float dy[8], t[8], wf[8];
            octet(r, v, dy, t);
            oct_unpack<WT>(w[v], wf);
            if (drop > 0) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    dy[e] = e < drop ? 0.0f : dy[e];
                    t[e] = e < drop ? 0.0f : t[e];
                }
            }
            float a[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float n = t[e] * r.rstd, dv = dy[e] * wf[e];
                s[0] += dv;
                s[1] = __builtin_fmaf(dv, n, s[1]);
                if constexpr (!KEPT) s[2] += TINY && column(v) + e >= d ? 0.0f : t[e];
                a[e] = n;
            }
            if (STAGE != SUMS && mine) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    ab[v][e] += dy[e];
                    aw[v][e] = __builtin_fmaf(dy[e], a[e], aw[v][e]);
                }
            }
        }
        if constexpr (STAGE == APPLY) {
            const uint32_t parts_of_row = (uint32_t)strips_of<SumsTeam>(d);
            const float *part = row_sums + (size_t)row * parts_of_row * SUMMED;
#pragma unroll
            for (int k = 0; k < SUMMED; ++k) s[k] = 0.0f;
            for (uint32_t i = 0; i < parts_of_row; ++i, part += SUMMED) {
#pragma unroll
                for (int k = 0; k < SUMMED; ++k) s[k] += part[k];
            }
        } else {
            team_sums<LANES>(s, slots[turn][team]);
            turn ^= 1;
        }
        if constexpr (STAGE == SUMS) {
            if (lane == 0) {
                float *part = row_sums + ((size_t)row * strips + strip) * SUMMED;
#pragma unroll
                for (int k = 0; k < SUMMED; ++k) part[k] = s[k];
            }
            continue;
        }
        float off = 0.0f;
        if constexpr (!KEPT) {
            off = off_centre(s[2], inv_d, r.mean, r.rstd);
            if (off != 0.0f) s[1] = __builtin_fmaf(-off * r.rstd, s[0], s[1]);
        }
        const float m1 = s[0] * inv_d, m2 = s[1] * inv_d * r.rstd;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = column(v);
            float dy[8], t[8], wf[8];
            octet(r, v, dy, t);
            oct_unpack<WT>(w[v], wf);
            if (!KEPT && off != 0.0f) {
                const int drop = mine ? dropped(v) : 8;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    t[e] -= off;
                    aw[v][e] = __builtin_fmaf(e < drop ? 0.0f : dy[e], -off * r.rstd, aw[v][e]);
                }
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) dy[e] = r.rstd * (dy[e] * wf[e] - __builtin_fmaf(t[e], m2, m1));
            if constexpr (TINY) oct_store<DT>(dx + (size_t)row * d + (uint32_t)c, dy, d - c);
            else oct_store<DT>(dx + (size_t)row * d + (uint32_t)(c < d - 8 ? c : d - 8), dy, 8);
        }
    }
    if constexpr (STAGE == SUMS) return;
    // one group in all: its sums are the gradients
    const bool last = groups == 1;
    float *pw = partial + (size_t)group * 2 * d, *pb = pw + d;
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
            const int c = column(v), drop = dropped(v), at = c < d - 8 ? c : d - 8;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if (e >= drop) {
                    put(0, at + e, aw[v][e]);
                    put(1, at + e, ab[v][e]);
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
                const int c = left + (int)(v * LANES + cl) * 8, drop = TINY ? 0 : c - (d - 8);
                const int col = (drop > 0 ? d - 8 : c) + (int)e;
                if ((int)e >= drop && col < d) put((int)which, col, t);
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
    hipStream_t stream;
};

template <int DT, bool WIDE, typename T>
hipError_t forward_as(const Forward &a) {
    using S = typename Elem<DT>::storage;
    using WS = typename Elem<weight_type<DT, WIDE>()>::storage;
    constexpr int BLOCK = forward_block<T::LANES>(), TEAMS = BLOCK / T::LANES;
    const dim3 grid((uint32_t)(((int64_t)a.rows + TEAMS - 1) / TEAMS)), block(BLOCK);
    const auto kernel = a.codes != nullptr ? forward_kernel<DT, WIDE, T, true> : forward_kernel<DT, WIDE, T, false>;
    return launch_kernel(kernel, grid, block, a.stream, (const S *)a.in, (const WS *)a.weight, (const WS *)a.bias,
                         (S *)a.out, (uint8_t *)a.codes, a.scales, a.stats, a.rows, a.d, a.eps, 1.0 / a.d, a.live);
}

template <int DT, bool WIDE>
hipError_t forward_dt(const Forward &a) {
    return by_width(a.d, [&](auto t) { return forward_as<DT, WIDE, decltype(t)>(a); });
}

struct Backward {
    const void *dout, *in, *codes;
    const float *scales, *stats;
    const void *weight;
    void *dx, *dweight, *dbias;
    bool kept;
    int32_t rows, d;
    const int32_t *live;
    int groups, cus;
    float *workspace;
    hipStream_t stream;
};

template <int DT, bool WIDE, typename T>
hipError_t backward_as(const Backward &a) {
    using S = typename Elem<DT>::storage;
    constexpr int WT = weight_type<DT, WIDE>();
    using WS = typename Elem<WT>::storage;
    const bool wide = in_strips(a.d);
    float *row_sums = a.workspace;
    float *partial = a.workspace + (wide ? ROW_SUMS * strips_of<SumsTeam>(a.d) * a.rows : 0);
    auto launch = [&](auto kept, auto team, auto stage, int64_t grid) {
        return launch_kernel(backward_kernel<DT, WIDE, decltype(team), decltype(kept)::value, decltype(stage)::value>,
                             dim3((uint32_t)grid), dim3(BACK_BLOCK), a.stream, (const S *)a.dout, (const S *)a.in,
                             (const uint8_t *)a.codes, a.scales, a.stats, (const WS *)a.weight, (S *)a.dx,
                             (WS *)a.dweight, (WS *)a.dbias, partial, row_sums, a.rows, a.d, a.live);
    };
    auto launches = [&](auto kept) {
        if constexpr (std::is_same<T, SumsTeam>::value) {
            if (wide) {
                // two workgroups to a compute unit: no sums over rows here
                const int64_t strips = strips_of<T>(a.d), most = 2 * a.cus / strips, rows = a.rows < 1 ? 1 : a.rows;
                const hipError_t e = launch(kept, T(), std::integral_constant<Stage, SUMS>(),
                                            strips * (rows < most ? rows : most));
                if (e != hipSuccess) return e;
                return launch(kept, ApplyTeam(), std::integral_constant<Stage, APPLY>(),
                              strips_of<ApplyTeam>(a.d) * a.groups);
            }
        }
        return launch(kept, T(), std::integral_constant<Stage, WHOLE>(), a.groups);
    };
    const hipError_t e = a.kept ? launches(std::true_type()) : launches(std::false_type());
    if (e != hipSuccess || a.groups == 1) return e;
    return launch_kernel(reduce_kernel<WT>, dim3((uint32_t)((2 * a.d + REDUCE_COLS - 1) / REDUCE_COLS)),
                         dim3(REDUCE_COLS * REDUCE_SLICES), a.stream, partial, (WS *)a.dweight, (WS *)a.dbias, a.groups,
                         a.d);
}

template <int DT, bool WIDE>
hipError_t backward_dt(const Backward &a) {
    return by_width_backward<DT == DT_F32>(a.d, [&](auto t) { return backward_as<DT, WIDE, decltype(t)>(a); });
}

}  // namespace

int layer_norm_lanes(int64_t d) {
    return by_width(d, [](auto t) { return decltype(t)::LANES; });
}

int layer_norm_groups(int64_t rows, int64_t d, bool f32, int cus) {
    auto teams_of = [](auto t) { return (int64_t)(BACK_BLOCK / decltype(t)::LANES); };
    const int64_t teams = f32 ? by_width_backward<true>(d, teams_of) : by_width_backward<false>(d, teams_of);
    const int64_t strips = in_strips(d) ? strips_of<ApplyTeam>(d) : 1;
    const int64_t of = in_strips(d) ? BACK_BLOCK / ApplyTeam::LANES : teams;
    const int64_t need = (rows + of - 1) / of, most = cus > strips ? cus / strips : 1;
    return (int)(need < 1 ? 1 : need < most ? need : most);
}

size_t layer_norm_workspace_bytes(int64_t rows, int64_t d, int groups) {
    return (groups > 1 ? (size_t)groups * 2 * (size_t)d * 4 : 0) +
           (in_strips(d) ? (size_t)rows * (size_t)strips_of<SumsTeam>(d) * ROW_SUMS * 4 : 0);
}

hipError_t launch_layer_norm(int dtype, bool wide, const void *in, const void *weight, const void *bias, void *out,
                             void *codes, float *scales, float *stats, int32_t rows, int32_t d, float eps,
                             const int32_t *live, hipStream_t stream) {
    const Forward a{in, weight, bias, out, codes, scales, stats, rows, d, eps, live, stream};
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
                                      const int32_t *live, int groups, int cus, float *workspace, hipStream_t stream) {
    const Backward a{dout, in, codes, scales, stats, weight, dx, dweight, dbias, kept, rows, d, live, groups, cus,
                     workspace, stream};
    switch (dtype) {
    case DT_F32: return backward_dt<DT_F32, true>(a);
    case DT_F16: return wide ? backward_dt<DT_F16, true>(a) : backward_dt<DT_F16, false>(a);
    case DT_BF16: return wide ? backward_dt<DT_BF16, true>(a) : backward_dt<DT_BF16, false>(a);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace ga
