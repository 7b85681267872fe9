// The feed-forward layer's product for few tokens (gfx950): device code shared
// by the 16-bit and the microscaled 4-bit kernels.
//
//   D[f, t] = sum over k of A[f, k] B[t, k],  at most 4 NT tokens
//
// Every weight is used for a few tokens once, so the call is bound by the
// weights' bytes and the work is to keep many of them in flight on every compute
// unit.  A workgroup owns 4 NF FG rows of A (half of them gate and half up rows
// where D has two halves) over all of k: 8 / FG wavefronts share 4 NF of them and
// take the units of 256 bytes of a row in turn, each lane 16 bytes of them
// straight into the registers that the matrix cores read, a unit ahead.  No
// barrier and no branch in the loop: what lies past a row's end, the last feature
// or the last live token is read past a buffer descriptor's end, as zero.
// Measured: bf16 one token, 2 * 16384 features of 2048 26 us and 2048 of 16384 13
// us, 5.1 TB/s both; 4 bits, four tokens, 2 * 16384 of 4096 12.4 us, 5.7 TB/s.
// One unit of each wavefront is in flight: two or more take registers, and with
// them wavefronts, and measured the same or slower.
//
// The 16 rows of a matrix instruction are four features, each over four parts of
// k: row 4 f + q holds the chunks q of 16 bytes in every 64 of feature f's row, so
// the lanes of a load hold 256 bytes of four rows, neighbours next to each other.
// (One feature a row puts every lane of a quad into another row: four times the
// address lookups, which then bound the call: 2048 features of 16384 bf16, one
// token, 21.4-24 us, 15.4 so.)  Columns are four tokens in the same
// parts, and of the result the four diagonal entries of a feature and a token, one
// for each part, are wanted: a lane picks its own, and its quad adds them.  A
// quarter of the matrix cores' work is used, of which there is plenty.
//
// Workgroups begin at different units of a row (turn), so that they do not all
// read the same columns, a power of two apart, at once.
//
// The wavefronts' sums are added in their order through LDS, and eight
// consecutive features of a token go to the epilogue of the tiled product
// (ga_tile.h).
#pragma once

#include "ga_tile.h"

namespace ga {

constexpr int STREAM_WAVES = 8, STREAM_UNIT = 256;

template <int DT>
__device__ __forceinline__ f32x4 mfma_of(const i32x4 a, const i32x4 b, f32x4 c, int sa, int sb) {
    if constexpr (DT == DT_BF16)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    else if constexpr (DT == DT_F16)
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
    else {
        const i32x8 wa = {a.x, a.y, a.z, a.w, 0, 0, 0, 0}, wb = {b.x, b.y, b.z, b.w, 0, 0, 0, 0};
        return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wa, wb, c, 4, 4, 0, sa, 0, sb);
    }
}

template <int DT, int NF, int NT, int FG, int EPI, bool PAIR, int OUT>
__global__ __launch_bounds__(STREAM_WAVES * 64) void stream_kernel(TileArgs p) {
    constexpr bool MX = DT == DT_MX4;
    constexpr bool GATED = (EPI == EPI_GATED || EPI == EPI_QUANTIZE) && PAIR;
    constexpr int WK = STREAM_WAVES / FG;          // wavefronts that share k
    constexpr int HALF = GATED ? NF / 2 : NF;      // fragments of a half
    constexpr int FW = HALF * 4 * FG;              // features of D a workgroup
    static_assert(HALF % 2 == 0 && (EPI != EPI_QUANTIZE || FW % 32 == 0), "whole epilogues");
    __shared__ float sums[STREAM_WAVES][NT * 4][NF * 4];

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int row = lane >> 2 & 3, q = lane & 3, g = lane >> 4, wk = wave % WK;
    const int32_t f0 = (int32_t)blockIdx.x * FW, fw = f0 + wave / WK * (HALF * 4);  // the workgroup's, the wavefront's first
    const int32_t T = p.live != nullptr ? clamp_live(p.live, p.T) : p.T;
    if (T <= 0) return;

    const uint8_t *a = (const uint8_t *)p.a;
    const int32_t rows = p.F - fw < HALF * 4 ? p.F - fw : HALF * 4;  // may be below zero: nothing is read
    const int64_t up = GATED ? p.F : 0;
    const __amdgpu_buffer_rsrc_t wa = window(a + fw * p.a_row, rows * p.a_row), wu = window(a + (up + fw) * p.a_row, rows * p.a_row),
                                 wb = window(p.b, T * p.b_row);
    const __amdgpu_buffer_rsrc_t sga = MX ? window(p.a_scales + (int64_t)fw * p.blocks, (int64_t)rows * p.blocks) : wa,
                                 sua = MX ? window(p.a_scales + (up + fw) * p.blocks, (int64_t)rows * p.blocks) : wa,
                                 sgb = MX ? window(p.b_scales, (int64_t)T * p.blocks) : wa;
    const int32_t bytes = (int32_t)(MX ? p.a_row : 2 * (int64_t)p.K);  // of a row
    const int32_t units = (bytes + STREAM_UNIT - 1) / STREAM_UNIT;
    const int32_t turn = (int32_t)(blockIdx.x % (uint32_t)units);
    const uint32_t chunk = g * 4 + q;  // of the unit's 16
    const uint32_t va = row * (uint32_t)p.a_row + chunk * 16, vb = row * (uint32_t)p.b_row + chunk * 16;
    const uint32_t vs = row * (uint32_t)p.blocks + chunk;

    i32x4 fa[NF], fb[NT];
    int sa[NF], sb[NT];
    const auto issue = [&](int32_t round) {
        const int32_t n = round * WK + wk, from = n + turn;
        const int32_t unit = n >= units ? units : from >= units ? from - units : from;
        const bool in = unit * STREAM_UNIT + (int32_t)chunk * 16 < bytes;
        const uint32_t oa = in ? va : FAR, ob = in ? vb : FAR, os = in ? vs : FAR;
        const int at = unit * STREAM_UNIT;
#pragma unroll
        for (int i = 0; i < NF; ++i) {
            fa[i] = __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(i < HALF ? wa : wu, oa,
                                                                                     at + (int)(i % HALF * 4 * p.a_row), 0));
            // a block's scale where its codes are; past the row's end 0, 2^-127, as they are zero
            if constexpr (MX) sa[i] = __builtin_amdgcn_raw_buffer_load_b8(i < HALF ? sga : sua, os, at / 16 + i % HALF * 4 * p.blocks, 0);
        }
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            fb[j] = __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(wb, ob, at + (int)(j * 4 * p.b_row), 0));
            if constexpr (MX) sb[j] = __builtin_amdgcn_raw_buffer_load_b8(sgb, os, at / 16 + j * 4 * p.blocks, 0);
        }
    };

    f32x4 acc[NF][NT];
#pragma unroll
    for (int i = 0; i < NF; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
    issue(0);
    const int32_t rounds = (units + WK - 1) / WK;
    for (int32_t n = 0; n < rounds; ++n) {
#pragma unroll
        for (int i = 0; i < NF; ++i)
#pragma unroll
            for (int j = 0; j < NT; ++j)
                acc[i][j] = mfma_of<DT>(fa[i], fb[j], acc[i][j], MX ? sa[i] : 0, MX ? sb[j] : 0);
        issue(n + 1);
    }

    // ---- sums: lane 16 g + 4 t + q holds part q of feature g and token t in its entry q ----
#pragma unroll
    for (int i = 0; i < NF; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const f32x4 c = acc[i][j];
            float v = q < 2 ? (q == 0 ? c.x : c.y) : (q == 2 ? c.z : c.w);
            v += dpp_move<0xB1>(v);
            v += dpp_move<0x4E>(v);
            if (q == 0) sums[wave][j * 4 + row][i * 4 + g] = v;
        }
    __syncthreads();
    constexpr int OCTS = FW / 8, EACH = HALF / 2;  // octets of a token, of a wavefront's features
    for (int32_t n = threadIdx.x; n < OCTS * NT * 4; n += STREAM_WAVES * 64) {
        const int oct = n % OCTS, t = n / OCTS;
        const auto get = [&](int half, float (&v)[8]) {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = 0.0f;
#pragma unroll
            for (int w = 0; w < WK; ++w) {
                const float *at = &sums[oct / EACH * WK + w][t][half * HALF * 4 + oct % EACH * 8];
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] += at[e];
            }
        };
        float v[8], u[8] = {};
        get(0, v);
        if constexpr (GATED) get(1, u);
        const int32_t f = f0 + oct * 8;
        finish8<EPI, PAIR, OUT>(p, t, f, t < T && f < p.F, v, u);
    }
}

template <int DT, int NF, int NT, int FG, int EPI, bool PAIR, int OUT>
hipError_t launch_stream(const TileArgs &p, hipStream_t stream) {
    constexpr bool GATED = (EPI == EPI_GATED || EPI == EPI_QUANTIZE) && PAIR;
    constexpr int64_t FW = (GATED ? NF / 2 : NF) * 4 * FG;
    return launch_kernel(stream_kernel<DT, NF, NT, FG, EPI, PAIR, OUT>, dim3((uint32_t)((p.F + FW - 1) / FW)),
                         dim3(STREAM_WAVES * 64), stream, p);
}

// Features a workgroup: sixteen from 4096 features on (then 256 workgroups are
// there), else eight: one token in 4 bits, 4096 features of 16384 8.5 us against
// 11.8, 2048 features 6.7 against 7.0.  Gated in 16 bits: eight, or 32 from nine
// tokens on, whose loads they share: 16384 features of 2048, one token 26.4 us
// against 29.2, sixteen 33.5 against 30.8.
template <int DT, int EPI, bool PAIR, int OUT, int NT>
hipError_t launch_stream_tokens(const TileArgs &p, hipStream_t stream) {
    if constexpr (EPI == EPI_QUANTIZE) {
        return launch_stream<DT, PAIR ? 4 : 2, NT, 4, EPI, PAIR, OUT>(p, stream);
    } else if constexpr (EPI == EPI_GATED && PAIR) {
        return launch_stream<DT, 4, NT, NT == 4 ? 4 : 1, EPI, PAIR, OUT>(p, stream);
    } else {
        return p.F >= PRODUCT_FEW_WIDE ? launch_stream<DT, 4, NT, 1, EPI, PAIR, OUT>(p, stream)
                           : launch_stream<DT, 2, NT, 1, EPI, PAIR, OUT>(p, stream);
    }
}

template <int DT, int EPI, bool PAIR, int OUT>
hipError_t launch_few(const TileArgs &p, hipStream_t stream) {
    return p.T <= 4   ? launch_stream_tokens<DT, EPI, PAIR, OUT, 1>(p, stream)
           : p.T <= 8 ? launch_stream_tokens<DT, EPI, PAIR, OUT, 2>(p, stream)
                      : launch_stream_tokens<DT, EPI, PAIR, OUT, 4>(p, stream);
}

// One product with the planner's choice (plan_product, ga_internal.h).
template <int DT, bool AK, bool BK, int EPI, bool PAIR, int OUT>
hipError_t launch_product(TileArgs p, bool halves, float *partial, hipStream_t stream) {
    using Big = Tile<DT, AK, BK, 2, 4, 8, 4>;
    using Mid = Tile<DT, AK, BK, 2, 2, 4, 4>;
    using Wide = Tile<DT, AK, BK, 2, 2, 4, 6>;
    using Deep = Tile<DT, AK, BK, 2, 2, 4, 4, 4>;
    using Slim = Tile<DT, AK, BK, 2, 2, 4, 2, 4>;
    using Thin = Tile<DT, AK, BK, 1, 4, 4, 1, 4>;
    const ProductPlan plan = plan_product(p.F, p.T, p.K, halves, AK + BK, KPerStep<DT>::value);
    p.splits = plan.splits;
    p.k_split = plan.k_split;
    p.partial = partial;
    switch (plan.tile) {
    case PRODUCT_BIG: return launch_tile<Big, EPI, PAIR, OUT>(p, halves, stream);
    case PRODUCT_WIDE:
        if constexpr (!AK && !BK && DT != DT_MX4) return launch_tile<Wide, EPI, PAIR, OUT>(p, halves, stream);
        return hipErrorInvalidValue;
    case PRODUCT_MID: return launch_tile<Mid, EPI, PAIR, OUT>(p, halves, stream);
    case PRODUCT_DEEP: return launch_tile<Deep, EPI, PAIR, OUT>(p, halves, stream);
    case PRODUCT_SLIM:
    case PRODUCT_THIN: break;
    default:
        if constexpr (!AK && !BK) return launch_few<DT, EPI, PAIR, OUT>(p, stream);
        return hipErrorInvalidValue;
    }
    const bool thin = plan.tile == PRODUCT_THIN;
    if (plan.splits == 1)
        return thin ? launch_tile<Thin, EPI, PAIR, OUT>(p, halves, stream) : launch_tile<Slim, EPI, PAIR, OUT>(p, halves, stream);
    // the slices' sums: with two halves only for the epilogues that join them
    constexpr bool JOINS = (EPI == EPI_GATED || EPI == EPI_QUANTIZE) && PAIR;
    const hipError_t e = thin ? launch_tile<Thin, EPI_PARTIAL, JOINS, DT_F32>(p, halves, stream)
                              : launch_tile<Slim, EPI_PARTIAL, JOINS, DT_F32>(p, halves, stream);
    return e != hipSuccess ? e : launch_finish<EPI, PAIR, OUT>(p, !BK, stream);
}

}  // namespace ga
