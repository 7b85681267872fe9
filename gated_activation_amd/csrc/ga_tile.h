// The tiled matrix product of the feed-forward layer (gfx950): device code
// shared by the 16-bit and the microscaled 4-bit kernels.
//
//   D[f, t] = sum over k of A[f, k] B[t, k]      f: features, t: tokens
//
// in fp32 on the matrix cores, then an epilogue.  Each operand is stored either
// with k contiguous (a row of A or B per feature or token) or with k strided (a
// row per k): a weight gradient sums over tokens, so both its operands are.
//
// A workgroup owns FT features x TT tokens, its WF x WT wavefronts NF x NT
// fragments of 16 x 16 each.  Per step 128 bytes of k (64 values of 16 bits, 256
// of 4) of both tiles are brought into LDS by loads that write LDS themselves,
// into a stage that an earlier step used, while the matrix cores work on another:
// one barrier a step, in its middle.
//
// What bounds it: from a few thousand tokens on the matrix cores (bf16 8192 x 4096
// by 16384 the gated product with z kept 1700 us, the plain one 850, 1.3 PFLOP/s:
// they are busy 72 % of the time, at the clock that the card holds under them, the
// rest goes to the barrier of each step; 4-bit 4096 x 4096 by 16384 125 us, 4.4
// PFLOP/s, 56 %), with fewer the loads of a round of workgroups (64 x 4096 by 2 * 8192 36
// us, 3.8 TB/s; 1001 x 2056 by 1032 with the backward epilogue 22 us).
//
// Bounds.  Every load goes through a buffer descriptor that ends with the
// operand's last row (the last live token's, where tokens are bounded), so what
// lies past it reads as zero and adds nothing; a k past the end of a contiguous
// row is given an offset past the descriptor's end.  Columns past the last
// feature or token of a strided operand read the next row: they reach only
// elements of D that are not stored.
//
// LDS layout.  The loads write 16-byte chunks in lane order, so the order in
// LDS is chosen by which chunk each lane asks for.  A row of a contiguous
// operand is eight chunks; chunk c of row r sits in slot c ^ (r >> 1 & 7), and
// the 16 rows that 16 lanes read at one c then cover all 64 banks.  A row of a
// strided operand is FT (TT) values; ds_read_b64_tr_b16 hands each lane four
// k of its own column from four rows, and chunks are moved by swizzle_a / _b of
// the row so that the 16 pieces of a read lie in different banks.
//
// Which feature a row of the MFMA holds is free: row m of fragment j is feature
// (m / 4) 4 NF + 4 j + m % 4 of the wavefront's 16 NF.  A lane's NF results of
// four rows are then 4 NF consecutive features of one token, 16-byte stores.
// With a gate and an up half fragments j < NF / 2 are gate and the others up of
// the same features, so one lane holds both.
#pragma once

#include "ga_internal.h"
#include "ga_mx.h"
#include "ga_train.h"

namespace ga {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

enum : int { DT_MX4 = 3 };  // operands of 4 bits with scales; the results have a type of their own
enum Epilogue : int { EPI_STORE, EPI_GATED, EPI_BACKWARD, EPI_QUANTIZE, EPI_PARTIAL };

constexpr int STEP_BYTES = 128;  // bytes of k a row and step
constexpr uint32_t FAR = 0x80000000u;  // past the end of every descriptor

// What a product reads and writes.  Rows are in bytes.
struct TileArgs {
    const void *a, *b;
    const uint8_t *a_scales, *b_scales;  // MX4: [rows, blocks]
    int64_t a_row, b_row;
    int32_t F, T, K;                     // K: values; strided operands: rows
    int32_t blocks;                      // MX4: blocks of 32 a row
    const int32_t *live;                 // bounds T, or K where both operands are strided
    int32_t act;                         // OP_* of the epilogues that have one
    int32_t splits, k_split;             // slices of k (values, a multiple of the step)
    float *partial;                      // EPI_PARTIAL: [splits, T, gated ? 2 F : F]
    void *out;                           // STORE y [T, F]; GATED h [T, F]; BACKWARD dz; QUANTIZE codes
    void *out2;                          // GATED z [T, 2 F] or null; BACKWARD h [T, F]; QUANTIZE scales
    const void *z;                       // BACKWARD: gate | up [T, 2 F]
};

template <int DT> struct KPerStep { static constexpr int value = DT == DT_MX4 ? 256 : 64; };

// ---------------------------------------------------------------------------
// Epilogues of eight consecutive features f .. f + 7 of token t (F is a multiple
// of eight, so they are all there or none is).
// ---------------------------------------------------------------------------
template <int DT, bool NT = false>
__device__ __forceinline__ void store8(void *base, int64_t at, const float (&v)[8]) {
    oct_store<DT, NT>((typename Elem<DT>::storage *)base + at, v, 8);
}

// act(gate) * up of eight features; PAIR false: the squared ReLU of the gate
// alone, of which a NaN stays one: a sum over a row, it stands for all of the row's
// values, and a 4-bit block's NaN scale for finite ones too.  EXACT: the erf GELU by
// the library's erfc, where a value's last bits may decide its 4-bit code, in place
// of the approximation of absolute error 1.5e-7.
template <bool PAIR, bool EXACT>
__device__ __forceinline__ void activate8(int act, const float (&g)[8], const float (&u)[8], float (&h)[8]) {
    const auto each = [&](auto f) {
#pragma unroll
        for (int e = 0; e < 8; ++e) h[e] = f(g[e]) * u[e];
    };
    if constexpr (!PAIR) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float r = above_zero<true>(g[e]);
            h[e] = r * r;
        }
    } else if (act == OP_SILU_MUL) {
        each([](float x) { return silu(x); });
    } else if (act == OP_GELU_TANH_MUL) {
        each([](float x) { return gelu_tanh(x); });
    } else if constexpr (EXACT) {
        each([](float x) { return 0.5f * x * erfcf(x * -0.70710678118654752f); });
    } else {
        each([](float x) { return gelu_erf(x); });
    }
}

// The activation and its slope.
template <bool PAIR>
__device__ __forceinline__ void slope8(int act, const float (&g)[8], float (&v)[8], float (&dv)[8]) {
    const auto each = [&](auto f) {
#pragma unroll
        for (int e = 0; e < 8; ++e) f(g[e], v[e], dv[e]);
    };
    if constexpr (!PAIR) {
        each([](float x, float &f, float &df) {
            const float r = above_zero<true>(x);
            f = r * r;
            df = 2.0f * r;
        });
    } else if (act == OP_SILU_MUL) {
        each([](float x, float &f, float &df) { silu_slope(x, f, df); });
    } else if (act == OP_GELU_TANH_MUL) {
        each([](float x, float &f, float &df) { gelu_tanh_slope(x, f, df); });
    } else {
        each([](float x, float &f, float &df) { gelu_erf_slope(x, f, df); });
    }
}

// h is rounded to the type, as the next product takes its operands (the error of y
// against 64 bits is 2.3e-3 in bf16, 1.7e-3 with h in fp32; 2.9e-4 and 2.1e-4 in fp16,
// where |h| from 65520 on is an infinity).
template <int DT, bool PAIR>
__device__ __forceinline__ void gated8(const TileArgs &p, int64_t t, int32_t f, const float (&g)[8], const float (&u)[8]) {
    constexpr bool GATED = PAIR;
    const int64_t F = p.F;
    if (p.out2 != nullptr) {
        // Read by the backward pass, after much else: past the caches (16384 x 2048 by
        // 768, 12288 live: 123 us against 128).  Not so dz and h of the backward pass,
        // which the next products read (1001 x 1032 by 2056: 82 us, 97 past the caches).
        store8<DT, true>(p.out2, t * (GATED ? 2 * F : F) + f, g);
        if constexpr (GATED) store8<DT, true>(p.out2, t * 2 * F + F + f, u);
    }
    float h[8];
    activate8<PAIR, false>(p.act, g, u, h);
    store8<DT>(p.out, t * F + f, h);
}

// zg, zu: the kept gate and up values there.  dz and h are rounded to the type, as the
// three gradients' products take them.
template <int DT, bool PAIR>
__device__ __forceinline__ void backward8(const TileArgs &p, int64_t t, int32_t f, const float (&dh)[8], const Oct<DT> &zg,
                                          const Oct<DT> &zu) {
    constexpr bool GATED = PAIR;
    const int64_t F = p.F, at = t * (GATED ? 2 * F : F) + f;
    float g[8], u[8], h[8], dg[8], du[8], v[8], dv[8];
    oct_unpack<DT>(zg, g);
    if constexpr (GATED) oct_unpack<DT>(zu, u);
    slope8<PAIR>(p.act, g, v, dv);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        if constexpr (GATED) {
            h[e] = v[e] * u[e];
            dg[e] = dh[e] * u[e] * dv[e];
            du[e] = dh[e] * v[e];
        } else {
            h[e] = v[e];
            dg[e] = dh[e] * dv[e];
        }
    }
    store8<DT>(p.out, at, dg);
    if constexpr (GATED) store8<DT>(p.out, at + F, du);
    store8<DT>(p.out2, t * F + f, h);
}

// Features f .. f + 7 of a row of any length.
template <int DT>
__device__ __forceinline__ void store_row(const TileArgs &p, int64_t t, int32_t f, const float (&v)[8]) {
    oct_store<DT, false>((typename Elem<DT>::storage *)p.out + t * p.F + f, v, p.F - f);
}

__device__ __forceinline__ uint32_t top8(const float (&h)[8]) {
    uint32_t top = magnitude(h[0]);
#pragma unroll
    for (int e = 1; e < 8; ++e) top = max(top, magnitude(h[e]));
    return top;
}

// What an epilogue does with eight features of a token (in: they are there).
// QUANTIZE: F is a multiple of 32, and the four lanes of a quad hold a block of it.
// BACKWARD: zg and zu as backward8 takes them.
template <int EPI, bool PAIR, int OUT>
__device__ __forceinline__ void finish8(const TileArgs &p, int64_t t, int32_t f, bool in, const float (&v)[8],
                                        const float (&u)[8], const Oct<OUT> &zg = Oct<OUT>(), const Oct<OUT> &zu = Oct<OUT>()) {
    if constexpr (EPI == EPI_QUANTIZE) {
        float h[8];
        activate8<PAIR, true>(p.act, v, u, h);
        uint32_t top = top8(h);
        top = dpp_umax<0xB1>(top);
        top = dpp_umax<0x4E>(top);
        if (in) {
            const uint32_t s = mx_scale_byte(top);
            const int64_t block = t * (p.F / MX_BLOCK) + f / MX_BLOCK;
            ((uint32_t *)p.out)[block * 4 + f / 8 % 4] = mx_codes8(h, s);
            if (f % MX_BLOCK == 0) ((uint8_t *)p.out2)[block] = (uint8_t)s;
        }
    } else if (in) {
        if constexpr (EPI == EPI_STORE) store_row<OUT>(p, t, f, v);
        else if constexpr (EPI == EPI_GATED) gated8<OUT, PAIR>(p, t, f, v, u);
        else backward8<OUT, PAIR>(p, t, f, v, zg, zu);
    }
}

// ---------------------------------------------------------------------------
// The workgroup's tile: the tiles are dealt to the eight XCDs in contiguous runs
// (workgroups go to them in turn), and a run walks panels of PANEL token tiles,
// so the workgroups that share an L2 share their operands' rows.
// ---------------------------------------------------------------------------
constexpr uint32_t XCDS = 8, PANEL = 4;

__device__ __forceinline__ void tile_of(uint32_t b, uint32_t n, uint32_t nf, uint32_t nt, uint32_t &ft, uint32_t &tt) {
    const uint32_t q = n / XCDS, r = n % XCDS, x = b % XCDS;
    const uint32_t id = x * q + (x < r ? x : r) + b / XCDS;
    const uint32_t panel = id / (PANEL * nf), first = panel * PANEL;
    const uint32_t height = nt - first < PANEL ? nt - first : PANEL, in = id - first * nf;
    tt = first + in % height;
    ft = in / height;
}

__device__ __forceinline__ __amdgpu_buffer_rsrc_t window(const void *base, int64_t bytes) {
    const int64_t n = bytes < 0 ? 0 : bytes > 0x7FFFFFF0 ? 0x7FFFFFF0 : bytes;
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), 0, (int)n, 0x00020000);
}

typedef __attribute__((address_space(3))) void lds_void;

__device__ __forceinline__ void to_lds(__amdgpu_buffer_rsrc_t r, void *lds, uint32_t voffset, int soffset) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void *)lds, 16, voffset, soffset, 0, 0);
}

// Chunk swizzles of strided operands by k row (see above): a read's four rows k % 4.
// A lane's pieces are 8 NF bytes apart: 64 of them, or 32 in rows of 256 or 128 bytes.
template <int FT, int NF>
__device__ __forceinline__ uint32_t swizzle_a(uint32_t k) {
    static_assert(NF == 8 || (NF == 4 && FT <= 128), "chunks within a row");
    return NF == 8 ? (k & 3) : FT == 64 ? (k >> 1 & 1) : (k & 1) | (k & 2) << 2;
}
__device__ __forceinline__ uint32_t swizzle_b(uint32_t k) { return (k & 3) << 1; }

// c += a b, written as assembly with the sum and the result in one register:
// left to choose, the compiler moves the large tile's 128 sums about and spills
// (8192 x 4096 x 16384 bf16: 1740-1960 us where it does, 810-860 tied; 4-bit
// 4096 x 4096 x 16384 182 us, 126 tied).  The compiler knows no waits of it: the
// two states ahead are for an operand that a vector instruction has just written,
// and sums are read only past settled().
template <int DT>
__device__ __forceinline__ void mfma(f32x4 &c, const i32x4 a, const i32x4 b, int sa, int sb, int byte) {
    if constexpr (DT == DT_BF16) {
        asm("s_nop 1\n\tv_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+v"(c) : "v"(a), "v"(b));
    } else if constexpr (DT == DT_F16) {
        asm("s_nop 1\n\tv_mfma_f32_16x16x32_f16 %0, %1, %2, %0" : "+v"(c) : "v"(a), "v"(b));
    } else {
        // formats 4: e2m1; the operand selects choose byte `byte` of both scale words
#define GA_MFMA4(SEL) \
    asm("s_nop 1\n\tv_mfma_scale_f32_16x16x128_f8f6f4 %0, %1, %2, %0, %3, %4 " SEL " cbsz:4 blgp:4" \
        : "+v"(c) : "v"(a), "v"(b), "v"(sa), "v"(sb))
        if (byte == 0) GA_MFMA4("op_sel:[0,0,0] op_sel_hi:[0,0,0]");
        else if (byte == 1) GA_MFMA4("op_sel:[1,1,0] op_sel_hi:[0,0,0]");
        else if (byte == 2) GA_MFMA4("op_sel:[0,0,0] op_sel_hi:[1,1,0]");
        else GA_MFMA4("op_sel:[1,1,0] op_sel_hi:[1,1,0]");
#undef GA_MFMA4
    }
}

// Ends the last product: 32 states.  A vector instruction may read the result of a
// matrix instruction of 16 passes 19 states after it, and those here have 8 passes at
// most.
template <int NF, int NT>
__device__ __forceinline__ void settled(f32x4 (&acc)[NF][NT]) {
    asm volatile("s_nop 15\n\ts_nop 15" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < NF; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) asm volatile("" : "+v"(acc[i][j]));
}

// ---------------------------------------------------------------------------
// The kernel.  AK / BK: the operand is strided.  GATED: A has 2 F rows.
// ---------------------------------------------------------------------------
// STAGES: steps of both tiles in LDS, all but one of them being loaded.
template <int DT_, bool AK_, bool BK_, int WF_, int WT_, int NF_, int NT_, int STAGES_ = 2> struct Tile {
    static constexpr int DT = DT_, WF = WF_, WT = WT_, NF = NF_, NT = NT_, STAGES = STAGES_;
    static constexpr bool AK = AK_, BK = BK_;
    static constexpr int W = WF * WT, FT = WF * NF * 16, TT = WT * NT * 16;
    static constexpr int KS = KPerStep<DT>::value;
    static constexpr int LA = FT / 8 / W, LB = TT / 8 / W;  // 1024-byte loads a wavefront and step
    static_assert(LA * 8 * W == FT && LB * 8 * W == TT, "loads");
    static_assert(STAGES == 2 || STAGES == 4, "stages");
    static_assert(DT != DT_MX4 || (!AK && !BK), "scales");
};

// The feature (of D, or of either half's) that row `row` of a contiguous A tile
// holds.  Rows 8 W apart are equally many features apart for every lane.
template <int NF, bool GATED>
__device__ __forceinline__ constexpr uint32_t feature_of(uint32_t row) {
    const uint32_t m = row & 15, frag = row / 16 % NF;
    return GATED ? row / (16 * NF) * (8 * NF) + (m >> 2) * (2 * NF) + frag % (NF / 2) * 4 + (m & 3)
                 : row / (16 * NF) * (16 * NF) + (m >> 2) * (4 * NF) + frag * 4 + (m & 3);
}

// Workgroup `block` of a product.  as, bs: each stage's LDS, FT and TT rows of
// STEP_BYTES, in arrays of their own by stage: the compiler then sees that a read of
// one does not wait for the loads into another.  sc: MX4, a row's scales of two
// steps, twice, and the last ones.
template <typename C, int EPI, bool PAIR, int OUT>
__device__ __forceinline__ void tile_body(const TileArgs &p, uint32_t block, uint8_t *const (&as)[4], uint8_t *const (&bs)[4],
                                          uint4 *sc) {
    constexpr int DT = C::DT, W = C::W, FT = C::FT, TT = C::TT, NF = C::NF, NT = C::NT;
    constexpr bool MX = DT == DT_MX4;
    constexpr bool GATED = (EPI == EPI_GATED || EPI == EPI_QUANTIZE || EPI == EPI_PARTIAL) && PAIR && !C::AK;
    constexpr int FW = GATED ? FT / 2 : FT;  // features of D a workgroup
    constexpr int S = C::STAGES;

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, g = lane >> 4, wf = wave / C::WT, wt = wave % C::WT;
    int32_t T = p.T, K = p.K;
    if (p.live != nullptr) {
        if constexpr (C::BK) K = clamp_live(p.live, K);
        else T = clamp_live(p.live, T);
    }
    // The live tokens' tiles alone are dealt out, so that every XCD has its share
    // (16384 x 2 * 768 x 2048, 12288 of the tokens live: 115 us with the others' dealt too).
    const uint32_t nf = (uint32_t)((p.F + FW - 1) / FW), nt = (uint32_t)((T + TT - 1) / TT), n = nf * nt;
    const uint32_t all = nf * (uint32_t)((p.T + TT - 1) / TT), split = block / all, id = block - split * all;
    if (id >= n) return;
    uint32_t ft, tt;
    tile_of(id, n, nf, nt, ft, tt);
    const int32_t f0 = (int32_t)(ft * FW), t0 = (int32_t)(tt * TT);
    const int32_t kb = (int32_t)split * p.k_split;
    const int32_t ke = p.k_split < K - kb ? kb + p.k_split : K;  // past it: zeros (may be below kb)
    const int32_t steps = ke > kb ? (ke - kb + C::KS - 1) / C::KS : 0;

    // ---- what this lane loads ----
    // One offset a lane and operand: load j of a wavefront is 8 W rows (or as many
    // k) further on for every lane, which is a uniform offset.
    uint32_t va, vb;
    uint32_t chunk_a, chunk_b;  // contiguous operands: the chunk of the row's 128 bytes
    if constexpr (C::AK) {
        constexpr int CPR = FT / 8, RPI = 64 / CPR;
        const uint32_t k = wave * RPI + lane / CPR;
        va = k * (uint32_t)p.a_row + ((lane % CPR) ^ swizzle_a<FT, NF>(k)) * 16;
    } else {
        const uint32_t row = wave * 8 + (lane >> 3);
        chunk_a = (lane & 7) ^ (row >> 1 & 7);
        va = feature_of<NF, GATED>(row) * (uint32_t)p.a_row + chunk_a * 16;
    }
    if constexpr (C::BK) {
        constexpr int CPR = TT / 8, RPI = 64 / CPR;
        const uint32_t k = wave * RPI + lane / CPR;
        vb = k * (uint32_t)p.b_row + ((lane % CPR) ^ swizzle_b(k)) * 16;
    } else {
        const uint32_t row = wave * 8 + (lane >> 3);
        chunk_b = (lane & 7) ^ (row >> 1 & 7);
        vb = row * (uint32_t)p.b_row + chunk_b * 16;
    }
    const uint8_t *a = (const uint8_t *)p.a, *b = (const uint8_t *)p.b;
    const int32_t rows_a = p.F - f0 < FW ? p.F - f0 : FW, rows_b = T - t0 < TT ? T - t0 : TT;
    __amdgpu_buffer_rsrc_t wa = window(a, 0), wu = wa, wb = wa;
    if constexpr (!C::AK) {
        wa = window(a + f0 * p.a_row, rows_a * p.a_row);
        if constexpr (GATED) wu = window(a + ((int64_t)p.F + f0) * p.a_row, rows_a * p.a_row);
    }
    if constexpr (!C::BK) wb = window(b + t0 * p.b_row, rows_b * p.b_row);

    // MX4: the row whose scales this thread brings, from the tile's first
    __amdgpu_buffer_rsrc_t ws = wa;
    uint32_t vs = 0;
    const int32_t first_block = kb / MX_BLOCK, blocks = MX ? (ke - kb + MX_BLOCK - 1) / MX_BLOCK : 0;  // of this slice
    if constexpr (MX) {
        if (wave >= (FT + TT) / 64) {
            vs = FAR;
        } else if (wave < FT / 64) {
            const uint32_t row = threadIdx.x;
            vs = feature_of<NF, GATED>(row) * (uint32_t)p.blocks;
            if (GATED && row / 16 % NF >= NF / 2) vs += (uint32_t)p.F * (uint32_t)p.blocks;
            ws = window(p.a_scales + (int64_t)f0 * p.blocks, ((GATED ? 2 * (int64_t)p.F : p.F) - f0) * p.blocks);
        } else {
            vs = (threadIdx.x - FT) * (uint32_t)p.blocks;
            ws = window(p.b_scales + (int64_t)t0 * p.blocks, (int64_t)rows_b * p.blocks);
        }
        if (wave < (FT + TT) / 64) vs += first_block;
    }

    // The loads of step s: where they read (aim), and one of them.
    uint32_t oa, ob;
    int so;
    const auto aim = [&](int32_t s) {
        const int32_t k0 = kb + s * C::KS;
        const bool tail = k0 + C::KS > ke;
        // chunks of this step that are there; a row of 4-bit codes ends with its last block's 16 bytes
        const uint32_t chunks = k0 >= ke ? 0 : MX ? (uint32_t)((ke - k0 + 31) / 32) : (uint32_t)((ke - k0 + 7) / 8);
        if constexpr (C::AK)
            wa = window(a + k0 * p.a_row + (int64_t)f0 * 2, (int64_t)(tail ? ke - k0 : C::KS) * p.a_row - (int64_t)f0 * 2);
        if constexpr (C::BK)
            wb = window(b + k0 * p.b_row + (int64_t)t0 * 2, (int64_t)(tail ? ke - k0 : C::KS) * p.b_row - (int64_t)t0 * 2);
        so = MX ? k0 / 2 : k0 * 2;
        oa = !C::AK && tail && chunk_a >= chunks ? FAR : va, ob = !C::BK && tail && chunk_b >= chunks ? FAR : vb;
    };
    const auto load_one = [&](int j, uint8_t *la, uint8_t *lb) {
        if (j < C::LA) {
            uint8_t *at = la + (j * W + wave) * 1024;
            if constexpr (C::AK) {
                to_lds(wa, at, oa, (int)(j * W * 64 / (FT / 8) * p.a_row));
            } else {
                const bool up = GATED && (j * W + wave) / 2 % NF >= NF / 2;
                to_lds(up ? wu : wa, at, oa, so + (int)(feature_of<NF, GATED>(j * W * 8) * p.a_row));
            }
        } else {
            j -= C::LA;
            uint8_t *at = lb + (j * W + wave) * 1024;
            if constexpr (C::BK) to_lds(wb, at, ob, (int)(j * W * 64 / (TT / 8) * p.b_row));
            else to_lds(wb, at, ob, so + (int)(j * W * 8 * p.b_row));
        }
    };
    const auto load = [&](int32_t s, uint8_t *la, uint8_t *lb) {
        aim(s);
#pragma unroll
        for (int j = 0; j < C::LA + C::LB; ++j) load_one(j, la, lb);
    };

    // Scales go through registers, 16 of a row for two steps at a time: into one
    // of two halves of sc, or where the slice ends within the 16, once and byte by
    // byte at the start, into the third.  (A branch to the byte loads inside the
    // loop made the compiler wait for every load in flight: 308 us against 187
    // without any scale, 4096 x 4096 x 16384.)
    const auto load_scales = [&](int32_t w) -> u32x4 {
        return __builtin_amdgcn_raw_buffer_load_b128(ws, vs + w * 16, 0, 0);
    };
    // Bytes b of words 0 .. 3 become word b: lane group g reads the scales of its
    // block of both instructions of both steps.
    const auto put_scales = [&](u32x4 v, uint4 *to) {
        const uint32_t lo0 = __builtin_amdgcn_perm(v.y, v.x, 0x05010400u), hi0 = __builtin_amdgcn_perm(v.y, v.x, 0x07030602u);
        const uint32_t lo1 = __builtin_amdgcn_perm(v.w, v.z, 0x05010400u), hi1 = __builtin_amdgcn_perm(v.w, v.z, 0x07030602u);
        if (W * 64 > FT + TT && wave >= (FT + TT) / 64) return;
        to[threadIdx.x] = uint4{__builtin_amdgcn_perm(lo1, lo0, 0x05040100u), __builtin_amdgcn_perm(lo1, lo0, 0x07060302u),
                                __builtin_amdgcn_perm(hi1, hi0, 0x05040100u), __builtin_amdgcn_perm(hi1, hi0, 0x07060302u)};
    };
    const auto put_last_scales = [&] {
        u32x4 v = {0, 0, 0, 0};  // 2^-127: the codes there are zero
#pragma unroll
        for (int e = 0; e < 15; ++e)
            if (e < blocks % 16)
                v[e / 4] |= (uint32_t)__builtin_amdgcn_raw_buffer_load_b8(ws, vs + blocks / 16 * 16 + e, 0, 0) << (e % 4 * 8);
        put_scales(v, sc + 2 * (FT + TT));
    };

    // ---- fragments ----
    f32x4 acc[NF][NT];
#pragma unroll
    for (int i = 0; i < NF; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = f32x4{0, 0, 0, 0};

    const auto read_row = [&](const uint8_t *tile, int row, int kk) -> i32x4 {
        return *reinterpret_cast<const i32x4 *>(tile + (row + r) * STEP_BYTES + (((kk * 4 + g) ^ (r >> 1)) * 16));
    };
    const auto read_tr = [&](const uint8_t *at) -> i16x4 {
        return __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) i16x4 *)at);
    };
    const int q = r & 3, kr = r >> 2;
    const auto read_b = [&](const uint8_t *lb, int kk, int j) -> i32x4 {
        if constexpr (C::BK) {
            const uint32_t k = kk * 32 + g * 8 + kr;
            const uint32_t chunk = ((wt * NT + j) * 2 + (q >> 1)) ^ swizzle_b(kr);
            const uint8_t *at = lb + k * (TT * 2) + chunk * 16 + (q & 1) * 8;
            const i16x4 lo = read_tr(at), hi = read_tr(at + 4 * TT * 2);
            return __builtin_bit_cast(i32x4, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
        } else {
            return read_row(lb, (wt * NT + j) * 16, kk);
        }
    };
    const auto read_a = [&](const uint8_t *la, int kk, int i) -> i32x4 {
        if constexpr (C::AK) {
            const uint32_t k = kk * 32 + g * 8 + kr;
            const uint32_t chunk = ((wf * NF * 16 + q * NF * 4 + i * 4) / 8) ^ swizzle_a<FT, NF>(kr);
            const uint8_t *at = la + k * (FT * 2) + chunk * 16 + (i & 1) * 8;
            const i16x4 lo = read_tr(at), hi = read_tr(at + 4 * FT * 2);
            return __builtin_bit_cast(i32x4, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
        } else {
            return read_row(la, (wf * NF + i) * 16, kk);
        }
    };
    // Half a step: multiplies (fa, fb), by rows of the tile; beside the rows' products
    // reads the next fragments (na, nb) from half kk of (la, lb) and, where LOAD,
    // issues the loads aimed into (da, db), a few a row: all at once they hold up
    // the wavefronts' other work (gated 16384 x 8192 x 4096: 1660 us, 1600 spread).
    const auto phase = [&](const i32x4 (&fa)[NF], const i32x4 (&fb)[NT], const int (&sa)[NF], const int (&sb)[NT], auto byte,
                           const uint8_t *la, const uint8_t *lb, int kk, i32x4 (&na)[NF], i32x4 (&nb)[NT], auto load,
                           uint8_t *da, uint8_t *db) {
        constexpr int READS = (NF + NT + NF - 3) / (NF - 2), LOADS = (C::LA + C::LB + NF - 1) / NF;  // a row
#pragma unroll
        for (int i = 0; i < NF; ++i) {
#pragma unroll
            for (int e = i * READS; e < (i + 1) * READS && e < NF + NT; ++e) {
                if (e < NT) nb[e] = read_b(lb, kk, e);
                else na[e - NT] = read_a(la, kk, e - NT);
            }
            if constexpr (decltype(load)::value) {
#pragma unroll
                for (int j = i * LOADS; j < (i + 1) * LOADS && j < C::LA + C::LB; ++j) load_one(j, da, db);
            }
#pragma unroll
            for (int j = 0; j < NT; ++j) mfma<DT>(acc[i][j], fa[i], fb[j], sa[i], sb[j], decltype(byte)::value);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    const auto read_scales = [&](int32_t w, int (&sa)[NF], int (&sb)[NT]) {
        // (past the last window that one: zeros are multiplied, and its bytes are scales)
        const int32_t v = w * 16 < blocks ? w : (blocks - 1) / 16;
        const uint32_t *h = reinterpret_cast<const uint32_t *>(sc + (v * 16 + 16 > blocks ? 2 : v & 1) * (FT + TT));
#pragma unroll
        for (int i = 0; i < NF; ++i) sa[i] = h[((wf * NF + i) * 16 + r) * 4 + g];
#pragma unroll
        for (int j = 0; j < NT; ++j) sb[j] = h[(FT + (wt * NT + j) * 16 + r) * 4 + g];
    };
    // Waits until at most `most` of the wavefront's loads are on their way and
    // its reads of LDS are done, and for the others to get there.
    const auto meet = [](auto most) {
        constexpr int N = decltype(most)::value;
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_waitcnt((N & 15) | 7 << 4 | (N >> 4) << 14);
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
    };
    // A step's second fragments are read while its first are multiplied, and the
    // next step's first while its second are: the barrier between has products
    // queued on either side.  Past it the step's own stage of LDS is free for the
    // loads of the step S further on.  Loads of steps that are not there read
    // nothing (their offsets are past the end).
    constexpr int L = C::LA + C::LB;
    const std::integral_constant<int, (S - 2) * L> but_last;
    const std::integral_constant<int, 0> none;
    const std::true_type loads;
    const std::false_type no_loads;
    i32x4 fa0[NF], fa1[NF], fb0[NT], fb1[NT];
    int sa[NF], sb[NT];
    u32x4 next{};
    if (steps > 0) {
        if constexpr (MX) {
            next = load_scales(0);
            if (blocks % 16 != 0) put_last_scales();
        }
#pragma unroll
        for (int e = 0; e < S - 1; ++e) load(e, as[e], bs[e]);
        if constexpr (MX) put_scales(next, sc);
        meet(but_last);
        load(S - 1, as[S - 1], bs[S - 1]);
#pragma unroll
        for (int j = 0; j < NT; ++j) fb0[j] = read_b(bs[0], 0, j);
#pragma unroll
        for (int i = 0; i < NF; ++i) fa0[i] = read_a(as[0], 0, i);
        if constexpr (MX) read_scales(0, sa, sb);
    }
    const auto step = [&](int32_t s, auto place) {
        constexpr int e = decltype(place)::value, n = (e + 1) % S, ODD = e & 1;
        int na[NF], nb[NT];
        if constexpr (MX && !ODD) next = load_scales(s / 2 + 1);
        phase(fa0, fb0, sa, sb, std::integral_constant<int, 2 * ODD>(), as[e], bs[e], 1, fa1, fb1, no_loads, as[e], bs[e]);
        if constexpr (MX && ODD) put_scales(next, sc + ((s / 2 + 1) & 1) * (FT + TT));
        aim(s + S);
        meet(but_last);
        if constexpr (MX && ODD) read_scales(s / 2 + 1, na, nb);
        phase(fa1, fb1, sa, sb, std::integral_constant<int, 2 * ODD + 1>(), as[n], bs[n], 0, fa0, fb0, loads, as[e], bs[e]);
        if constexpr (MX && ODD) {
#pragma unroll
            for (int i = 0; i < NF; ++i) sa[i] = na[i];
#pragma unroll
            for (int j = 0; j < NT; ++j) sb[j] = nb[j];
        }
    };
    if constexpr (S == 2) {
        for (int32_t s = 0; s + 2 <= steps; s += 2) {
            step(s, std::integral_constant<int, 0>());
            step(s + 1, std::integral_constant<int, 1>());
        }
        if (steps & 1) {
            phase(fa0, fb0, sa, sb, std::integral_constant<int, 0>(), as[0], bs[0], 1, fa1, fb1, no_loads, as[0], bs[0]);
            phase(fa1, fb1, sa, sb, std::integral_constant<int, 1>(), as[0], bs[0], 1, fa0, fb0, no_loads, as[0], bs[0]);
        }
    } else {
        // up to three steps of zeros at the end
        for (int32_t s = 0; s < steps; s += 4) {
            step(s, std::integral_constant<int, 0>());
            step(s + 1, std::integral_constant<int, 1>());
            step(s + 2, std::integral_constant<int, 2>());
            step(s + 3, std::integral_constant<int, 3>());
        }
    }
    settled(acc);

    // ---- epilogue ----
    // Through LDS, SPACE bytes a wavefront and JT x 16 tokens at a time, so that a lane
    // ends up with eight consecutive features and neighbouring lanes with the
    // next ones.  (Straight from the accumulators the unrolled epilogue spills.)
    // Four results of a lane are 16 bytes of a token's row; chunk c of token t
    // sits in c ^ t % 16, so that 16 tokens' writes fall into all banks.
    constexpr int ARRAYS = FT == TT ? 4 : 2, PER = W / ARRAYS;  // arrays in use, wavefronts an array
    constexpr int SPACE = FT * STEP_BYTES / PER;
    constexpr int MOST = SPACE / (NF * 16 * 16 * 4), JT = MOST < NT ? MOST : NT, CHUNKS = NF * 4;  // chunks a token
    static_assert(JT > 0 && NT % JT == 0 && W % ARRAYS == 0, "whole tokens");
    uint8_t *const mine = (wave / PER == 0 ? as[0] : wave / PER == ARRAYS / 2 ? as[1] : wave / PER == 1 ? bs[0] : bs[1]) + wave % PER * SPACE;
    constexpr int LANES = CHUNKS / (GATED ? 4 : 2), TOKENS = 64 / LANES;  // lanes a token, tokens a pass
    constexpr int PASSES = JT * 16 / TOKENS, AHEAD = PASSES < 4 ? PASSES : 4;
    static_assert(PASSES % AHEAD == 0, "passes");
    const int oct = lane % LANES, token = lane / LANES;
    const int32_t f = f0 + wf * (LANES * 8) + oct * 8;
    // BACKWARD: the kept values of four passes are on their way (one at a time they
    // took most of the epilogue)
    Oct<OUT> zg[AHEAD], zu[AHEAD];
    constexpr int64_t ZROW = EPI == EPI_BACKWARD ? (PAIR ? 4 : 2) : 0;  // bytes of z a feature
    const __amdgpu_buffer_rsrc_t wz = window((const uint8_t *)p.z + t0 * ZROW * p.F, rows_b * ZROW * p.F);
    const auto fetch = [&](int pass, Oct<OUT> &kg, Oct<OUT> &ku) {
        if constexpr (EPI == EPI_BACKWARD) {
            const uint32_t at = (wt * NT * 16 + pass * TOKENS + token) * (uint32_t)(ZROW * p.F) + f * 2;
            kg = __builtin_bit_cast(Oct<OUT>, __builtin_amdgcn_raw_buffer_load_b128(wz, at, 0, 0));
            if constexpr (PAIR) ku = __builtin_bit_cast(Oct<OUT>, __builtin_amdgcn_raw_buffer_load_b128(wz, at, 2 * p.F, 0));
        }
    };
#pragma unroll
    for (int d = 0; d < AHEAD; ++d) fetch(d, zg[d], zu[d]);
    meet(none);
#pragma unroll
    for (int half = 0; half < NT / JT; ++half) {
#pragma unroll
        for (int jj = 0; jj < JT; ++jj) {
#pragma unroll
            for (int i = 0; i < NF; ++i) {
                constexpr int HF = NF / 2;
                const int chunk = GATED ? (i < HF ? g * HF + i : CHUNKS / 2 + g * HF + i - HF) : g * NF + i;
                *reinterpret_cast<f32x4 *>(mine + ((jj * 16 + r) * CHUNKS + (chunk ^ r)) * 16) = acc[i][half * JT + jj];
            }
        }
#pragma unroll 1
        for (int first = 0; first < PASSES; first += AHEAD) {
#pragma unroll
            for (int d = 0; d < AHEAD; ++d) {
                const int pass = half * PASSES + first + d, tok = (first + d) * TOKENS + token;
                const auto get = [&](int chunk, float (&v)[8]) {
                    const f32x4 lo = *reinterpret_cast<const f32x4 *>(mine + (tok * CHUNKS + (chunk ^ (tok & 15))) * 16);
                    const f32x4 hi = *reinterpret_cast<const f32x4 *>(mine + (tok * CHUNKS + ((chunk + 1) ^ (tok & 15))) * 16);
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[e] = lo[e], v[4 + e] = hi[e];
                };
                float v[8], u[8] = {};
                get(2 * oct, v);
                if constexpr (GATED) get(CHUNKS / 2 + 2 * oct, u);
                const int32_t t = t0 + wt * NT * 16 + pass * TOKENS + token;
                if constexpr (EPI == EPI_PARTIAL) {
                    if (t < T && f < p.F) {
                        uint32_t *at = (uint32_t *)p.partial + ((int64_t)split * p.T + t) * (GATED ? 2 : 1) * p.F + f;
                        oct_store<DT_F32, false>(at, v, p.F - f);
                        if constexpr (GATED) oct_store<DT_F32, false>(at + p.F, u, p.F - f);
                    }
                } else {
                    finish8<EPI, PAIR, OUT>(p, t, f, t < T && f < p.F, v, u, zg[d], zu[d]);
                }
                fetch(pass + AHEAD, zg[d], zu[d]);
            }
        }
    }
}

template <typename C, int EPI, bool PAIR, int OUT>
__global__ __launch_bounds__(C::W * 64) void tile_kernel(TileArgs p) {
    constexpr int A = C::FT * STEP_BYTES, B = C::TT * STEP_BYTES, S = C::STAGES;
    __shared__ __attribute__((aligned(16))) uint8_t a0[A], b0[B], a1[A], b1[B];
    __shared__ __attribute__((aligned(16))) uint8_t a2[S > 2 ? A : 16], b2[S > 2 ? B : 16], a3[S > 2 ? A : 16], b3[S > 2 ? B : 16];
    __shared__ uint4 sc[C::DT == DT_MX4 ? 3 * (C::FT + C::TT) : 1];
    uint8_t *const as[4] = {a0, a1, a2, a3}, *const bs[4] = {b0, b1, b2, b3};
    tile_body<C, EPI, PAIR, OUT>(p, blockIdx.x, as, bs, sc);
}

// ---------------------------------------------------------------------------
// Three products in one launch, where none of them fills the card: x (A strided) in
// tiles of 64 x 64, in and down (both strided) of 128 x 128.  Both tiles take 64 KB
// of LDS, so any two are on a unit at a time.  Bound by the loads of steps that few
// wavefronts wait for (fp16 1001 x 1032 by 2056 47 us, the three one after another
// 65).
// ---------------------------------------------------------------------------
template <int DT, bool CUT_X, bool CUT_W>
__global__ __launch_bounds__(256) void three_kernel(TileArgs x, TileArgs in, TileArgs down, uint32_t n_x, uint32_t n_in) {
    constexpr int EPI_X = CUT_X ? EPI_PARTIAL : EPI_STORE, OUT_X = CUT_X ? DT_F32 : DT;
    constexpr int EPI_W = CUT_W ? EPI_PARTIAL : EPI_STORE, OUT_W = CUT_W ? DT_F32 : DT;
    using X = Tile<DT, true, false, 1, 4, 4, 1, 4>;
    using W = Tile<DT, true, true, 2, 2, 4, 4>;
    constexpr int HALF = X::FT * STEP_BYTES;
    static_assert(2 * HALF == W::FT * STEP_BYTES && X::TT == X::FT && W::TT == W::FT, "arrays");
    __shared__ __attribute__((aligned(16))) uint8_t s0[2 * HALF], s1[2 * HALF], s2[2 * HALF], s3[2 * HALF];
    if (blockIdx.x < n_x) {
        uint8_t *const as[4] = {s0, s1, s2, s3}, *const bs[4] = {s0 + HALF, s1 + HALF, s2 + HALF, s3 + HALF};
        tile_body<X, EPI_X, false, OUT_X>(x, blockIdx.x, as, bs, nullptr);
    } else {
        uint8_t *const as[4] = {s0, s2, nullptr, nullptr}, *const bs[4] = {s1, s3, nullptr, nullptr};
        const uint32_t block = blockIdx.x - n_x;
        if (block < n_in) tile_body<W, EPI_W, false, OUT_W>(in, block, as, bs, nullptr);
        else tile_body<W, EPI_W, false, OUT_W>(down, block - n_in, as, bs, nullptr);
    }
}

// ---------------------------------------------------------------------------
// The epilogue of a product whose k was cut into slices: adds the slices'
// partial sums in their order.  Eight features of a token a thread.
// ---------------------------------------------------------------------------
constexpr int FINISH_BLOCK = 256;

template <int EPI, bool PAIR, int OUT>
__device__ __forceinline__ void finish_body(const TileArgs &p, bool bound_tokens, uint32_t block) {
    constexpr bool GATED = (EPI == EPI_GATED || EPI == EPI_QUANTIZE) && PAIR;
    const int32_t octs = (p.F + 7) / 8;
    const int32_t T = bound_tokens && p.live != nullptr ? clamp_live(p.live, p.T) : p.T;
    const int64_t i = (int64_t)block * FINISH_BLOCK + threadIdx.x;
    const int64_t t = i / octs;
    const int32_t f = (int32_t)(i - t * octs) * 8;
    float v[8] = {}, u[8] = {};
    Oct<OUT> zg, zu;
    if (t < T) {
        const int64_t row = GATED ? 2 * (int64_t)p.F : p.F;
        const uint32_t *at = (const uint32_t *)p.partial + t * row + f;
        if constexpr (EPI == EPI_BACKWARD) {
            using Z = typename Elem<OUT>::storage;
            const Z *z = (const Z *)p.z + t * (PAIR ? 2 * (int64_t)p.F : p.F) + f;
            oct_load<OUT, false>(zg, z, 8);
            if constexpr (PAIR) oct_load<OUT, false>(zu, z + p.F, 8);
        }
        // whole: no row ends within eight features, so the loads have no branch and several are on their way
        const auto add = [&](auto whole) {
            const int n = decltype(whole)::value ? 8 : p.F - f;
#pragma unroll 4
            for (int s = 0; s < p.splits; ++s) {
                Oct<DT_F32> o;
                float w[8];
                oct_load<DT_F32, false>(o, at + s * ((int64_t)p.T * row), n);
                oct_unpack<DT_F32>(o, w);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] += w[e];
                if constexpr (GATED) {
                    oct_load<DT_F32, false>(o, at + s * ((int64_t)p.T * row) + p.F, n);
                    oct_unpack<DT_F32>(o, w);
#pragma unroll
                    for (int e = 0; e < 8; ++e) u[e] += w[e];
                }
            }
        };
        if (p.F % 8 == 0) add(std::true_type());
        else add(std::false_type());
    }
    finish8<EPI, PAIR, OUT>(p, t, f, t < T, v, u, zg, zu);
}

template <int EPI, bool PAIR, int OUT>
__global__ __launch_bounds__(FINISH_BLOCK) void finish_kernel(TileArgs p, bool bound_tokens) {
    finish_body<EPI, PAIR, OUT>(p, bound_tokens, blockIdx.x);
}

// Those of three_kernel's products that were cut: n_x and n_in workgroups of the
// first two (0: not cut), the third's the rest.
template <int OUT>
__global__ __launch_bounds__(FINISH_BLOCK) void finish_three_kernel(TileArgs x, TileArgs in, TileArgs down, uint32_t n_x,
                                                                    uint32_t n_in) {
    const uint32_t block = blockIdx.x - n_x;
    if (blockIdx.x < n_x) finish_body<EPI_STORE, false, OUT>(x, true, blockIdx.x);
    else if (block < n_in) finish_body<EPI_STORE, false, OUT>(in, false, block);
    else finish_body<EPI_STORE, false, OUT>(down, false, block - n_in);
}

// ---------------------------------------------------------------------------
// Launches.
// ---------------------------------------------------------------------------
template <typename C, int EPI, bool PAIR, int OUT>
hipError_t launch_tile(const TileArgs &p, bool halves, hipStream_t stream) {
    const int64_t fw = halves ? C::FT / 2 : C::FT;
    const int64_t n = ((p.F + fw - 1) / fw) * (((int64_t)p.T + C::TT - 1) / C::TT) * p.splits;
    return launch_kernel(tile_kernel<C, EPI, PAIR, OUT>, dim3((uint32_t)n), dim3(C::W * 64), stream, p);
}

inline uint32_t finish_blocks(const TileArgs &p) {
    return (uint32_t)(((int64_t)p.T * ((p.F + 7) / 8) + FINISH_BLOCK - 1) / FINISH_BLOCK);
}

template <int EPI, bool PAIR, int OUT>
hipError_t launch_finish(const TileArgs &p, bool bound_tokens, hipStream_t stream) {
    return launch_kernel(finish_kernel<EPI, PAIR, OUT>, dim3(finish_blocks(p)), dim3(FINISH_BLOCK), stream, p, bound_tokens);
}

// Any of the three may be cut, in and down both or neither; a second launch then adds
// the slices of all of them.
template <int DT>
hipError_t launch_three(TileArgs x, TileArgs in, TileArgs down, const ThreePlan &plan, float *partial, hipStream_t stream) {
    const auto take = [&](TileArgs &p, const ProductPlan &q) {
        p.splits = q.splits;
        p.k_split = q.k_split;
        p.partial = partial;
        partial += q.partial_bytes / 4;
    };
    take(x, plan.x);
    take(in, plan.in);
    take(down, plan.down);
    const uint32_t n_x = (uint32_t)plan.x.workgroups, n_in = (uint32_t)plan.in.workgroups;
    const bool cut_x = x.splits > 1, cut_w = plan.cut_w;
    const auto kernel = cut_x ? cut_w ? three_kernel<DT, true, true> : three_kernel<DT, true, false>
                              : cut_w ? three_kernel<DT, false, true> : three_kernel<DT, false, false>;
    const hipError_t e = launch_kernel(kernel, dim3(n_x + n_in + (uint32_t)plan.down.workgroups), dim3(256), stream, x, in, down,
                                       n_x, n_in);
    if (e != hipSuccess || (!cut_x && !cut_w)) return e;
    const uint32_t f_x = cut_x ? finish_blocks(x) : 0, f_in = cut_w ? finish_blocks(in) : 0;
    return launch_kernel(finish_three_kernel<DT>, dim3(f_x + f_in + (cut_w ? finish_blocks(down) : 0)), dim3(FINISH_BLOCK),
                         stream, x, in, down, f_x, f_in);
}

}  // namespace ga
