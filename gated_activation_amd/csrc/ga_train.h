// Device-side building blocks of the training kernels (gfx950, wave64): rows
// moved in octets of eight consecutive elements, fp64 row statistics, the
// 8-bit block code of activation checkpoints, and the activations with their
// derivatives.
#pragma once

#include "ga_device.h"

namespace ga {

// ---------------------------------------------------------------------------
// Octets: eight consecutive elements of a row per lane, so a 16-lane DPP row
// holds one block of BLOCK8 = 128 values and a block's maximum needs no LDS.
// The accesses are 16 bytes (two for fp32; 8 for codes) at the element's own
// alignment: gfx950 runs global memory in unaligned-access mode, so one form
// serves every alignment and only a row's last, partial octet (n < 8) goes
// element by element.  Elements past the row read as zero.
// ---------------------------------------------------------------------------
constexpr int BLOCK8 = 128;

typedef u32x4 u32x4_a4 __attribute__((aligned(4)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef u32x2 u32x2_a1 __attribute__((aligned(1)));

// An octet as loaded: the raw words, widened only when used.
template <int DT> struct Oct {
    static constexpr int WORDS = DT == DT_F32 ? 8 : 4;
    uint32_t w[WORDS];
};

template <int DT>
__device__ __forceinline__ void oct_zero(Oct<DT> &o) {
#pragma unroll
    for (int i = 0; i < Oct<DT>::WORDS; ++i) o.w[i] = 0;
}

template <int DT, bool NT = true>
__device__ __forceinline__ void oct_load(Oct<DT> &o, const typename Elem<DT>::storage *p, int n) {
    if (n >= 8) {
        if constexpr (DT == DT_F32) {
            const u32x4_a4 *q = reinterpret_cast<const u32x4_a4 *>(p);
            u32x4 a, b;
            if constexpr (NT) { a = __builtin_nontemporal_load(q); b = __builtin_nontemporal_load(q + 1); }
            else { a = q[0]; b = q[1]; }
            o.w[0] = a.x; o.w[1] = a.y; o.w[2] = a.z; o.w[3] = a.w;
            o.w[4] = b.x; o.w[5] = b.y; o.w[6] = b.z; o.w[7] = b.w;
        } else {
            const u32x4_a2 *q = reinterpret_cast<const u32x4_a2 *>(p);
            u32x4 a;
            if constexpr (NT) a = __builtin_nontemporal_load(q);
            else a = *q;
            o.w[0] = a.x; o.w[1] = a.y; o.w[2] = a.z; o.w[3] = a.w;
        }
    } else {
        oct_zero(o);
#pragma unroll
        for (int e = 0; e < 7; ++e) {
            if (e < n) {
                if constexpr (DT == DT_F32) o.w[e] = p[e];
                else o.w[e >> 1] |= (uint32_t)p[e] << ((e & 1) * 16);
            }
        }
    }
}

template <int DT>
__device__ __forceinline__ void oct_unpack(const Oct<DT> &o, float (&f)[8]) {
    if constexpr (DT == DT_F32) {
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = __builtin_bit_cast(float, o.w[e]);
    } else {
        Elem<DT>::unpack(uint4{o.w[0], o.w[1], o.w[2], o.w[3]}, f);
    }
}

// Rounds to the element type (ties to even) and stores the first n elements.
template <int DT, bool NT = true>
__device__ __forceinline__ void oct_store(typename Elem<DT>::storage *p, const float (&f)[8], int n) {
    if constexpr (DT == DT_F32) {
        if (n >= 8) {
            u32x4_a4 *q = reinterpret_cast<u32x4_a4 *>(p);
            const float lo[4] = {f[0], f[1], f[2], f[3]}, hi[4] = {f[4], f[5], f[6], f[7]};
            const uint4 a = Elem<DT>::pack(lo), b = Elem<DT>::pack(hi);
            const u32x4 va = {a.x, a.y, a.z, a.w}, vb = {b.x, b.y, b.z, b.w};
            if constexpr (NT) { __builtin_nontemporal_store(va, q); __builtin_nontemporal_store(vb, q + 1); }
            else { q[0] = va; q[1] = vb; }
        } else {
#pragma unroll
            for (int e = 0; e < 7; ++e)
                if (e < n) p[e] = Elem<DT>::from_f32(f[e]);
        }
    } else {
        const uint4 a = Elem<DT>::pack(f);
        if (n >= 8) {
            u32x4_a2 *q = reinterpret_cast<u32x4_a2 *>(p);
            const u32x4 va = {a.x, a.y, a.z, a.w};
            if constexpr (NT) __builtin_nontemporal_store(va, q);
            else *q = va;
        } else {
            const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int e = 0; e < 7; ++e)
                if (e < n) p[e] = (uint16_t)(w[e >> 1] >> ((e & 1) * 16));
        }
    }
}

// Between two uses of the same raw octet: without it the compiler keeps the
// first use's eight fp32 values for the second, twice the registers of a
// 16-bit octet and four times those of codes.
template <int DT>
__device__ __forceinline__ void stay_raw(Oct<DT> &o) {
#pragma unroll
    for (int i = 0; i < Oct<DT>::WORDS; ++i) asm volatile("" : "+v"(o.w[i]));
}
__device__ __forceinline__ void stay_raw(uint2 &k) { asm volatile("" : "+v"(k.x), "+v"(k.y)); }

// Eight codes of a checkpoint (two words, element e in byte e).
__device__ __forceinline__ uint2 codes_load(const uint8_t *p, int n) {
    if (n >= 8) {
        const u32x2 v = __builtin_nontemporal_load(reinterpret_cast<const u32x2_a1 *>(p));
        return uint2{v.x, v.y};
    }
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int e = 0; e < 7; ++e)
        if (e < n) w[e >> 2] |= (uint32_t)p[e] << ((e & 3) * 8);
    return uint2{w[0], w[1]};
}

__device__ __forceinline__ void codes_store(uint8_t *p, uint2 c, int n) {
    if (n >= 8) {
        __builtin_nontemporal_store(u32x2{c.x, c.y}, reinterpret_cast<u32x2_a1 *>(p));
        return;
    }
    const uint32_t w[2] = {c.x, c.y};
#pragma unroll
    for (int e = 0; e < 7; ++e)
        if (e < n) p[e] = (uint8_t)(w[e >> 2] >> ((e & 3) * 8));
}

// ---------------------------------------------------------------------------
// The same for kernels that hold a row in registers and load ahead.  A branch
// around a load makes the compiler wait for it where the paths meet, so these
// loads have none: fetch reads the eight elements from column c, or where they
// would pass the row's end the row's last eight, and trim, called when the
// octet is used, moves a partial octet's elements into place and clears the
// rest (all of an octet past the end).  TINY rows (d < 8) go element by
// element.
// ---------------------------------------------------------------------------
template <int DT, bool TINY, bool NT = true>
__device__ __forceinline__ void oct_fetch(Oct<DT> &o, const typename Elem<DT>::storage *row, int c, int d) {
    if constexpr (TINY) oct_load<DT, NT>(o, row + (uint32_t)c, d - c);
    else oct_load<DT, NT>(o, row + (uint32_t)(c < d - 8 ? c : d - 8), 8);
}

// Words i take words i + K where `on`, and 0 past the last.
template <int K, int DT>
__device__ __forceinline__ void words_down(Oct<DT> &o, bool on) {
#pragma unroll
    for (int i = 0; i < Oct<DT>::WORDS; ++i) {
        const uint32_t from = i + K < Oct<DT>::WORDS ? o.w[i + K < Oct<DT>::WORDS ? i + K : 0] : 0u;
        o.w[i] = on ? from : o.w[i];
    }
}

template <int DT, bool TINY>
__device__ __forceinline__ void oct_trim(Oct<DT> &o, int c, int d) {
    if constexpr (!TINY) {
        const int s = c - (d - 8);  // elements to drop
        if (s > 0) {
            if constexpr (DT == DT_F32) {
                words_down<4>(o, (s & 4) != 0);
                words_down<2>(o, (s & 2) != 0);
                words_down<1>(o, (s & 1) != 0);
            } else {
                words_down<2>(o, (s & 4) != 0);
                words_down<1>(o, (s & 2) != 0);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t from = o.w[i] >> 16 | (i < 3 ? o.w[i < 3 ? i + 1 : 0] << 16 : 0u);
                    o.w[i] = (s & 1) != 0 ? from : o.w[i];
                }
            }
            if (s >= 8) oct_zero(o);
        }
    }
}

template <bool TINY>
__device__ __forceinline__ uint2 codes_fetch(const uint8_t *row, int c, int d) {
    if constexpr (TINY) return codes_load(row + (uint32_t)c, d - c);
    else return codes_load(row + (uint32_t)(c < d - 8 ? c : d - 8), 8);
}

template <bool TINY>
__device__ __forceinline__ void codes_trim(uint2 &k, int c, int d) {
    if constexpr (!TINY) {
        if (c > d - 8) {
            const int s = c - (d - 8);
            const uint64_t v = s >= 8 ? 0 : ((uint64_t)k.y << 32 | k.x) >> (8 * s);
            k = uint2{(uint32_t)v, (uint32_t)(v >> 32)};
        }
    }
}

// ---------------------------------------------------------------------------
// The 8-bit block code.  For a block of up to 128 values with largest
// magnitude m (counted as at least 2^-100):
//     code = round-half-even(127 x / m), the exact quotient,
//     scale = m / 127 in fp32 (within 2^-23), the value it stands for code * scale.
// A block that holds a NaN, an infinity or a magnitude of 2^126 or more has
// the scale NaN, so every value restored from it is NaN and shows.
//
// The quotient is formed in fp32 as y = x inv, inv = 127 rcp(m).  Adding
// 1.5 * 2^23 rounds y to an integer (ties to even) and leaves the code in the
// low byte of the sum.  That is the exact quotient's rounding unless a
// half-integer h / 2 (h odd) lies on the quotient or between it and y:
//   x and m of 11 significant bits or fewer (fp16 and bf16 inputs), as
//   u 2^-j and M in units of m's last bit: 127 x / m = h / 2 or
//   |127 x / m - h / 2| = |254 u 2^-j - h M| / (2 M) >= 2^-j / 4094.  inv is
//   raised by 3 * 2^-23 here, so it lies above 127 / m, by at most 5 * 2^-23 of
//   it (the reciprocal is within 2^-23, two products round by 2^-24 each), and
//   y is off by less than 254 * 6e-7 * 2^-j.  So only ties matter: h M =
//   254 u 2^-j needs 127 to divide h M.  h = +-127 is x = +-m / 2, whose y above
//   63.5 rounds to 64, as ties to even do; otherwise 127 divides M (one block
//   in about 128), and that block's quotients are formed in fp64.
//   any fp32 x: y is within 2^-22 of itself, 3.03e-5 at 127.  A lane that has a
//   y within 4e-5 of a half-integer forms its quotients again in fp64, where
//   127 x is exact and the quotient's distance from a half-integer, if not
//   zero, is at least 2^-26.
//   fp32 differences of 16-bit rows from their mean or cutoff: y as it is, so a
//   quotient within 3.03e-5 of a half-integer may go to either side (the check
//   is 2.5 instructions a value of about 40).
// (Checking every y of 16-bit inputs too took the fp64 path in most
// wavefronts, since a bf16 block often holds half its largest value: the silu
// forward at 12288 rows of 768 then took 18.2 us, 14.1 us without, fastest of a
// trace.)
// POSITIVE keeps the code of every x > 0 at 1 or more, so x > 0 can be read
// back from the code exactly (an x below m / 254 then comes back as m / 127).
// All 16 lanes of a DPP row hold octets of one block and call this together.
// ---------------------------------------------------------------------------
constexpr float ROUND_MAGIC = 12582912.0f;
constexpr uint32_t LEAST_BITS = (127u - 100u) << 23;  // 2^-100
constexpr uint32_t MOST_BITS = (127u + 126u) << 23;   // 2^126: below it the reciprocal is normal

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_umax(uint32_t v) {
    const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false);
    return v > o ? v : o;
}

// Which of the three an octet's values are.
enum CodeOf { OF_F16, OF_BF16, OF_F32, OF_DIFFERENCE };
template <int DT> constexpr CodeOf code_of() { return DT == DT_F32 ? OF_F32 : DT == DT_F16 ? OF_F16 : OF_BF16; }
template <int DT> constexpr CodeOf difference_of() { return DT == DT_F32 ? OF_F32 : OF_DIFFERENCE; }

// What encodes a block: 127 / m, the scale, and m itself.
struct Block8 {
    float inv, scale, m;
    bool bad, check;
};

template <CodeOf OF>
__device__ __forceinline__ Block8 block_scale(const float (&x)[8]) {
    // the IEEE maximum, which a NaN wins
    float a = __builtin_fabsf(x[0]);
#pragma unroll
    for (int e = 1; e < 8; ++e) a = __builtin_elementwise_maximum(a, __builtin_fabsf(x[e]));
    // as integers: NaN above infinity above every number
    uint32_t top = __builtin_bit_cast(uint32_t, a) & 0x7FFFFFFFu;
    top = dpp_umax<0xB1>(top);
    top = dpp_umax<0x4E>(top);
    top = dpp_umax<0x141>(top);
    top = dpp_umax<0x140>(top);
    Block8 b;
    b.bad = top >= MOST_BITS;
    top = top > LEAST_BITS ? top : LEAST_BITS;
    b.m = __builtin_bit_cast(float, b.bad ? 0x3F800000u : top);
    b.inv = 127.0f * __builtin_amdgcn_rcpf(b.m);
    if constexpr (OF == OF_F16 || OF == OF_BF16) b.inv *= 1.0f + 0x3p-23f;
    b.scale = b.bad ? __builtin_nanf("") : b.m * (1.0f / 127.0f);
    // does 127 divide m's significand?
    if constexpr (OF == OF_F16) b.check = (1024u + ((top >> 13) & 0x3FFu)) % 127u == 0u;
    else b.check = OF == OF_BF16 && (top & 0x7F0000u) == 0x7E0000u;
    return b;
}

template <CodeOf OF, bool POSITIVE>
__device__ __forceinline__ uint2 block_codes(const Block8 &b, const float (&x)[8]) {
    float y[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = __builtin_fmaf(x[e], b.inv, ROUND_MAGIC);
    bool again = b.check;
    if constexpr (OF == OF_F32) {
        float off = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            off = __builtin_fmaxf(off, __builtin_fabsf(__builtin_fmaf(x[e], b.inv, -(y[e] - ROUND_MAGIC))));
        again = off > 0.49996f;
    }
    if (OF != OF_DIFFERENCE && again) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            y[e] = (float)__builtin_rint(127.0 * (double)x[e] / (double)b.m) + ROUND_MAGIC;
    }
    if constexpr (POSITIVE) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (x[e] > 0.0f) y[e] = __builtin_fmaxf(y[e], ROUND_MAGIC + 1.0f);
    }
    uint32_t w[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t b0 = __builtin_bit_cast(uint32_t, y[4 * h]), b1 = __builtin_bit_cast(uint32_t, y[4 * h + 1]);
        const uint32_t b2 = __builtin_bit_cast(uint32_t, y[4 * h + 2]), b3 = __builtin_bit_cast(uint32_t, y[4 * h + 3]);
        // v_perm_b32 selects bytes of {src0, src1}: 0..3 from src1, 4..7 from src0
        const uint32_t lo = __builtin_amdgcn_perm(b1, b0, 0x0C0C0400u);
        const uint32_t hi = __builtin_amdgcn_perm(b3, b2, 0x0C0C0400u);
        w[h] = b.bad ? 0u : __builtin_amdgcn_perm(hi, lo, 0x05040100u);
    }
    return uint2{w[0], w[1]};
}

template <CodeOf OF, bool POSITIVE>
__device__ __forceinline__ uint2 block_encode(const float (&x)[8], float &scale) {
    const Block8 b = block_scale<OF>(x);
    scale = b.scale;
    return block_codes<OF, POSITIVE>(b, x);
}

// code * scale, rounded once: the byte with its sign bit flipped is code + 128,
// and -128 * scale is exact.
__device__ __forceinline__ void block_decode(uint2 c, float scale, float (&f)[8]) {
    const float base = -128.0f * scale;
    const uint32_t w[2] = {c.x ^ 0x80808080u, c.y ^ 0x80808080u};
#pragma unroll
    for (int e = 0; e < 8; ++e)
        f[e] = __builtin_fmaf((float)((w[e >> 2] >> ((e & 3) * 8)) & 0xFFu), scale, base);
}

// max(x, 0).  A NaN gives 0, as in the forward pass; restored from codes (KEPT)
// it stays NaN, since a block's NaN scale stands for finite values too.
template <bool KEPT>
__device__ __forceinline__ float above_zero(float x) {
    if constexpr (KEPT) return __builtin_elementwise_maximum(x, 0.0f);
    else return __builtin_fmaxf(x, 0.0f);
}

// ---------------------------------------------------------------------------
// Row sums in fp64 (as fast as fp32 on this device outside packed math): lanes
// paired as in wave_sum, so the result is the same on every lane.
// ---------------------------------------------------------------------------
template <int CTRL>
__device__ __forceinline__ double dpp_move64(double v) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_mov_dpp((int)(uint32_t)b, CTRL, 0xF, 0xF, true);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_mov_dpp((int)(uint32_t)(b >> 32), CTRL, 0xF, 0xF, true);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

__device__ __forceinline__ double read_lane64(double v, int lane) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)b, lane);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(b >> 32), lane);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

__device__ __forceinline__ double row16_sum(double v) {
    v += dpp_move64<0xB1>(v);
    v += dpp_move64<0x4E>(v);
    v += dpp_move64<0x141>(v);
    v += dpp_move64<0x140>(v);
    return v;
}

__device__ __forceinline__ float row16_sum(float v) {
    v += dpp_move<0xB1>(v);
    v += dpp_move<0x4E>(v);
    v += dpp_move<0x141>(v);
    v += dpp_move<0x140>(v);
    return v;
}

__device__ __forceinline__ double wave_sum(double v) {
    v = row16_sum(v);
    return (read_lane64(v, 0) + read_lane64(v, 16)) + (read_lane64(v, 32) + read_lane64(v, 48));
}

// A team's row as a scalar where a team is one wavefront or more.
template <int LANES>
__device__ __forceinline__ uint32_t team_row(uint32_t row) {
    if constexpr (LANES >= 64) return (uint32_t)__builtin_amdgcn_readfirstlane((int)row);
    else return row;
}

// Sums of N values over the team that shares a row: 16 lanes, a wavefront, or
// LANES / 64 wavefronts of a workgroup (all of whose teams call it together).
// `slots`: LDS of the team's own, N * LANES / 64 values that nothing else
// touches until the next barrier after this call.
template <int LANES, int N, typename T>
__device__ __forceinline__ void team_sums(T (&v)[N], T *slots) {
#pragma unroll
    for (int k = 0; k < N; ++k) {
        if constexpr (LANES == 16) v[k] = row16_sum(v[k]);
        else v[k] = wave_sum(v[k]);
    }
    if constexpr (LANES > 64) {
        constexpr int W = LANES / 64;
        const int wave = (threadIdx.x % LANES) >> 6;
        if ((threadIdx.x & 63) == 0) {
#pragma unroll
            for (int k = 0; k < N; ++k) slots[N * wave + k] = v[k];
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < N; ++k) v[k] = slots[k];
#pragma unroll
        for (int i = 1; i < W; ++i)
#pragma unroll
            for (int k = 0; k < N; ++k) v[k] += slots[N * i + k];
    }
}

template <int LANES, typename T>
__device__ __forceinline__ void team_sum2(T &a, T &b, T *slots) {
    T v[2] = {a, b};
    team_sums<LANES>(v, slots);
    a = v[0];
    b = v[1];
}

// The value a row's sums are taken from: the median of its first, middle and
// last, so that one value far out is not it.
template <int DT>
__device__ __forceinline__ float row_pivot(const typename Elem<DT>::storage *row, int d) {
    return __builtin_amdgcn_fmed3f(Elem<DT>::to_f32(row[0]), Elem<DT>::to_f32(row[d / 2]), Elem<DT>::to_f32(row[d - 1]));
}

// Adds an octet's x - x0 and (x - x0)^2 to fp64 sums.  The differences are
// fp64 for 16-bit rows too: the pivot may be far out (two of the three values it
// is the median of), and fp32 differences to it would then carry 2^-24 of it,
// one-sided where many values are alike: 1.4e-3 of the mean for rows of 1.46e-3
// with 60000 in those places.
__device__ __forceinline__ void add_shifted(const float (&x)[8], float x0, double &s1, double &s2) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const double a = (double)x[e] - (double)x0;
        s1 += a;
        s2 = __builtin_fma(a, a, s2);
    }
}

// x - at, at an fp64 value of the row.  16-bit rows take at as the sum of two
// fp32 numbers: x - hi is exact where x is near hi, so the difference's sign
// is exact and its value within two roundings; fp32 rows round it once.
template <int DT> struct RowOrigin {
    float hi, lo;
    double at;
    __device__ __forceinline__ explicit RowOrigin(double v) : hi((float)v), lo((float)(v - (double)(float)v)), at(v) {}
    __device__ __forceinline__ float from(float x) const {
        if constexpr (DT == DT_F32) return (float)((double)x - at);
        else return (x - hi) - lo;
    }
};

// Mean and population variance of d values from the sums of x - x0 and of its
// square, x0 being the row's pivot: one pass, one reduction, and a row
// of one repeated value has variance 0 exactly.  In fp64 the differences of
// fp32 values are exact or carry 2^-53, and the subtraction loses at most
// (mean - x0)^2 / var <= d <= 2^16 times that.
__device__ __forceinline__ void shifted_moments(double s1, double s2, double x0, double inv_d, double &mean, double &var) {
    const double m = s1 * inv_d;
    const double v = s2 * inv_d - m * m;
    mean = x0 + m;
    var = v > 0.0 ? v : (v == v ? 0.0 : v);  // a NaN stays one
}

// ---------------------------------------------------------------------------
// Activations with their derivatives, fp32.  ACT: the op codes of ga_internal.h.
//   silu: p = 1 / (1 + e^-x); f = x p, f' = p + f (1 - p)
//   gelu, tanh form: p = 1 / (1 + 2^(-x (A + B x^2))) (see gelu_tanh); f = x p,
//     f' = p + f (1 - p) (1 + 3 * 0.044715 x^2) 2 sqrt(2 / pi)
//   gelu, erf form: f = x Phi(x), f' = Phi(x) + x phi(x)
//   squared relu: r = max(x, 0); f = r^2, f' = 2 r
// For x << 0 p is 0 and f (1 - p) is x * 0; the power can overflow to +inf
// (p = 0), never to NaN for finite x.
// ---------------------------------------------------------------------------
constexpr float GELU_DA = 1.5957691216057308f;   // 2 sqrt(2 / pi)
constexpr float GELU_DB = 0.21406444881780073f;  // 3 * 0.044715 * 2 sqrt(2 / pi)
constexpr float INV_SQRT_2PI = 0.3989422804014327f;

__device__ __forceinline__ void gelu_tanh_slope(float x, float &f, float &df) {
    const float x2 = x * x;
    const float p = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-x * __builtin_fmaf(GELU_B, x2, GELU_A)));
    f = x * p;
    const float q = f * (1.0f - p);
    df = q == 0.0f ? p : __builtin_fmaf(q, __builtin_fmaf(GELU_DB, x2, GELU_DA), p);  // x^2 may be +inf there
}

__device__ __forceinline__ void silu_slope(float x, float &f, float &df) {
    const float p = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-x * LOG2_E));
    f = x * p;
    df = __builtin_fmaf(f, 1.0f - p, p);
}

// Phi(x) = 0.5 erfc(-x / sqrt 2) with erfc_nonneg's rational approximation
// (absolute error below 1.5e-7), whose e^(-x^2 / 2) also gives phi(x).
__device__ __forceinline__ void gelu_erf_slope(float x, float &f, float &df) {
    const float a = __builtin_fabsf(x) * 0.70710678118654752f;
    const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.3275911f, a, 1.0f));
    const float e = __builtin_amdgcn_exp2f(-a * a * LOG2_E);
    float poly = __builtin_fmaf(1.061405429f, t, -1.453152027f);
    poly = __builtin_fmaf(poly, t, 1.421413741f);
    poly = __builtin_fmaf(poly, t, -0.284496736f);
    poly = __builtin_fmaf(poly, t, 0.254829592f);
    const float h = 0.5f * poly * t * e;
    const float cdf = x < 0.0f ? h : 1.0f - h;
    f = x * cdf;
    df = __builtin_fmaf(x, INV_SQRT_2PI * e, cdf);
}

// Division of n < 2^31 by a fixed divisor, by Granlund and Montgomery's round-up
// multiplication (1994): (mulhi(n, mul) + n) >> shift with
// shift = ceil(log2 divisor), mul = floor(2^32 (2^shift - divisor) / divisor) + 1.
struct FastDiv {
    uint32_t mul, shift;
    __host__ explicit FastDiv(uint32_t divisor) {
        shift = 0;
        while (((uint64_t)1 << shift) < divisor) ++shift;
        mul = (uint32_t)((((uint64_t)1 << 32) * (((uint64_t)1 << shift) - divisor)) / divisor + 1);
    }
    __device__ __forceinline__ uint32_t operator()(uint32_t n) const { return (__umulhi(n, mul) + n) >> shift; }
};

}  // namespace ga
