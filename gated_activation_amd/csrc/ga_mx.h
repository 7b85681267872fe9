// Microscaled 4-bit values (OCP MX, e2m1 with E8M0 scales): device code shared
// by the quantising kernels and the products' epilogues.
//
// A block is 32 consecutive values of a row, the last one of a row shorter.
// With m its largest magnitude, E m's exponent field (so floor(log2 m) = E - 127
// where m is normal):
//     scale byte s = max(E - 2, 0), standing for 2^(s - 127); the 2 brings m
//     into [4, 8), the binade of the largest value, 6
//     code = x 2^(127 - s) rounded to the nearest of 0, 1/2, 1, 3/2, 2, 3, 4, 6
//     with x's sign, ties to the even code, 6 above 6
// x 2^(127 - s) is exact in fp32 (what underflows is far below 1/4), so a code is
// the correctly rounded one of any fp16, bf16 or fp32 value.  A block that holds
// a NaN or an infinity has s = 255 and codes of 0: it stands for NaNs.
#pragma once

#include "ga_device.h"

namespace ga {

constexpr int MX_BLOCK = 32;
constexpr uint32_t MX_NAN = 255;

// As integers, the magnitudes of finite numbers keep their order below infinity
// and NaN.
__device__ __forceinline__ uint32_t magnitude(float x) { return __builtin_bit_cast(uint32_t, x) & 0x7FFFFFFFu; }

__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t top) {
    const uint32_t e = top >> 23;
    return e == 255 ? MX_NAN : e > 2 ? e - 2 : 0;
}

// Eight codes of a block with scale byte s, element e in nibble e.
__device__ __forceinline__ uint32_t mx_codes8(const float (&x)[8], uint32_t s) {
    const float up = __builtin_bit_cast(float, (254 - s) << 23);
    uint32_t w = 0;
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[0] * up, x[1] * up, 1.0f, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[2] * up, x[3] * up, 1.0f, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[4] * up, x[5] * up, 1.0f, 2);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[6] * up, x[7] * up, 1.0f, 3);
    return s == MX_NAN ? 0 : w;
}

// 2^(s - 127) (a denormal for s = 0), NaN for 255.
__device__ __forceinline__ float mx_scale(uint32_t s) {
    return __builtin_bit_cast(float, s == 0 ? 0x00400000u : s == MX_NAN ? 0x7FC00000u : s << 23);
}

__device__ __forceinline__ void mx_values8(uint32_t w, uint32_t s, float (&x)[8]) {
    const float scale = mx_scale(s);
    f32x2 v[4];
    v[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 0);
    v[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 1);
    v[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 2);
    v[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 3);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = v[e / 2][e % 2] * scale;
}

}  // namespace ga
