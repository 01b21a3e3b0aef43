// Device functions of the 4-bit block-scaled kernels.
#pragma once

#include "mxfp4_internal.h"

namespace dps {

typedef float mx_f32x2 __attribute__((ext_vector_type(2)));
typedef float mx_f32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int mx_u32x2 __attribute__((ext_vector_type(2)));
typedef unsigned int mx_u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int mx_u32x4_e __attribute__((ext_vector_type(4), aligned(2)));
typedef __bf16 mx_bf16x2 __attribute__((ext_vector_type(2)));

// The scale byte of a block whose largest magnitude has the bits `top` (an
// fp32 pattern without its sign; NaN and infinity compare above every number):
// floor(log2 max) - 2, so that the largest value lands in e2m1's top octave
// [4, 8) and is held as 4 or 6; at least 2^-127. 255 marks a block with a NaN
// or an infinity.
__device__ __forceinline__ unsigned mx_scale_byte(unsigned top)
{
    return top >= 0x7f800000u ? 255u : (unsigned)max((int)(top >> 23) - 2, 0);
}
// 2^-e, by which a block's values are multiplied (exact: a power of two); the
// bytes 0 .. 252 of finite blocks give normal numbers
__device__ __forceinline__ float mx_inverse(unsigned byte) { return __uint_as_float((254u - byte) << 23); }

// 8 values (already multiplied by the inverse scale) to 8 codes, round to
// nearest even, saturating at 6
__device__ __forceinline__ unsigned mx_pack8(const float (&y)[8])
{
    unsigned w = 0;
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, y[0], y[1], 1.0f, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, y[2], y[3], 1.0f, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, y[4], y[5], 1.0f, 2);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, y[6], y[7], 1.0f, 3);
    return w;
}

}  // namespace dps
