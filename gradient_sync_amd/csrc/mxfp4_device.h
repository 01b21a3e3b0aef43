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
// 2^e as a float (2^-127 is one of fp32's subnormal numbers; the conversions below
// take it as they take the others)
__device__ __forceinline__ float mx_scale(unsigned byte)
{
    return __uint_as_float(byte == 0u ? 0x00400000u : byte << 23);
}

// 8 values over 2^e to 8 codes: round to nearest even, saturating at 6
__device__ __forceinline__ unsigned mx_pack8(const unsigned (&x)[8], float scale)
{
    unsigned w = 0;
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, __uint_as_float(x[0]), __uint_as_float(x[1]), scale, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, __uint_as_float(x[2]), __uint_as_float(x[3]), scale, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, __uint_as_float(x[4]), __uint_as_float(x[5]), scale, 2);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, __uint_as_float(x[6]), __uint_as_float(x[7]), scale, 3);
    return w;
}
// the same for 4 pairs of bf16
__device__ __forceinline__ unsigned mx_pack8(const unsigned (&x)[4], float scale)
{
    unsigned w = 0;
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(mx_bf16x2, x[0]), scale, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(mx_bf16x2, x[1]), scale, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(mx_bf16x2, x[2]), scale, 2);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(mx_bf16x2, x[3]), scale, 3);
    return w;
}

// larger magnitude so far, as bits: of fp32 values, or of the two halves of bf16 pairs
__device__ __forceinline__ unsigned mx_max_f32(unsigned top, unsigned x) { return max(top, x & 0x7fffffffu); }
__device__ __forceinline__ unsigned mx_max_bf16x2(unsigned top, unsigned x)
{
    typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(unsigned, __builtin_elementwise_max(__builtin_bit_cast(u16x2, top),
                                                                  __builtin_bit_cast(u16x2, x & 0x7fff7fffu)));
}

}  // namespace dps
