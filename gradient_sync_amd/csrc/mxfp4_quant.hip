// Quantisation to 4-bit floating point with a power-of-two scale per block of
// 32 values, and its inverse.
//
//   e = max(floor(log2 max|x|) - 2, -127);  code = e2m1(x 2^-e)
//
// rounded to nearest even over e2m1's values 0, 1/2, 1, 3/2, 2, 3, 4, 6 (a
// value above 5 is held as 6). The multiplication by 2^-e is exact, so the
// codes depend on nothing but x.
//
// A product sums along the blocks, so a matrix whose transpose enters another
// product (the backward pass) is needed in both orientations; one launch
// reads it once and writes either or both.
#include "mxfp4_device.h"

namespace dps {
namespace {

constexpr int kTile = 128;      // rows and columns of a workgroup's tile: 64-byte runs of codes both ways
constexpr int kNT = 256;

template <int DT> struct In;
template <> struct In<kBF16> { static constexpr int W = 4; };   // dwords per 8 elements
template <> struct In<kF32> { static constexpr int W = 8; };

template <int DT>
__device__ __forceinline__ float elem(const unsigned *w, int i)
{
    if constexpr (DT == kF32) return __uint_as_float(w[i]);
    return __uint_as_float(i & 1 ? w[i >> 1] & 0xffff0000u : w[i >> 1] << 16);
}

// 8 consecutive elements of a row from column c, zero past the matrix
template <int DT>
__device__ __forceinline__ void load8(const MxQuantParams &p, long long r, long long c, unsigned (&w)[In<DT>::W])
{
    constexpr int ES = DT == kBF16 ? 2 : 4;
    const char *at = p.src + (r * p.ld + c) * ES;
    if (r < p.rows && c + 8 <= p.cols) {
#pragma unroll
        for (int h = 0; h < In<DT>::W / 4; ++h) {
            const mx_u32x4 v = *reinterpret_cast<const mx_u32x4_e *>(at + 16 * h);
#pragma unroll
            for (int i = 0; i < 4; ++i) w[4 * h + i] = v[i];
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < In<DT>::W; ++i) w[i] = 0;
    if (r >= p.rows) return;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (c + i < p.cols) {
            if constexpr (DT == kF32)
                w[i] = reinterpret_cast<const unsigned *>(at)[i];
            else
                w[i >> 1] |= (unsigned)reinterpret_cast<const unsigned short *>(at)[i] << (16 * (i & 1));
        }
}

template <int DT, bool ROW, bool COL>
__global__ __launch_bounds__(kNT) void mxfp4_quantize_kernel(const MxQuantParams p, int tiles_c)
{
    constexpr int W = In<DT>::W;
    // the tile, its 4-column groups permuted within a row by the row's block,
    // so that the column reads below, 4 row blocks side by side, hit
    // distinct banks
    __shared__ __attribute__((aligned(16))) unsigned lds[COL ? kTile * kTile * (DT == kBF16 ? 2 : 4) / 4 : 1];
    const int tid = threadIdx.x;
    const int tr = blockIdx.x / tiles_c, tc = blockIdx.x - tr * tiles_c;
    const long long row0 = (long long)tr * kTile, col0 = (long long)tc * kTile;
    const int c8 = tid & 15;
    unsigned w[8][W];
#pragma unroll
    for (int q = 0; q < 8; ++q) load8<DT>(p, row0 + q * 16 + (tid >> 4), col0 + c8 * 8, w[q]);
    const long long pitch = mx_pitch(p.cols), st = mx_scale_tiles(p.cols);
#pragma unroll
    for (int q = 0; q < 8; ++q) {
        const int lr = q * 16 + (tid >> 4);
        const long long r = row0 + lr;
        if constexpr (ROW) {
            unsigned top = 0;
            if constexpr (DT == kF32) {
#pragma unroll
                for (int i = 0; i < 8; ++i) top = max(top, w[q][i] & 0x7fffffffu);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    top = max(top, max((w[q][i] << 16) & 0x7fffffffu, w[q][i] & 0x7fff0000u));
            }
            top = max(top, (unsigned)__builtin_amdgcn_update_dpp(0, (int)top, 0xB1, 0xf, 0xf, false));  // lane ^ 1
            top = max(top, (unsigned)__builtin_amdgcn_update_dpp(0, (int)top, 0x4E, 0xf, 0xf, false));  // lane ^ 2
            const unsigned byte = mx_scale_byte(top);
            const float inv = mx_inverse(byte);
            float y[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = elem<DT>(w[q], i) * inv;
            const unsigned code = byte == 255u ? 0u : mx_pack8(y);
            if (r < p.rows) {
                *reinterpret_cast<unsigned *>(p.codes + r * pitch + tc * 64 + c8 * 4) = code;
                if ((tid & 3) == 0) p.scales[mx_scale_at(r, tc * 4 + (c8 >> 2), st)] = (unsigned char)byte;
            }
        }
        if constexpr (COL) {
            const int swz = (lr >> 5) & 3;
#pragma unroll
            for (int h = 0; h < W / 4; ++h) {
                const int chunk = (c8 * (W / 4) + h) ^ (swz * W);
                *reinterpret_cast<mx_u32x4 *>(&lds[lr * (kTile * W / 8) + chunk * 4]) =
                    mx_u32x4{w[q][4 * h], w[q][4 * h + 1], w[q][4 * h + 2], w[q][4 * h + 3]};
            }
        }
    }
    if constexpr (COL) {
        __syncthreads();
        const int rb = tid & 3, cp = tid >> 2;       // block of 32 rows, pair of columns
        const long long pitch_t = mx_pitch(p.rows), st_t = mx_scale_tiles(p.rows);
        float x[2][32];
#pragma unroll
        for (int j = 0; j < 32; ++j) {
            const int at = (rb * 32 + j) * (kTile * W / 8) + (cp ^ (16 * rb)) * (W / 4);
            if constexpr (DT == kBF16) {
                x[0][j] = __uint_as_float(lds[at] << 16);
                x[1][j] = __uint_as_float(lds[at] & 0xffff0000u);
            } else {
                const mx_u32x2 v = *reinterpret_cast<const mx_u32x2 *>(&lds[at]);
                x[0][j] = __uint_as_float(v[0]);
                x[1][j] = __uint_as_float(v[1]);
            }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            unsigned top = 0;
#pragma unroll
            for (int j = 0; j < 32; ++j) top = max(top, __float_as_uint(x[h][j]) & 0x7fffffffu);
            const unsigned byte = mx_scale_byte(top);
            const float inv = mx_inverse(byte);
            mx_u32x4 code;
#pragma unroll
            for (int o = 0; o < 4; ++o) {
                float y[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] = x[h][8 * o + i] * inv;
                code[o] = byte == 255u ? 0u : mx_pack8(y);
            }
            const long long c = col0 + cp * 2 + h;
            if (c < p.cols) {
                *reinterpret_cast<mx_u32x4 *>(p.codes_t + c * pitch_t + tr * 64 + rb * 16) = code;
                p.scales_t[mx_scale_at(c, tr * 4 + rb, st_t)] = (unsigned char)byte;
            }
        }
    }
}

// One thread expands 8 codes (half of them for an odd tail).
template <int DT>
__global__ __launch_bounds__(kNT) void mxfp4_dequantize_kernel(const MxExpandParams p, long long groups)
{
    const long long id = (long long)blockIdx.x * kNT + threadIdx.x;
    const long long r = id / groups, g = id - r * groups;
    if (r >= p.rows) return;
    const unsigned w = *reinterpret_cast<const unsigned *>(p.codes + r * mx_pitch(p.cols) + g * 4);
    const unsigned byte = p.scales[mx_scale_at(r, (int)(g >> 2), mx_scale_tiles(p.cols))];
    const float scale = byte == 255u ? __uint_as_float(0x7fc00000u)
                        : byte == 0u ? 0x1p-127f : __uint_as_float(byte << 23);
    float x[8];
#define DPS_EXPAND(i)                                                              \
    {                                                                              \
        const auto v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, i);       \
        x[2 * i] = v[0] * scale;                                                   \
        x[2 * i + 1] = v[1] * scale;                                               \
    }
    DPS_EXPAND(0) DPS_EXPAND(1) DPS_EXPAND(2) DPS_EXPAND(3)
#undef DPS_EXPAND
    const long long at = r * p.ld + g * 8;
    const int n = (int)min(8LL, p.cols - g * 8);
    if constexpr (DT == kF32) {
        float *d = reinterpret_cast<float *>(p.dst) + at;
        typedef float f32x4_e __attribute__((ext_vector_type(4), aligned(4)));
        if (n == 8) {
            *reinterpret_cast<f32x4_e *>(d) = f32x4_e{x[0], x[1], x[2], x[3]};
            *reinterpret_cast<f32x4_e *>(d + 4) = f32x4_e{x[4], x[5], x[6], x[7]};
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < n) d[i] = x[i];
        }
    } else {
        unsigned short *d = reinterpret_cast<unsigned short *>(p.dst) + at;
        mx_u32x4 o;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const mx_f32x2 v = {x[2 * i], x[2 * i + 1]};
            o[i] = __builtin_bit_cast(unsigned, __builtin_convertvector(v, mx_bf16x2));
        }
        if (n == 8) {
            *reinterpret_cast<mx_u32x4_e *>(d) = o;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < n) d[i] = (unsigned short)(o[i >> 1] >> (16 * (i & 1)));
        }
    }
}

template <int DT>
hipError_t quantize_typed(const MxQuantParams &p, hipStream_t stream)
{
    const long long tr = (p.rows + kTile - 1) / kTile, tc = (p.cols + kTile - 1) / kTile;
    const int grid = (int)(tr * tc);
    if (p.codes && p.codes_t)
        mxfp4_quantize_kernel<DT, true, true><<<grid, kNT, 0, stream>>>(p, (int)tc);
    else if (p.codes)
        mxfp4_quantize_kernel<DT, true, false><<<grid, kNT, 0, stream>>>(p, (int)tc);
    else
        mxfp4_quantize_kernel<DT, false, true><<<grid, kNT, 0, stream>>>(p, (int)tc);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_mxfp4_quantize(const MxQuantParams &p, int dt, hipStream_t stream)
{
    return dt == kBF16 ? quantize_typed<kBF16>(p, stream) : quantize_typed<kF32>(p, stream);
}

hipError_t launch_mxfp4_dequantize(const MxExpandParams &p, int dt, hipStream_t stream)
{
    const long long groups = (p.cols + 7) / 8;
    const unsigned grid = (unsigned)((p.rows * groups + kNT - 1) / kNT);
    if (dt == kBF16)
        mxfp4_dequantize_kernel<kBF16><<<grid, kNT, 0, stream>>>(p, groups);
    else
        mxfp4_dequantize_kernel<kF32><<<grid, kNT, 0, stream>>>(p, groups);
    return hipGetLastError();
}

}  // namespace dps
