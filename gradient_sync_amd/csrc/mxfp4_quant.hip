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

// 8 consecutive elements of a row from column c, zero past the matrix
template <int DT>
__device__ __forceinline__ void load8(const MxQuantParams &p, long long r, long long c, unsigned (&w)[In<DT>::W])
{
    constexpr int ES = DT == kBF16 ? 2 : 4;
    const char *at = p.src + (r * p.ld + c) * ES;
    if (r < p.rows && c + 8 <= p.cols) {
#pragma unroll
        for (int h = 0; h < In<DT>::W / 4; ++h) {
            // read once: nontemporal (8192 x 4096 bf16: 15.5 us for 17.1)
            const mx_u32x4 v = __builtin_nontemporal_load(reinterpret_cast<const mx_u32x4_e *>(at + 16 * h));
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

// The codes of this lane's 8 values of a row, 4 lanes a block, and their scale byte.
template <int DT>
__device__ __forceinline__ unsigned row_codes(const unsigned (&w)[In<DT>::W], unsigned &byte)
{
    unsigned top = 0;
#pragma unroll
    for (int i = 0; i < In<DT>::W; ++i) top = DT == kF32 ? mx_max_f32(top, w[i]) : mx_max_bf16x2(top, w[i]);
    if constexpr (DT == kBF16) top = max(top << 16, top & 0xffff0000u);
    top = max(top, (unsigned)__builtin_amdgcn_update_dpp(0, (int)top, 0xB1, 0xf, 0xf, false));  // lane ^ 1
    top = max(top, (unsigned)__builtin_amdgcn_update_dpp(0, (int)top, 0x4E, 0xf, 0xf, false));  // lane ^ 2
    byte = mx_scale_byte(top);
    return byte == 255u ? 0u : mx_pack8(w, mx_scale(byte));
}

// Along the rows alone: a workgroup takes 16 rows by 512 columns, one tile of
// scales, a wave 4 of the rows. A row is 1 KiB (bf16) of consecutive loads and
// 256 bytes of codes; the tile's 256 scale bytes are put in order in LDS and
// leave in one store. HBM-bound: 8192 x 4096 bf16 in 15.5 us (5.5 TB/s).
template <int DT>
__global__ __launch_bounds__(kNT) void mxfp4_quantize_rows_kernel(const MxQuantParams p, int tiles)
{
    __shared__ __attribute__((aligned(16))) unsigned char lds[256];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int group = blockIdx.x / tiles, kt = blockIdx.x - group * tiles;
    const long long pitch = mx_pitch(p.cols), col = kt * 512LL + lane * 8;
    const int at = kt * 256 + lane * 4;
    unsigned w[4][In<DT>::W];
#pragma unroll
    for (int r = 0; r < 4; ++r) load8<DT>(p, group * 16LL + wave * 4 + r, col, w[r]);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const long long row = group * 16LL + wave * 4 + r;
        unsigned byte;
        const unsigned code = row_codes<DT>(w[r], byte);
        if (row < p.rows && at < pitch) *reinterpret_cast<unsigned *>(p.codes + row * pitch + at) = code;
        if ((lane & 3) == 0) lds[mx_scale_at(wave * 4 + r, lane >> 2, 1)] = (unsigned char)byte;
    }
    __syncthreads();
    if (wave == 0)
        reinterpret_cast<unsigned *>(p.scales + blockIdx.x * 256LL)[lane] = reinterpret_cast<const unsigned *>(lds)[lane];
}

// Along the columns, and along the rows too with ROW: a workgroup reads a tile of
// 128 x 128, quantises its rows from registers, and its columns from LDS, a
// thread 32 rows of two neighbouring columns. HBM-bound, with 9% more written
// than needed (scale bytes leave one by one): 14336 x 4096 bf16 both ways in
// 37.8 us (4.75 TB/s), along the columns alone in 29.1 (5.1 TB/s).
template <int DT, bool ROW>
__global__ __launch_bounds__(kNT) void mxfp4_quantize_cols_kernel(const MxQuantParams p, int tiles_c)
{
    constexpr int W = In<DT>::W, PITCH = kTile * W / 8;      // dwords per row of the tile
    // 4-column groups permuted within a row by the row's block, so that the
    // column reads below, 4 row blocks side by side, hit distinct banks
    __shared__ __attribute__((aligned(16))) unsigned lds[kTile * PITCH];
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
#pragma unroll
        for (int h = 0; h < W / 4; ++h) {
            const int chunk = (c8 * (W / 4) + h) ^ (((lr >> 5) & 3) * W);
            *reinterpret_cast<mx_u32x4 *>(&lds[lr * PITCH + chunk * 4]) =
                mx_u32x4{w[q][4 * h], w[q][4 * h + 1], w[q][4 * h + 2], w[q][4 * h + 3]};
        }
        if constexpr (ROW) {
            const long long r = row0 + lr;
            unsigned byte;
            const unsigned code = row_codes<DT>(w[q], byte);
            if (r < p.rows) {
                *reinterpret_cast<unsigned *>(p.codes + r * pitch + tc * 64 + c8 * 4) = code;
                if ((tid & 3) == 0) p.scales[mx_scale_at(r, tc * 4 + (c8 >> 2), st)] = (unsigned char)byte;
            }
        }
    }
    __syncthreads();
    const int rb = tid & 3, cp = tid >> 2;           // block of 32 rows, pair of columns
    const long long pitch_t = mx_pitch(p.rows), st_t = mx_scale_tiles(p.rows);
    const unsigned *mine = lds + rb * 32 * PITCH + (cp ^ (16 * rb)) * (W / 4);
    unsigned top[2] = {0, 0}, x[DT == kBF16 ? 1 : 2][32];
#pragma unroll
    for (int j = 0; j < 32; ++j) {
        if constexpr (DT == kBF16) {
            x[0][j] = mine[j * PITCH];
            top[0] = mx_max_bf16x2(top[0], x[0][j]);
        } else {
            const mx_u32x2 v = *reinterpret_cast<const mx_u32x2 *>(mine + j * PITCH);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                x[h][j] = v[h];
                top[h] = mx_max_f32(top[h], v[h]);
            }
        }
    }
    if constexpr (DT == kBF16) {
        top[1] = top[0] & 0xffff0000u;
        top[0] <<= 16;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const unsigned byte = mx_scale_byte(top[h]);
        const float scale = mx_scale(byte);
        mx_u32x4 code;
#pragma unroll
        for (int o = 0; o < 4; ++o) {
            unsigned y[W];
#pragma unroll
            for (int i = 0; i < W; ++i) {
                if constexpr (DT == kBF16)           // one column's values of two rows
                    y[i] = __builtin_amdgcn_perm(x[0][8 * o + 2 * i + 1], x[0][8 * o + 2 * i], h ? 0x07060302u : 0x05040100u);
                else
                    y[i] = x[h][8 * o + i];
            }
            code[o] = byte == 255u ? 0u : mx_pack8(y, scale);
        }
        const long long c = col0 + cp * 2 + h;
        if (c < p.cols) {
            *reinterpret_cast<mx_u32x4 *>(p.codes_t + c * pitch_t + tr * 64 + rb * 16) = code;
            p.scales_t[mx_scale_at(c, tr * 4 + rb, st_t)] = (unsigned char)byte;
        }
    }
}

// One thread expands 8 codes, fewer at a row's end. HBM-bound: 14336 x 4096 to
// bf16 in 24.2 us (6.1 TB/s).
template <int DT>
__global__ __launch_bounds__(kNT) void mxfp4_dequantize_kernel(const MxExpandParams p, long long groups, unsigned first)
{
    const long long id = ((long long)first + blockIdx.x) * kNT + threadIdx.x;
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
    if (!p.codes_t) {
        const long long tiles = mx_scale_tiles(p.cols);
        mxfp4_quantize_rows_kernel<DT><<<(unsigned)((p.rows + 15) / 16 * tiles), kNT, 0, stream>>>(p, (int)tiles);
        return hipGetLastError();
    }
    const long long tr = (p.rows + kTile - 1) / kTile, tc = (p.cols + kTile - 1) / kTile;
    if (p.codes)
        mxfp4_quantize_cols_kernel<DT, true><<<(unsigned)(tr * tc), kNT, 0, stream>>>(p, (int)tc);
    else
        mxfp4_quantize_cols_kernel<DT, false><<<(unsigned)(tr * tc), kNT, 0, stream>>>(p, (int)tc);
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
    return launch_groups256((p.rows * groups + kNT - 1) / kNT, [&](unsigned first, unsigned grid) {
        if (dt == kBF16)
            mxfp4_dequantize_kernel<kBF16><<<grid, kNT, 0, stream>>>(p, groups, first);
        else
            mxfp4_dequantize_kernel<kF32><<<grid, kNT, 0, stream>>>(p, groups, first);
    });
}

}  // namespace dps
