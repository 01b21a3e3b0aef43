// Quantisation to 8-bit floating point (e4m3) with a power-of-two scale per
// block of 32 values, and its inverse.
//
//   e = the smallest with max|x| <= 448 * 2^e, at least -127;  code = e4m3(x 2^-e)
//
// rounded to nearest even. The multiplication by 2^-e is exact, so the codes
// depend on nothing but x. The largest finite values round to 256 * 2^120 = 2^128,
// which expanded is infinite. A product sums along the blocks, so a matrix whose
// transpose enters another product (the backward pass) is needed in both
// orientations; one launch reads it once and writes either or both.
#include "mxfp8_device.h"

namespace dps {
namespace {

constexpr int kTile = 128;      // rows and columns of a workgroup's tile: 128-byte runs of codes both ways
constexpr int kNT = 256;

template <int DT> constexpr int kWords = DT == kBF16 ? 4 : 8;   // dwords per 8 elements

// 8 consecutive elements of a row from column c, zero past the matrix
template <int DT>
__device__ __forceinline__ void load8(const MxQuantParams &p, long long r, long long c, unsigned (&w)[kWords<DT>])
{
    constexpr int ES = DT == kBF16 ? 2 : 4;
    const char *at = p.src + (r * p.ld + c) * ES;
    if (r < p.rows && c + 8 <= p.cols) {
#pragma unroll
        for (int h = 0; h < kWords<DT> / 4; ++h) {
            const mx_u32x4 v = __builtin_nontemporal_load(reinterpret_cast<const mx_u32x4_e *>(at + 16 * h));
#pragma unroll
            for (int i = 0; i < 4; ++i) w[4 * h + i] = v[i];
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < kWords<DT>; ++i) w[i] = 0;
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
__device__ __forceinline__ mx_u32x2 row_codes(const unsigned (&w)[kWords<DT>], unsigned &byte)
{
    unsigned top = 0;
#pragma unroll
    for (int i = 0; i < kWords<DT>; ++i) top = DT == kF32 ? mx_max_f32(top, w[i]) : mx_max_bf16x2(top, w[i]);
    if constexpr (DT == kBF16) top = max(top << 16, top & 0xffff0000u);
    byte = mx8_scale_byte(mx_max_quad(top));
    return byte == 255u ? mx_u32x2{0u, 0u} : mx8_pack8(w, mx_scale(byte));
}

// Along the rows alone: a workgroup takes 16 rows by 512 columns, one tile of
// scales, a wave 4 of the rows. The tile's 256 scale bytes are put in order in LDS
// and leave in one store.
template <int DT>
__global__ __launch_bounds__(kNT) void mxfp8_quantize_rows_kernel(const MxQuantParams p, int tiles)
{
    __shared__ __attribute__((aligned(16))) unsigned char lds[256];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int group = blockIdx.x / tiles, kt = blockIdx.x - group * tiles;
    const long long pitch = mx8_pitch(p.cols), col = kt * 512LL + lane * 8;
    unsigned w[4][kWords<DT>];
#pragma unroll
    for (int r = 0; r < 4; ++r) load8<DT>(p, group * 16LL + wave * 4 + r, col, w[r]);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const long long row = group * 16LL + wave * 4 + r;
        unsigned byte;
        const mx_u32x2 code = row_codes<DT>(w[r], byte);
        if (row < p.rows && col < pitch) *reinterpret_cast<mx_u32x2 *>(p.codes + row * pitch + col) = code;
        if ((lane & 3) == 0) lds[mx_scale_at(wave * 4 + r, lane >> 2, 1)] = (unsigned char)byte;
    }
    __syncthreads();
    if (wave == 0)
        reinterpret_cast<unsigned *>(p.scales + blockIdx.x * 256LL)[lane] = reinterpret_cast<const unsigned *>(lds)[lane];
}

// Along the columns, and along the rows too with ROW: a workgroup reads a tile of
// 128 x 128, quantises its rows from registers, and its columns from LDS, a
// thread 32 rows of two neighbouring columns. Bound by HBM: 8192 x 14336 bf16 both ways 85.8 us, the 489 MB
// that it reads and writes at 5.7 TB/s; 4096 x 4096 15.0, the transpose alone 11.9.
template <int DT, bool ROW>
__global__ __launch_bounds__(kNT) void mxfp8_quantize_cols_kernel(const MxQuantParams p, int tiles_c)
{
    constexpr int W = kWords<DT>, PITCH = kTile * W / 8;     // dwords per row of the tile
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
    const long long pitch = mx8_pitch(p.cols), st = mx_scale_tiles(p.cols);
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
            const mx_u32x2 code = row_codes<DT>(w[q], byte);
            if (r < p.rows) {
                *reinterpret_cast<mx_u32x2 *>(p.codes + r * pitch + tc * 128 + c8 * 8) = code;
                if ((tid & 3) == 0) p.scales[mx_scale_at(r, tc * 4 + (c8 >> 2), st)] = (unsigned char)byte;
            }
        }
    }
    __syncthreads();
    const int rb = tid & 3, cp = tid >> 2;           // block of 32 rows, pair of columns
    const long long pitch_t = mx8_pitch(p.rows), st_t = mx_scale_tiles(p.rows);
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
        const unsigned byte = mx8_scale_byte(top[h]);
        const float scale = mx_scale(byte);
        mx_u32x4 code[2];
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
            const mx_u32x2 v = byte == 255u ? mx_u32x2{0u, 0u} : mx8_pack8(y, scale);
            code[o >> 1][2 * (o & 1)] = v[0];
            code[o >> 1][2 * (o & 1) + 1] = v[1];
        }
        const long long c = col0 + cp * 2 + h;
        if (c < p.cols) {
            mx_u32x4 *to = reinterpret_cast<mx_u32x4 *>(p.codes_t + c * pitch_t + tr * 128LL + rb * 32);
            to[0] = code[0];
            to[1] = code[1];
            p.scales_t[mx_scale_at(c, tr * 4 + rb, st_t)] = (unsigned char)byte;
        }
    }
}

// One thread expands 8 codes, fewer at a row's end. 8192 x 14336 to bf16 69 us, 5.2 TB/s; 8192 x 4096 17.4.
template <int DT>
__global__ __launch_bounds__(kNT) void mxfp8_dequantize_kernel(const MxExpandParams p, long long groups, unsigned first)
{
    const long long id = ((long long)first + blockIdx.x) * kNT + threadIdx.x;
    const long long r = id / groups, g = id - r * groups;
    if (r >= p.rows) return;
    const mx_u32x2 w = *reinterpret_cast<const mx_u32x2 *>(p.codes + r * mx8_pitch(p.cols) + g * 8);
    const unsigned byte = p.scales[mx_scale_at(r, (int)(g >> 2), mx_scale_tiles(p.cols))];
    const float scale = byte == 255u ? __uint_as_float(0x7fc00000u) : mx_scale(byte);
    float x[8];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[h], false), hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[h], true);
        x[4 * h] = lo[0] * scale;
        x[4 * h + 1] = lo[1] * scale;
        x[4 * h + 2] = hi[0] * scale;
        x[4 * h + 3] = hi[1] * scale;
    }
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
        mxfp8_quantize_rows_kernel<DT><<<(unsigned)((p.rows + 15) / 16 * tiles), kNT, 0, stream>>>(p, (int)tiles);
        return hipGetLastError();
    }
    const long long tr = (p.rows + kTile - 1) / kTile, tc = (p.cols + kTile - 1) / kTile;
    if (p.codes)
        mxfp8_quantize_cols_kernel<DT, true><<<(unsigned)(tr * tc), kNT, 0, stream>>>(p, (int)tc);
    else
        mxfp8_quantize_cols_kernel<DT, false><<<(unsigned)(tr * tc), kNT, 0, stream>>>(p, (int)tc);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_mxfp8_quantize(const MxQuantParams &p, int dt, hipStream_t stream)
{
    return dt == kBF16 ? quantize_typed<kBF16>(p, stream) : quantize_typed<kF32>(p, stream);
}

hipError_t launch_mxfp8_dequantize(const MxExpandParams &p, int dt, hipStream_t stream)
{
    const long long groups = (p.cols + 7) / 8;
    return launch_groups256((p.rows * groups + kNT - 1) / kNT, [&](unsigned first, unsigned grid) {
        if (dt == kBF16)
            mxfp8_dequantize_kernel<kBF16><<<grid, kNT, 0, stream>>>(p, groups, first);
        else
            mxfp8_dequantize_kernel<kF32><<<grid, kNT, 0, stream>>>(p, groups, first);
    });
}

}  // namespace dps
