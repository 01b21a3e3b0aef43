// Product of 4-bit block-scaled matrices, C[M, N] = A[M, K] . B[N, K]^T with
// both operands quantised along K, on gfx950's scaled matrix instruction
// v_mfma_scale_f32_16x16x128_f8f6f4: it multiplies 16 x 128 by 128 x 16 e2m1
// values, each block of 32 along K times 2^(its row's A scale + its column's B
// scale), into fp32 sums.
//
// Operand layout (lane l = 16 g + i): the lane holds the 32 codes (16 bytes) of
// row i, block g of the step's four, and its scale operand's byte `opsel` is
// that block's scale. D register r of lane l: D[4 (l / 16) + r][l % 16]. The
// instruction gets B's rows first, so that a lane ends with 4 consecutive
// columns of one row of C.
#include "mxfp4_device.h"

namespace dps {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));

template <int T>
__device__ __forceinline__ f32x4 mfma(u32x4 first, unsigned fs, u32x4 second, unsigned ss, f32x4 c)
{
    const i32x8 a = {(int)first[0], (int)first[1], (int)first[2], (int)first[3], 0, 0, 0, 0};
    const i32x8 b = {(int)second[0], (int)second[1], (int)second[2], (int)second[3], 0, 0, 0, 0};
    // formats 4: e2m1
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 4, 4, T, (int)fs, T, (int)ss);
}

// n (1..4) consecutive outputs of a row
template <int CT>
__device__ __forceinline__ void store_c(const MxGemmParams &p, long long row, long long col, f32x4 v)
{
    const int n = (int)min(4LL, p.n - col);
    if (row >= p.m || n <= 0) return;
    if constexpr (CT == kF32) {
        float *c = reinterpret_cast<float *>(p.c) + row * p.n + col;
        typedef float f32x4_e __attribute__((ext_vector_type(4), aligned(4)));
        if (n == 4) {
            if (p.accumulate) v += *reinterpret_cast<const f32x4_e *>(c);
            *reinterpret_cast<f32x4_e *>(c) = v;
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (i < n) c[i] = p.accumulate ? c[i] + v[i] : v[i];
        }
    } else {
        unsigned short *c = reinterpret_cast<unsigned short *>(p.c) + row * p.n + col;
        typedef unsigned int u32x2_e __attribute__((ext_vector_type(2), aligned(2)));
        const mx_f32x2 lo = {v[0], v[1]}, hi = {v[2], v[3]};
        const unsigned w[2] = {__builtin_bit_cast(unsigned, __builtin_convertvector(lo, mx_bf16x2)),
                               __builtin_bit_cast(unsigned, __builtin_convertvector(hi, mx_bf16x2))};
        if (n == 4) {
            *reinterpret_cast<u32x2_e *>(c) = u32x2_e{w[0], w[1]};
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (i < n) c[i] = (unsigned short)(w[i >> 1] >> (16 * (i & 1)));
        }
    }
}

// The 32 values of row `row`, block kb of x as codes; their scale byte in
// `byte`. The same rounding as the quantising kernel: the same bits.
template <int XT>
__device__ __forceinline__ u32x4 quantize_block(const MxGemmParams &p, long long row, long long kb, unsigned &byte)
{
    unsigned x[32];
    const long long c0 = kb * 32;
    const char *at = p.x + (row * p.ldx + c0) * (XT == kBF16 ? 2 : 4);
    if (c0 + 32 <= p.k) {
        if constexpr (XT == kBF16) {
#pragma unroll
            for (int h = 0; h < 4; ++h) {
                const u32x4 v = *reinterpret_cast<const mx_u32x4_e *>(at + 16 * h);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x[8 * h + 2 * i] = v[i] << 16;
                    x[8 * h + 2 * i + 1] = v[i] & 0xffff0000u;
                }
            }
        } else {
#pragma unroll
            for (int h = 0; h < 8; ++h) {
                const u32x4 v = *reinterpret_cast<const mx_u32x4_e *>(at + 16 * h);
#pragma unroll
                for (int i = 0; i < 4; ++i) x[4 * h + i] = v[i];
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            x[i] = 0;
            if (c0 + i < p.k)
                x[i] = XT == kBF16 ? (unsigned)reinterpret_cast<const unsigned short *>(at)[i] << 16
                                   : reinterpret_cast<const unsigned *>(at)[i];
        }
    }
    unsigned top = 0;
#pragma unroll
    for (int i = 0; i < 32; ++i) top = max(top, x[i] & 0x7fffffffu);
    byte = mx_scale_byte(top);
    const float inv = mx_inverse(byte);
    u32x4 code;
#pragma unroll
    for (int o = 0; o < 4; ++o) {
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = __uint_as_float(x[8 * o + i]) * inv;
        code[o] = byte == 255u ? 0u : mx_pack8(y);
    }
    return code;
}

// A workgroup computes 16 MB rows of C by 16 columns; its 4 waves take
// 512-wide pieces of K in turn, straight from global memory, and their sums
// meet in LDS in a fixed order.
template <int MB, int CT, int XT>
__global__ __launch_bounds__(256) void mxfp4_gemm_few_kernel(const MxGemmParams p)
{
    __shared__ f32x4 part[3][MB][64];
    const int lane = threadIdx.x & 63;
    // a scalar, so that what depends on it is skipped by a jump: the matrix
    // instructions run whatever the lane mask says
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int i = lane & 15, g = lane >> 4;
    const unsigned blocks_n = (unsigned)((p.n + 15) >> 4), bm = blockIdx.x / blocks_n;
    const long long n0 = (long long)(blockIdx.x - bm * blocks_n) * 16, m0 = (long long)bm * 16 * MB;
    const long long pitch = mx_pitch(p.k), tiles = mx_scale_tiles(p.k);
    const long long steps = (p.k + 127) / 128;
    const long long rb = min(n0 + i, p.n - 1);
    f32x4 acc[MB];
#pragma unroll
    for (int b = 0; b < MB; ++b) acc[b] = f32x4{};
    for (long long kt = wave; kt < tiles; kt += 4) {
        const int here = (int)min(4LL, steps - kt * 4);
        const unsigned bs = *reinterpret_cast<const unsigned *>(p.b_scales + ((n0 >> 4) * tiles + kt) * 256 + lane * 4);
        u32x4 bw[4], aw[MB][4];
        unsigned as[MB];
#pragma unroll
        for (int t = 0; t < 4; ++t)
            if (t < here) bw[t] = *reinterpret_cast<const u32x4 *>(p.b + rb * pitch + kt * 256 + t * 64 + g * 16);
#pragma unroll
        for (int b = 0; b < MB; ++b) {
            const long long ra = min(m0 + b * 16 + i, p.m - 1);
            if constexpr (XT < 0) {
                // a row group past the last is the last one's: its rows are not stored
                as[b] = *reinterpret_cast<const unsigned *>(p.a_scales + ((ra >> 4) * tiles + kt) * 256 + (g * 16 + (int)(ra & 15)) * 4);
#pragma unroll
                for (int t = 0; t < 4; ++t)
                    if (t < here) aw[b][t] = *reinterpret_cast<const u32x4 *>(p.a + ra * pitch + kt * 256 + t * 64 + g * 16);
            } else {
                as[b] = 0;
#pragma unroll
                for (int t = 0; t < 4; ++t)
                    if (t < here) {
                        unsigned byte = 0;
                        aw[b][t] = u32x4{};
                        const long long kb = kt * 16 + t * 4 + g;
                        if (kb * 32 < p.k) aw[b][t] = quantize_block<XT>(p, ra, kb, byte);
                        as[b] |= byte << (8 * t);
                    }
            }
        }
#pragma unroll
        for (int b = 0; b < MB; ++b) {
            acc[b] = mfma<0>(bw[0], bs, aw[b][0], as[b], acc[b]);
            if (here > 1) acc[b] = mfma<1>(bw[1], bs, aw[b][1], as[b], acc[b]);
            if (here > 2) acc[b] = mfma<2>(bw[2], bs, aw[b][2], as[b], acc[b]);
            if (here > 3) acc[b] = mfma<3>(bw[3], bs, aw[b][3], as[b], acc[b]);
        }
    }
    if (wave > 0) {
#pragma unroll
        for (int b = 0; b < MB; ++b) part[wave - 1][b][lane] = acc[b];
    }
    __syncthreads();
    if (wave > 0) return;
#pragma unroll
    for (int b = 0; b < MB; ++b) {
#pragma unroll
        for (int w = 0; w < 3; ++w) acc[b] += part[w][b][lane];
        store_c<CT>(p, m0 + b * 16 + i, n0 + 4 * g, acc[b]);
    }
}

template <int MB, int CT>
hipError_t launch_few(const MxGemmParams &p, int x_dt, hipStream_t stream)
{
    const unsigned grid = (unsigned)((p.n + 15) / 16 * ((p.m + 16 * MB - 1) / (16 * MB)));
    if constexpr (MB == 1) {
        if (x_dt == kBF16) {
            mxfp4_gemm_few_kernel<1, CT, kBF16><<<grid, 256, 0, stream>>>(p);
            return hipGetLastError();
        }
        if (x_dt == kF32) {
            mxfp4_gemm_few_kernel<1, CT, kF32><<<grid, 256, 0, stream>>>(p);
            return hipGetLastError();
        }
    }
    mxfp4_gemm_few_kernel<MB, CT, -1><<<grid, 256, 0, stream>>>(p);
    return hipGetLastError();
}

template <int CT>
hipError_t launch_typed(const MxGemmParams &p, int x_dt, hipStream_t stream)
{
    return p.m <= 16 ? launch_few<1, CT>(p, x_dt, stream) : launch_few<4, CT>(p, x_dt, stream);
}

}  // namespace

hipError_t launch_mxfp4_gemm(const MxGemmParams &p, int c_dt, int x_dt, hipStream_t stream)
{
    return c_dt == kF32 ? launch_typed<kF32>(p, x_dt, stream) : launch_typed<kBF16>(p, x_dt, stream);
}

}  // namespace dps
