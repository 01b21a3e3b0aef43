// Product of a few rows of plain values with a 4-bit block-scaled matrix,
// C[M, N] = x[M, K] . B[N, K]^T, M <= 64, without rounding x.
//
// On v_mfma_f32_16x16x32_bf16, which multiplies 16 x 32 by 32 x 16 into fp32
// sums: lane l = 16 g + i holds 8 values of row i of each operand, and which eight of K
// they are is free as long as both hold the same. A lane takes a whole block, 32 codes
// of a row of B, and expands them eight at a time: e2m1 times the block's power of two is
// exact in bf16. x in bf16 enters as it is. x in fp32 is the sum of three
// bf16 values (its 24 bits cut into 8, 8 and 8), and takes three
// instructions; exactly so from 2^-110 on, below which the last of its bits are under
// bf16's smallest, 2^-133, and lost.
#include <algorithm>
#include <type_traits>

#include "mx_gemm_device.h"
#include "mxfp8_internal.h"

namespace dps {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// 8 codes times 2^e
__device__ __forceinline__ bf16x8 expand8(unsigned w, float scale)
{
    u32x4 v;
    v[0] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0));
    v[1] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1));
    v[2] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2));
    v[3] = __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3));
    return __builtin_bit_cast(bf16x8, v);
}

// 8 values of x of a row, from `at` on, the first n of them (zero past them), as bf16 addends: one, or three of fp32, cut into
// the upper 16 bits, the upper 16 of what these leave, and the upper 16 of the rest (all of it, from 2^-110 on). An
// infinity leaves NaN; SAFE: nothing of an infinity or a NaN is left, and a NaN keeps a bit among its upper 16.
template <int XT> constexpr int kPlanes = XT == kF32 ? 3 : 1;
template <int XT> struct Values { u32x4 v[XT == kF32 ? 2 : 1]; };

template <int XT>
__device__ __forceinline__ Values<XT> load_x(const char *at, int n)
{
    Values<XT> x;
    if (n >= 8) {
        x.v[0] = reinterpret_cast<const mx_u32x4_e *>(at)[0];
        if constexpr (XT == kF32) x.v[1] = reinterpret_cast<const mx_u32x4_e *>(at)[1];
        return x;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if constexpr (XT == kF32) {
            x.v[i >> 2][i & 3] = i < n ? reinterpret_cast<const unsigned *>(at)[i] : 0u;
        } else {
            const unsigned h = i < n ? (unsigned)reinterpret_cast<const unsigned short *>(at)[i] << (16 * (i & 1)) : 0u;
            x.v[0][i >> 1] = i & 1 ? x.v[0][i >> 1] | h : h;
        }
    }
    return x;
}
template <int XT, bool SAFE>
__device__ __forceinline__ void split_x(const Values<XT> &x, u32x4 (&to)[kPlanes<XT>])
{
    if constexpr (XT == kBF16) {
        to[0] = x.v[0];
    } else {
        unsigned y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            y[i] = x.v[i >> 2][i & 3];
            if (SAFE) y[i] |= (y[i] & 0x7fffffffu) > 0x7f800000u ? 0x00400000u : 0u;
        }
#pragma unroll
        for (int part = 0; part < 3; ++part) {
#pragma unroll
            for (int i = 0; i < 4; ++i) to[part][i] = __builtin_amdgcn_perm(y[2 * i + 1], y[2 * i], 0x07060302u);
            if (part < 2) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const unsigned left = __float_as_uint(__uint_as_float(y[i]) - __uint_as_float(y[i] & 0xffff0000u));
                    y[i] = SAFE && (y[i] & 0x7f800000u) == 0x7f800000u ? 0u : left;
                }
            }
        }
    }
}

// c += w x over 8 values of K a lane
template <int XT>
__device__ __forceinline__ f32x4 product8(bf16x8 w, const u32x4 (&x)[kPlanes<XT>], f32x4 c)
{
#pragma unroll
    for (int a = 0; a < kPlanes<XT>; ++a) c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, __builtin_bit_cast(bf16x8, x[a]), c, 0, 0, 0);
    return c;
}
// the 8 codes' scale; a block that is NaN as a whole: the conversion takes the scale's NaN
__device__ __forceinline__ float scale_of(unsigned byte)
{
    return byte == 255u ? __uint_as_float(0x7fc00000u) : mx_scale(byte);
}

constexpr int kWaves = 8;
constexpr int kLine = 1024 + 16;     // bytes of a row of a plane of x in LDS: rows side by side hit distinct banks
// the waves' sums of a workgroup's blocks, added in the waves' order, to C
template <int BLOCKS, int CT, typename F>
__device__ __forceinline__ void join(const MxGemmParams &p, f32x4 *sums, const f32x4 (&acc)[BLOCKS], int wave, F place)
{
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int b = 0; b < BLOCKS; ++b) sums[(wave * BLOCKS + b) * 64 + lane] = acc[b];
    __syncthreads();
    for (int b = wave; b < BLOCKS; b += kWaves) {
        f32x4 sum = sums[b * 64 + lane];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) sum += sums[(w * BLOCKS + b) * 64 + lane];
        place(b, sum);
    }
}

// Very few rows: a workgroup computes them by 16 columns; its 8 waves take 512-wide pieces of K in
// turn. A wave brings its piece of x into an LDS part of its own, row by row in whole
// lines (as an operand of 16 rows it would be read 16 / M times over), and takes its operands from there. Bound by
// the weight's way from HBM and by a launch: 1 x 14336 x 4096 7.7 us, its 31 MB at 4.1 TB/s.
template <int CT, int XT>
__global__ __launch_bounds__(64 * kWaves) void mxfp4_matvec_kernel(const MxGemmParams p)
{
    constexpr int ES = XT == kBF16 ? 2 : 4, PL = kPlanes<XT>;
    extern __shared__ __attribute__((aligned(16))) unsigned char lds[];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int i = lane & 15, g = lane >> 4, rows = (int)p.m;
    const long long n0 = blockIdx.x * 16LL, tiles = mx_scale_tiles(p.k);
    const int steps = (int)((p.k + 127) / 128);
    const unsigned char *brow = p.b + min(n0 + i, p.n - 1) * mx_pitch(p.k) + g * 16;
    const unsigned char *srow = p.b_scales + (n0 >> 4) * tiles * 256 + lane * 4;
    unsigned char *mine = lds + wave * (PL * rows * kLine);
    // rows past the last are the last one: they are not stored
    const unsigned char *xrow = mine + min(i, rows - 1) * kLine + g * 64;
    f32x4 acc[1];
    auto all = [&](auto safe) __attribute__((always_inline)) {
        acc[0] = f32x4{};
        for (int kt = wave; kt < (int)tiles; kt += kWaves) {
            const int here = min(4, steps - kt * 4), col = kt * 512 + lane * 8;
            u32x4 codes[4];
            const unsigned bytes = *reinterpret_cast<const unsigned *>(srow + kt * 256);
#pragma unroll
            for (int t = 0; t < 4; ++t)
                if (t < here) codes[t] = *reinterpret_cast<const u32x4 *>(brow + kt * 256LL + t * 64);
            const int n = (int)min(8LL, p.k - col);
            for (int r0 = 0; r0 < rows; r0 += 4) {
                Values<XT> x[4];
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (r0 + r < rows) x[r] = load_x<XT>(p.x + ((r0 + r) * p.ldx + col) * ES, n);
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (r0 + r < rows) {
                        u32x4 v[PL];
                        split_x<XT, decltype(safe)::value>(x[r], v);
#pragma unroll
                        for (int a = 0; a < PL; ++a)
                            *reinterpret_cast<u32x4 *>(mine + (a * rows + r0 + r) * kLine + lane * 16) = v[a];
                    }
            }
            // the wave's own LDS operations are in order; nothing else touches its part
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                if (s >= here) continue;
                const float scale = scale_of(bytes >> (8 * s) & 255u);
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    u32x4 v[PL];
#pragma unroll
                    for (int a = 0; a < PL; ++a) v[a] = *reinterpret_cast<const u32x4 *>(xrow + a * rows * kLine + s * 256 + t * 16);
                    acc[0] = product8<XT>(expand8(codes[s][t], scale), v, acc[0]);
                }
            }
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        }
    };
    all(std::false_type{});
    if constexpr (XT == kF32) {
        // of an infinity NaN is left, so what has come out as NaN is computed again
        bool nan = false;
#pragma unroll
        for (int r = 0; r < 4; ++r) nan |= acc[0][r] != acc[0][r];
        if (__ballot(nan)) all(std::true_type{});
    }
    __syncthreads();
    join<1, CT>(p, reinterpret_cast<f32x4 *>(lds), acc, wave, [&](int, f32x4 sum) { store_c<CT>(p, i, n0 + 4 * g, sum); });
}

// More rows: a workgroup computes 16 MB rows by 16 NB columns; its 8 waves take 128-wide steps of K in turn,
// operands straight from global memory.
template <int MB, int NB, int CT, int XT>
__global__ __launch_bounds__(64 * kWaves) void mxfp4_rows_kernel(const MxGemmParams p, unsigned blocks_n)
{
    constexpr int ES = XT == kBF16 ? 2 : 4;
    __shared__ f32x4 sums[kWaves * MB * NB * 64];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int i = lane & 15, g = lane >> 4;
    const unsigned bm = blockIdx.x / blocks_n;
    const long long n0 = (blockIdx.x - bm * blocks_n) * (16LL * NB), m0 = bm * (16LL * MB);
    const long long tiles = mx_scale_tiles(p.k), last = p.n - 1;
    const int steps = (int)((p.k + 127) / 128);
    const unsigned char *brow[NB], *srow[NB];
#pragma unroll
    for (int c = 0; c < NB; ++c) {
        brow[c] = p.b + min(n0 + c * 16 + i, last) * mx_pitch(p.k) + g * 16;
        srow[c] = p.b_scales + (min(n0 + c * 16, last) >> 4) * tiles * 256 + lane * 4;
    }
    // rows past the last are the last one: they are not stored
    const char *xrow[MB];
#pragma unroll
    for (int b = 0; b < MB; ++b) xrow[b] = p.x + (min(m0 + b * 16 + i, p.m - 1) * p.ldx + g * 32) * ES;
    f32x4 acc[MB * NB];
    auto all = [&](auto safe) __attribute__((always_inline)) {
#pragma unroll
        for (int b = 0; b < MB * NB; ++b) acc[b] = f32x4{};
        for (int s = wave; s < steps; s += kWaves) {
            u32x4 codes[NB];
            float scale[NB];
#pragma unroll
            for (int c = 0; c < NB; ++c) {
                codes[c] = *reinterpret_cast<const u32x4 *>(brow[c] + s * 64LL);
                scale[c] = scale_of(srow[c][(s >> 2) * 256 + (s & 3)]);
            }
            const bool whole = (s + 1) * 128LL <= p.k;
            // of 64 fp32 rows by 64 columns half a step's x at once: all of it does not fit the registers
            constexpr int TC = XT == kF32 && MB * NB == 16 ? 2 : 4;
#pragma unroll
            for (int t0 = 0; t0 < 4; t0 += TC) {
                Values<XT> x[TC][MB];
#pragma unroll
                for (int b = 0; b < MB; ++b)
#pragma unroll
                    for (int t = 0; t < TC; ++t) {
                        const long long col = s * 128LL + (t0 + t) * 8;
                        x[t][b] = load_x<XT>(xrow[b] + col * ES, whole ? 8 : (int)min(8LL, max(0LL, p.k - col - g * 32)));
                    }
#pragma unroll
                for (int t = 0; t < TC; ++t) {
                    bf16x8 w[NB];
#pragma unroll
                    for (int c = 0; c < NB; ++c) w[c] = expand8(codes[c][t0 + t], scale[c]);
#pragma unroll
                    for (int b = 0; b < MB; ++b) {
                        u32x4 v[kPlanes<XT>];
                        split_x<XT, decltype(safe)::value>(x[t][b], v);
#pragma unroll
                        for (int c = 0; c < NB; ++c) acc[b * NB + c] = product8<XT>(w[c], v, acc[b * NB + c]);
                    }
                }
                if (TC < 4) MX_FENCE();
            }
        }
    };
    all(std::false_type{});
    if constexpr (XT == kF32) {
        bool nan = false;
#pragma unroll
        for (int b = 0; b < MB * NB; ++b)
#pragma unroll
            for (int r = 0; r < 4; ++r) nan |= acc[b][r] != acc[b][r];
        if (__ballot(nan)) all(std::true_type{});
    }
    join<MB * NB, CT>(p, sums, acc, wave, [&](int b, f32x4 sum) { store_c<CT>(p, m0 + b / NB * 16 + i, n0 + b % NB * 16 + 4 * g, sum); });
}

template <int MB, int NB, int CT, int XT>
hipError_t launch_rows(const MxGemmParams &p, hipStream_t stream)
{
    const unsigned blocks_n = (unsigned)((p.n + 16 * NB - 1) / (16 * NB)), blocks_m = (unsigned)((p.m + 16 * MB - 1) / (16 * MB));
    mxfp4_rows_kernel<MB, NB, CT, XT><<<blocks_n * blocks_m, 64 * kWaves, 0, stream>>>(p, blocks_n);
    return hipGetLastError();
}
// Which of the two, by the rows of x that a wave brings to LDS. Measured, us through LDS and straight (bf16): 1 x
// 14336 x 4096 8.7 and 12.5, 4 x 8192 x 4096 7.2 and 8.2, 8 x 4096 x 4096 5.3 and 6.3, 8 x 14336 x 4096 12.8 and
// 10.8; fp32, three planes a row: 2 x 8192 x 4096 8.1 and 9.9, 4 x 8192 x 4096 11.8 and 10.1. K up to 512 is one piece,
// for one wave of the eight: 3 x 1000 x 500 3.6 and 3.1.
template <int CT, int XT>
hipError_t launch_typed(const MxGemmParams &p, hipStream_t stream)
{
    const long long lines = kPlanes<XT> * p.m;
    if (p.k > 512 && lines <= (p.n <= 32 * 256 ? 8 : 6)) {
        const size_t lds = std::max<size_t>((size_t)kWaves * lines * kLine, kWaves * 1024);
        mxfp4_matvec_kernel<CT, XT><<<(unsigned)((p.n + 15) / 16), 64 * kWaves, lds, stream>>>(p);
        return hipGetLastError();
    }
    // Otherwise as few rows and columns a workgroup as leave no more workgroups than CUs: what a CU reads of x costs most.
    // Measured, us for 16 x 16 outputs a workgroup, 16 x 32, 16 x 64, 32 x 64, 64 x 64 (bf16): 64 x 1000 x 2000 5.2, 5.3, 6.7,
    // 9.3, 14.3; 20 x 4096 x 4096 10.4, 8.6, 11.1, 13.5, 16.4; 64 x 4096 x 4096 21.3, 14.3, 11.0, 15.2, 24.0; 64 x 8192 x 4096 40.5,
    // 26.6, 19.6, 16.1, 24.8; 64 x 14336 x 4096 69.4, 44.8, 35.2, 29.5, 25.4.
    auto fits = [&](int mb, int nb) { return (p.m + 16 * mb - 1) / (16 * mb) * ((p.n + 16 * nb - 1) / (16 * nb)) <= 256; };
    if (fits(1, 1)) return launch_rows<1, 1, CT, XT>(p, stream);
    if (fits(1, 2)) return launch_rows<1, 2, CT, XT>(p, stream);
    if (fits(1, 4) || p.m <= 16) return launch_rows<1, 4, CT, XT>(p, stream);
    if (fits(2, 4) || p.m <= 32) return launch_rows<2, 4, CT, XT>(p, stream);
    return p.m <= 48 ? launch_rows<3, 4, CT, XT>(p, stream) : launch_rows<4, 4, CT, XT>(p, stream);
}

}  // namespace

hipError_t launch_mxfp4_matvec(const MxGemmParams &p, int c_dt, int x_dt, hipStream_t stream)
{
    if (c_dt == kF32) return x_dt == kF32 ? launch_typed<kF32, kF32>(p, stream) : launch_typed<kF32, kBF16>(p, stream);
    return x_dt == kF32 ? launch_typed<kBF16, kF32>(p, stream) : launch_typed<kBF16, kBF16>(p, stream);
}

}  // namespace dps
