// What the block-scaled products share: the stores of C, the order of its tiles, and
// the waits of the tiled kernels.
#pragma once

#include "mxfp4_device.h"

namespace dps {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));

#define MX_FENCE() __builtin_amdgcn_sched_barrier(0)

// 4 consecutive outputs of a row, fewer at its end; added to what is there with p.accumulate (fp32)
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
            for (int i = 0; i < 3; ++i)
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
            for (int i = 0; i < 3; ++i)
                if (i < n) c[i] = (unsigned short)(w[i >> 1] >> (16 * (i & 1)));
        }
    }
}

// Workgroup id -> tile of C: ids go round-robin to the 8 XCDs, so each XCD is
// handed a contiguous range of tiles, 4 tile rows at a time, and its L2 holds
// the rows of A and B that its workgroups share (2, 8 or 16 rows: within 2%).
__device__ __forceinline__ void tile_of(int id, int tiles_m, int tiles_n, int &tm, int &tn)
{
    const int total = tiles_m * tiles_n;
    constexpr int XCDS = 8, GROUP = 4;
    if (total % XCDS == 0) id = (id % XCDS) * (total / XCDS) + id / XCDS;
    const int g = id / (GROUP * tiles_n), first = g * GROUP;
    const int rows = min(GROUP, tiles_m - first), in = id - g * GROUP * tiles_n;
    tm = first + in % rows;
    tn = in / rows;
}

typedef __attribute__((address_space(3))) void lds_void;

// until at most NEWER loads of this wave are on their way and, with READS, none of its LDS reads
template <int NEWER, bool READS>
__device__ __forceinline__ void mx_wait()
{
    __builtin_amdgcn_s_waitcnt((NEWER & 15) | 0x70 | (READS ? 0 : 0xF00) | (NEWER >> 4 << 14));
}
// names a value as one in a vector register at this point
__device__ __forceinline__ void mx_pin(unsigned &x)
{
    asm volatile("" : "+v"(x));
}
// 32 wait states: longer than the instruction takes until its sums may be read (the compiler leaves 8 behind one with
// operands in 4 bits, 12 with one in 8) and than a vector instruction's result takes to reach it
__device__ __forceinline__ void mx_settle() { asm volatile("s_nop 15\n\ts_nop 15" ::: "memory"); }


// A wave's WB x WB blocks of C, the first at (m0, n0): lane l = 16 g + i holds columns 4 g .. 4 g + 3 of row
// i of each block. VEC: rows of C on 16 bytes, bf16.
template <int WB, int CT, bool VEC>
__device__ __forceinline__ void put_tile(const MxGemmParams &p, f32x4 (&acc)[WB][WB], long long m0, long long n0)
{
    const int i = threadIdx.x & 15, g = (threadIdx.x & 63) >> 4;
    const long long row = m0 + i;
    if constexpr (VEC) {
        // pairs of blocks trade halves between lane rows g and g ^ 1, so that a lane holds 8
        // consecutive columns: one 16-byte store (nontemporal: 1% slower at k 4096, 10% at k 1024)
        typedef unsigned short u16;
        const long long c8 = n0 + 16 * (g & 1) + 8 * (g >> 1);
        u16 *c = reinterpret_cast<u16 *>(p.c) + row * p.n + c8;
#pragma unroll
        for (int a = 0; a < WB; ++a)
#pragma unroll
            for (int b = 0; b < WB; b += 2) {
                const f32x4 x = acc[a][b], y = acc[a][b + 1];
                const mx_f32x2 x0 = {x[0], x[1]}, x1 = {x[2], x[3]}, y0 = {y[0], y[1]}, y1 = {y[2], y[3]};
                const auto s0 = __builtin_amdgcn_permlane16_swap(
                    __builtin_bit_cast(unsigned, __builtin_convertvector(x0, mx_bf16x2)),
                    __builtin_bit_cast(unsigned, __builtin_convertvector(y0, mx_bf16x2)), false, false);
                const auto s1 = __builtin_amdgcn_permlane16_swap(
                    __builtin_bit_cast(unsigned, __builtin_convertvector(x1, mx_bf16x2)),
                    __builtin_bit_cast(unsigned, __builtin_convertvector(y1, mx_bf16x2)), false, false);
                const u32x4 v = {s0[0], s1[0], s0[1], s1[1]};
                if (row + a * 16 < p.m && c8 + b * 16 < p.n)
                    *reinterpret_cast<u32x4 *>(c + (long long)a * 16 * p.n + b * 16) = v;
            }
    } else {
#pragma unroll
        for (int a = 0; a < WB; ++a) {
#pragma unroll
            for (int b = 0; b < WB; ++b) store_c<CT>(p, row + a * 16, n0 + b * 16 + 4 * g, acc[a][b]);
            MX_FENCE();
        }
    }
}

}  // namespace
}  // namespace dps
