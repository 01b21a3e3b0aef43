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
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "mxfp4_device.h"

namespace dps {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));

#define MX_FENCE() __builtin_amdgcn_sched_barrier(0)

template <int T>
__device__ __forceinline__ f32x4 mfma(u32x4 first, unsigned fs, u32x4 second, unsigned ss, f32x4 c)
{
    const i32x8 a = {(int)first[0], (int)first[1], (int)first[2], (int)first[3], 0, 0, 0, 0};
    const i32x8 b = {(int)second[0], (int)second[1], (int)second[2], (int)second[3], 0, 0, 0, 0};
    // formats 4: e2m1
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 4, 4, T, (int)fs, T, (int)ss);
}

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

// The 32 values of row `row`, block kb of x as codes; their scale byte in
// `byte`. The same rounding as the quantising kernel: the same bits.
template <int XT>
__device__ __forceinline__ u32x4 quantize_block(const MxGemmParams &p, long long row, long long kb, unsigned &byte)
{
    constexpr int W = XT == kBF16 ? 4 : 8;           // dwords per 8 values
    unsigned x[4][W], top = 0;
    const long long c0 = kb * 32;
    const char *at = p.x + (row * p.ldx + c0) * (XT == kBF16 ? 2 : 4);
    if (c0 + 32 <= p.k) {
#pragma unroll
        for (int h = 0; h < W; ++h) {
            const u32x4 v = *reinterpret_cast<const mx_u32x4_e *>(at + 16 * h);
#pragma unroll
            for (int i = 0; i < 4; ++i) x[h * 4 / W][h * 4 % W + i] = v[i];
        }
    } else {
        // the row's last, short block, 8 values at a time and twice over, so
        // that this rare case costs the others no registers; 8 loads are issued
        // together, from the row's last value where there is none
        const int n = (int)(p.k - c0);
        auto values = [&](int o, unsigned (&y)[8]) __attribute__((always_inline)) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int j = min(8 * o + i, n - 1);
                const unsigned v = XT == kBF16 ? (unsigned)reinterpret_cast<const unsigned short *>(at)[j] << 16
                                               : reinterpret_cast<const unsigned *>(at)[j];
                y[i] = 8 * o + i < n ? v : 0u;
            }
        };
        unsigned y[8];
#pragma unroll 1
        for (int o = 0; 8 * o < n; ++o) {
            values(o, y);
#pragma unroll
            for (int i = 0; i < 8; ++i) top = mx_max_f32(top, y[i]);
        }
        byte = mx_scale_byte(top);
        u32x4 code = {};
#pragma unroll 1
        for (int o = 0; 8 * o < n && byte != 255u; ++o) {
            values(o, y);
            const unsigned w = mx_pack8(y, mx_scale(byte));
#pragma unroll
            for (int i = 0; i < 4; ++i) code[i] = i == o ? w : code[i];
        }
        return code;
    }
#pragma unroll
    for (int i = 0; i < 4 * W; ++i)
        top = XT == kBF16 ? mx_max_bf16x2(top, x[i / W][i % W]) : mx_max_f32(top, x[i / W][i % W]);
    if constexpr (XT == kBF16) top = max(top << 16, top & 0xffff0000u);
    byte = mx_scale_byte(top);
    const float scale = mx_scale(byte);
    u32x4 code;
#pragma unroll
    for (int o = 0; o < 4; ++o) code[o] = byte == 255u ? 0u : mx_pack8(x[o], scale);
    return code;
}

// A workgroup computes 16 MB rows of C by 16 columns; its 4 waves take
// 512-wide pieces of K in turn, two at a time, straight from global memory, and
// their sums meet in LDS in a fixed order. B is read once, and reading it is
// what the kernel's time is made of.
//
// XT >= 0 (up to 16 rows): A comes as plain values. While its pieces of B are on
// their way, a wave quantises the blocks of A that they meet, one a lane, into
// LDS in the operand's layout: with a block's lane as owner of the
// matrix operand instead, all 16 rows' lanes would do the work of row 0 for a
// single token (1 x 14336 x 4096: 15.5 us against 7.6, 31 MB read).
constexpr int kPieces = 2;
template <int MB, int CT, int XT>
__global__ __launch_bounds__(256) void mxfp4_gemm_few_kernel(const MxGemmParams p, unsigned first)
{
    __shared__ f32x4 part[3][MB][64];
    __shared__ __attribute__((aligned(16))) unsigned char xc[XT < 0 ? 1 : 4 * kPieces * 16 * 256];
    __shared__ __attribute__((aligned(16))) unsigned char xs[XT < 0 ? 1 : 4 * kPieces * 256];
    const int lane = threadIdx.x & 63;
    // a scalar, so that what depends on it is skipped by a jump: the matrix
    // instructions run whatever the lane mask says
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int i = lane & 15, g = lane >> 4;
    const unsigned id = first + blockIdx.x, blocks_n = (unsigned)((p.n + 15) >> 4), bm = id / blocks_n;
    const long long n0 = (long long)(id - bm * blocks_n) * 16, m0 = (long long)bm * 16 * MB;
    const long long pitch = mx_pitch(p.k), tiles = mx_scale_tiles(p.k);
    const int steps = (int)((p.k + 127) / 128);
    const long long rb = min(n0 + i, p.n - 1);
    f32x4 acc[MB];
#pragma unroll
    for (int b = 0; b < MB; ++b) acc[b] = f32x4{};
    for (int kt0 = wave * kPieces; kt0 < (int)tiles; kt0 += 4 * kPieces) {
        u32x4 bw[kPieces][4];
        unsigned bs[kPieces];
#pragma unroll
        for (int h = 0; h < kPieces; ++h) {
            const int kt = kt0 + h, here = min(4, steps - kt * 4);
            if (here <= 0) continue;
            bs[h] = *reinterpret_cast<const unsigned *>(p.b_scales + ((n0 >> 4) * tiles + kt) * 256 + lane * 4);
#pragma unroll
            for (int t = 0; t < 4; ++t)
                if (t < here) bw[h][t] = *reinterpret_cast<const u32x4 *>(p.b + rb * pitch + kt * 256 + t * 64 + g * 16);
        }
        unsigned char *codes = xc + wave * (kPieces * 4096), *bytes = xs + wave * (kPieces * 256);
        if constexpr (XT >= 0) {
            const int blocks = (int)p.m * 16 * kPieces;
            for (int at = lane; at < blocks; at += 64) {
                const int row = at / (16 * kPieces), h = at / 16 % kPieces, bk = at % 16;
                const long long kb = (kt0 + h) * 16LL + bk;
                unsigned byte = 0;
                u32x4 code = {};
                if (kb * 32 < p.k) code = quantize_block<XT>(p, row, kb, byte);
                *reinterpret_cast<u32x4 *>(codes + h * 4096 + row * 256 + bk * 16) = code;
                bytes[h * 256 + mx_scale_at(row, bk, 1)] = (unsigned char)byte;
            }
            // the wave's own LDS operations are in order; nothing else touches its part
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        }
#pragma unroll
        for (int h = 0; h < kPieces; ++h) {
            const int kt = kt0 + h, here = min(4, steps - kt * 4);
            if (here <= 0) continue;
            u32x4 aw[MB][4];
            unsigned as[MB];
#pragma unroll
            for (int b = 0; b < MB; ++b) {
                // rows past the last are the last one: they are not stored
                const long long ra = min(m0 + b * 16 + i, p.m - 1);
                const int at = (g * 16 + (int)(ra & 15)) * 4;
                if constexpr (XT < 0)
                    as[b] = *reinterpret_cast<const unsigned *>(p.a_scales + ((ra >> 4) * tiles + kt) * 256 + at);
                else
                    as[b] = *reinterpret_cast<const unsigned *>(bytes + h * 256 + at);
#pragma unroll
                for (int t = 0; t < 4; ++t)
                    if (t < here) {
                        if constexpr (XT < 0)
                            aw[b][t] = *reinterpret_cast<const u32x4 *>(p.a + ra * pitch + kt * 256 + t * 64 + g * 16);
                        else
                            aw[b][t] = *reinterpret_cast<const u32x4 *>(codes + h * 4096 + ra * 256 + t * 64 + g * 16);
                    }
            }
#pragma unroll
            for (int b = 0; b < MB; ++b) {
                acc[b] = mfma<0>(bw[h][0], bs[h], aw[b][0], as[b], acc[b]);
                if (here > 1) acc[b] = mfma<1>(bw[h][1], bs[h], aw[b][1], as[b], acc[b]);
                if (here > 2) acc[b] = mfma<2>(bw[h][2], bs[h], aw[b][2], as[b], acc[b]);
                if (here > 3) acc[b] = mfma<3>(bw[h][3], bs[h], aw[b][3], as[b], acc[b]);
            }
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
    const long long groups = (p.n + 15) / 16 * ((p.m + 16 * MB - 1) / (16 * MB));
    return launch_groups256(groups, [&](unsigned first, unsigned grid) {
        if constexpr (MB == 1) {
            if (x_dt == kBF16) return mxfp4_gemm_few_kernel<1, CT, kBF16><<<grid, 256, 0, stream>>>(p, first);
            if (x_dt == kF32) return mxfp4_gemm_few_kernel<1, CT, kF32><<<grid, 256, 0, stream>>>(p, first);
        }
        mxfp4_gemm_few_kernel<MB, CT, -1><<<grid, 256, 0, stream>>>(p, first);
    });
}

// ------------------------------------------------------------ tiled kernel

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

// The matrix instruction with its sums in the accumulation registers for good:
// left to the compiler, part of the 256 sums of the large tile sit in other
// registers and are copied around every pass of the loop. The compiler sees
// neither the instruction's latency nor its hazards, so a read of the sums and a
// write of an operand by a vector instruction are kept apart from it by
// mx_settle() below. Scale byte T of both operands.
template <int T>
__device__ __forceinline__ void mfma_acc(f32x4 &c, u32x4 first, unsigned fs, u32x4 second, unsigned ss)
{
#define MX_MFMA(sel)                                                                       \
    asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 %0, %1, %2, %0, %3, %4 " sel " cbsz:4 blgp:4" \
                 : "+a"(c) : "v"(first), "v"(second), "v"(fs), "v"(ss))
    if constexpr (T == 0)
        MX_MFMA("op_sel_hi:[0,0,0]");
    else if constexpr (T == 1)
        MX_MFMA("op_sel:[1,1,0] op_sel_hi:[0,0,0]");
    else if constexpr (T == 2)
        MX_MFMA("op_sel_hi:[1,1,0]");
    else
        MX_MFMA("op_sel:[1,1,0] op_sel_hi:[1,1,0]");
#undef MX_MFMA
}
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
// 32 cycles: longer than the instruction takes to write its sums (16) and than
// a vector instruction's result takes to reach it
__device__ __forceinline__ void mx_settle() { asm volatile("s_nop 15\n\ts_nop 15" ::: "memory"); }

// Tile of 32 WB x 32 WB, 4 waves of 16 WB x 16 WB (WB x WB instructions per
// 128-wide step of K). A stage is 256 of K, 128 bytes a row, and goes from
// global memory straight into one of two LDS buffers (buffer_load ... lds, 8
// rows an instruction): chunk c (16 bytes, one block) of row r sits at position
// c ^ (r % 8), so the 16 rows that a fragment read touches at one chunk hit
// distinct banks. Stage t is computed in two steps: step 0 while the fragments
// of step 1 are read; then step 1 while the first fragments of stage t + 1 are
// read, B's and then A's, and the loads of stage t + 2 go into the buffer just
// left, B's and then A's. Each wave waits for its loads of B of stage t + 1 and
// the workgroup meets before step 1, and the same for A half way through it:
// the later a load is issued, the later it is needed.
//
// Scales come as one 32-bit load per 16 rows and two stages (their layout is
// the operand's), loaded a pair of stages ahead and kept in registers.
//
// K is walked in pairs of stages (512). In the last pair a stage past the row's
// end is loaded from the row's last 128 bytes instead, so that no load leaves
// the operand; a half stage then stands in the second half of its buffer. Steps
// without data get scale bytes of zero on both sides: whatever codes stand there
// (each is a finite number), their products are at most 2^-254 * 36 and
// vanish against fp32's smallest 2^-149. One byte permutation with a scalar
// selector does both. Rows past M or N are loads of the last row, and their
// results are not stored.
//
// Measured: 8192^3 224-251 us on several cards (4.4-4.9 PFLOP/s), 4096^3 35-37 us, 2048
// x 4096 x 4096 22-24 (tiles of 128). Two things bound the large ones. The matrix units are
// busy 57% (8192 x 14336 x 4096) to 67% (8192^3) of the cycles: waves wait 14% of them for
// loads and each other and are held at issue in 30%, the LDS reads and loads going out between
// the matrix instructions. And the card's power sets the clock, 1.66-1.77 GHz here:
// codes of zero take 190 us, and a loop of nothing but these instructions runs at 1.68
// GHz on random codes (6.8 PFLOP/s; 6.1 in the 32x32x64 form), at 2.38 on zeros (9.7).
//
// LOOP: a workgroup of the large tile has a CU to itself, so that nothing runs
// while it starts and while it writes C. With more tiles than CUs, 256 workgroups
// go through them instead, and load a tile's first stages during the last
// ones of the tile before (8192 x 14336 x 4096: 211 us in place of 238; with one
// tile a workgroup the loop around costs 2%).
template <int WB, int CT, bool VEC, bool LOOP>
__global__ __launch_bounds__(256) void mxfp4_gemm_tile_kernel(const MxGemmParams p, int tiles_m, int tiles_n)
{
#ifdef __HIP_DEVICE_COMPILE__                        // the host pass rejects the body's operands, and needs none
    constexpr int T = 32 * WB;                       // tile side
    constexpr int BYTES = T * 128;
    __shared__ __attribute__((aligned(1024))) unsigned char A0[BYTES], A1[BYTES], B0[BYTES], B1[BYTES];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wi = wave >> 1, wj = wave & 1, i = lane & 15, g = lane >> 4;
    const int pitch = (int)mx_pitch(p.k), ktiles = (int)mx_scale_tiles(p.k);
    const int steps = (int)((p.k + 127) / 128), pairs = (steps + 3) / 4;
    // selection of the last pair's scale bytes (see above; 0x0c selects a zero byte)
    const int rest = steps % 4;
    const unsigned tail = rest == 0 ? 0x03020100u : rest == 1 ? 0x0c0c000cu : rest == 2 ? 0x0c0c0100u : 0x020c0100u;
    auto abuf = [&](int buf) __attribute__((always_inline)) { return buf ? A1 : A0; };
    auto bbuf = [&](int buf) __attribute__((always_inline)) { return buf ? B1 : B0; };

    // the tile that is being loaded: its corner in C, and offsets within its
    // rows of codes and scales, which fit 31 bits (checked by the launcher)
    long long lm0, ln0;
    const unsigned char *la, *lb, *lsa, *lsb;
    int off[2 * WB], soff[2 * WB];
    auto place = [&](int tile) __attribute__((always_inline)) {
        int tm, tn;
        tile_of(tile, tiles_m, tiles_n, tm, tn);
        lm0 = (long long)tm * T;
        ln0 = (long long)tn * T;
        const int rows_a = (int)min((long long)T, p.m - lm0), rows_b = (int)min((long long)T, p.n - ln0);
        la = p.a + lm0 * pitch;
        lb = p.b + ln0 * pitch;
        lsa = p.a_scales + lm0 / 16 * ktiles * 256;
        lsb = p.b_scales + ln0 / 16 * ktiles * 256;
#pragma unroll
        for (int q = 0; q < 2 * WB; ++q) {
            const int row = wave * 8 * WB + (q % WB) * 8 + (lane >> 3);
            off[q] = min(row, (q < WB ? rows_b : rows_a) - 1) * pitch + (((lane & 7) ^ (lane >> 3)) << 4);
        }
#pragma unroll
        for (int x = 0; x < WB; ++x) {
            soff[x] = min(wi * WB + x, (rows_a - 1) >> 4) * ktiles * 256 + lane * 4;
            soff[WB + x] = min(wj * WB + x, (rows_b - 1) >> 4) * ktiles * 256 + lane * 4;
        }
    };
    auto rsrc = [](const unsigned char *base) __attribute__((always_inline)) {
        return __builtin_amdgcn_make_buffer_rsrc((void *)base, (short)0, 0x7fffffff, 0x00020000);
    };
    // a stage that reaches past the row is taken from the row's last 128 bytes
    auto dtl = [&](int buf, int stage, int q) __attribute__((always_inline)) {
        const int row0 = wave * 8 * WB + (q % WB) * 8;
        const int so = __builtin_amdgcn_readfirstlane(min(stage * 128, pitch - 128));
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc(q < WB ? lb : la),
                                                 (lds_void *)((q < WB ? bbuf(buf) : abuf(buf)) + row0 * 128), 16, off[q], so,
                                                 0, 0);
    };
    // scales of 16-row group x of this wave's rows (x < WB: A's group x, else B's x - WB), pair of stages kt
    auto scale = [&](int x, int kt) __attribute__((always_inline)) {
        return (unsigned)__builtin_amdgcn_raw_buffer_load_b32(rsrc(x < WB ? lsa : lsb), soff[x], kt * 256, 0);
    };

    f32x4 acc[WB][WB];
    auto clear = [&]() __attribute__((always_inline)) {
#pragma unroll
        for (int a = 0; a < WB; ++a)
#pragma unroll
            for (int b = 0; b < WB; ++b) {
                acc[a][b] = f32x4{};
                asm volatile("" : "+a"(acc[a][b]));
            }
        mx_settle();
    };
    clear();
    u32x4 af[2][WB], bf[2][WB];
    unsigned sa[WB], sb[WB], ns[2 * WB];

    int tile = blockIdx.x;
    place(tile);
    long long m0 = lm0, n0 = ln0;
#pragma unroll
    for (int q = 0; q < 2 * WB; ++q) dtl(0, 0, q);
#pragma unroll
    for (int q = 0; q < 2 * WB; ++q) dtl(1, 1, q);
#pragma unroll
    for (int x = 0; x < 2 * WB; ++x) ns[x] = scale(x, 0);
    MX_FENCE();
    auto take = [&](unsigned &x, unsigned next, unsigned sel) __attribute__((always_inline)) {
        x = __builtin_amdgcn_perm(0u, next, sel);
        mx_pin(x);
    };
#pragma unroll
    for (int x = 0; x < WB; ++x) {
        take(sa[x], ns[x], pairs == 1 ? tail : 0x03020100u);
        take(sb[x], ns[WB + x], pairs == 1 ? tail : 0x03020100u);
    }
    mx_settle();
    // fragment read q of a step: q < WB B's block q, else A's block q - WB
    const int fp = i * 128, fx = lane & 7;
    auto rdq = [&](int set, int buf, int ks, int q) __attribute__((always_inline)) {
        const int x = q % WB;
        const int at = fp + (((ks * 4 + g) ^ fx) << 4);
        if (q >= WB)
            af[set][x] = *reinterpret_cast<const u32x4 *>(abuf(buf) + (wi * WB + x) * 2048 + at);
        else
            bf[set][x] = *reinterpret_cast<const u32x4 *>(bbuf(buf) + (wj * WB + x) * 2048 + at);
    };
    // instructions per step; per fragment read in step 1 (EV) and step 0 (RV); per load
    constexpr int N = WB * WB, EV = WB / 2, RV = WB == 8 ? 3 : 2, DV = WB / 2;
    // In step 1's instructions stand, in this order, a load of B every DV, then
    // those of A, and in even stages a scale load every EV. So many loads are
    // newer than the last one of B (of A) where it has to have landed:
    constexpr int kLoads = (N / 2 + DV - 1) / DV, kScales = (N / 2 + EV - 2) / EV;
    constexpr int kScalesAfterB = 2 * WB - (DV * (WB - 1) + EV - 1) / EV;
    // waits until at most that many of this wave's loads are on their way, then for
    // the other waves. Before step 1 its reads of step 1's fragments have to be
    // over too, as the next loads go where they read.
    // kStores: stores of the tile before that may be on their way besides.
    constexpr int kStores = LOOP && VEC ? N / 2 : 0;
    auto meet = [&](auto newer, auto reads, bool stores) __attribute__((always_inline)) {
        MX_FENCE();
        if (kStores && stores)
            mx_wait<decltype(newer)::value + kStores, decltype(reads)::value>();
        else
            mx_wait<decltype(newer)::value, decltype(reads)::value>();
        __builtin_amdgcn_s_barrier();
        MX_FENCE();
    };
    // stage 2 kt + buf; `next`: the stage to load two ahead, `sel`: the next pair's selection of scale bytes
    auto stage = [&](auto buf_, int next, int next_kt, unsigned sel, bool stores) __attribute__((always_inline)) {
        constexpr int buf = decltype(buf_)::value;
#pragma unroll
        for (int q = 0; q < N; ++q) {
            if (q % RV == 0 && q / RV < 2 * WB) rdq(1, buf, 1, q / RV);
            mfma_acc<2 * buf>(acc[q / WB][q % WB], bf[0][q % WB], sb[q % WB], af[0][q / WB], sa[q / WB]);
            MX_FENCE();
        }
        // B of stage t + 1 is there
        meet(std::integral_constant<int, WB + (buf == 1 ? kScalesAfterB : 0)>{}, std::true_type{}, buf == 0 && stores);
#pragma unroll
        for (int q = 0; q < N; ++q) {
            if (q == N / 2)                          // A of stage t + 1 is there
                meet(std::integral_constant<int, kLoads + (buf == 0 ? kScales : 0)>{}, std::false_type{}, buf == 0 && stores);
            if (q % EV == 0) rdq(0, buf ^ 1, 0, q / EV);
            if constexpr (buf == 0) {
                if (q % EV == 1) ns[q / EV] = scale(q / EV, next_kt);
            }
            if (q % DV == 0 && q / DV < 2 * WB) dtl(buf, next, q / DV);
            mfma_acc<2 * buf + 1>(acc[q / WB][q % WB], bf[1][q % WB], sb[q % WB], af[1][q / WB], sa[q / WB]);
            // the next pair's scales take their place as soon as this one's
            // have been used, at least WB - 1 instructions before their first use
            if constexpr (buf == 1) {
                if (q % WB == 0 && q > 0) take(sa[q / WB - 1], ns[q / WB - 1], sel);
                if (q > N - WB) take(sb[q - N + WB - 1], ns[WB + q - N + WB - 1], sel);
                if (q == N - 1) {
                    take(sa[WB - 1], ns[WB - 1], sel);
                    take(sb[WB - 1], ns[2 * WB - 1], sel);
                }
            }
            MX_FENCE();
        }
    };
    __builtin_amdgcn_s_waitcnt(0x0F70);
    __syncthreads();
#pragma unroll
    for (int q = 0; q < 2 * WB; ++q) rdq(0, 0, 0, q);
    MX_FENCE();
    // C: lane (i, g) holds columns 4 g .. 4 g + 3 of row i of each block
    auto put = [&](long long m0, long long n0) __attribute__((always_inline)) {
        const long long row = m0 + wi * 16 * WB + i, col = n0 + wj * 16 * WB;
        if constexpr (VEC) {
            // pairs of blocks trade halves between lane rows g and g ^ 1, so that a
            // lane holds 8 consecutive columns: one 16-byte store (nontemporal: 1% slower at
        // k 4096, 10% at k 1024)
            typedef unsigned short u16;
            const long long c8 = col + 16 * (g & 1) + 8 * (g >> 1);
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
                for (int b = 0; b < WB; ++b) store_c<CT>(p, row + a * 16, col + b * 16 + 4 * g, acc[a][b]);
                MX_FENCE();
            }
        }
    };
    const int tiles = tiles_m * tiles_n;
    bool stores = false;
    for (;;) {
        const int following = tile + gridDim.x;
        for (int kt = 0; kt < pairs; ++kt) {
            // the last pair loads the first pair of the workgroup's next tile, whose
            // first stage then goes on without a pause (without a next tile, this
            // one's again, to be read by no one)
            const int next = kt + 1 < pairs ? kt + 1 : 0;
            if (LOOP && next == 0 && following < tiles) place(following);
            stage(std::integral_constant<int, 0>{}, 2 * next, next, 0u, stores);
            stage(std::integral_constant<int, 1>{}, 2 * next + 1, 0, next + 1 == pairs ? tail : 0x03020100u, false);
            stores = false;
        }
        // the last loads land before the workgroup ends, and its LDS is another's
        const bool done = !LOOP || following >= tiles;
        if (done) __builtin_amdgcn_s_waitcnt(0x0F70);
        mx_settle();
#pragma unroll
        for (int a = 0; a < WB; ++a)
#pragma unroll
            for (int b = 0; b < WB; ++b) asm volatile("" : "+a"(acc[a][b]));
        put(m0, n0);
        if (done) return;
        // a whole tile's stores are counted; of one at the edge of C some are not made
        stores = m0 + T <= p.m && n0 + T <= p.n;
        tile = following;
        m0 = lm0;
        n0 = ln0;
        clear();
    }
#endif
}

template <int WB, int CT>
hipError_t launch_tile(const MxGemmParams &p, hipStream_t stream)
{
    const int T = 32 * WB;
    const int tm = (int)((p.m + T - 1) / T), tn = (int)((p.n + T - 1) / T);
    constexpr int CUS = 256;
    const bool loop = WB == 8 && tm * tn > CUS;
    const int grid = loop ? CUS : tm * tn;
    if constexpr (CT == kBF16) {
        // rows of C on 16 bytes: 16-byte stores
        if ((uintptr_t)p.c % 16 == 0 && p.n % 8 == 0) {
            if (loop)
                mxfp4_gemm_tile_kernel<WB, CT, true, WB == 8><<<grid, 256, 0, stream>>>(p, tm, tn);
            else
                mxfp4_gemm_tile_kernel<WB, CT, true, false><<<grid, 256, 0, stream>>>(p, tm, tn);
            return hipGetLastError();
        }
    }
    if (loop)
        mxfp4_gemm_tile_kernel<WB, CT, false, WB == 8><<<grid, 256, 0, stream>>>(p, tm, tn);
    else
        mxfp4_gemm_tile_kernel<WB, CT, false, false><<<grid, 256, 0, stream>>>(p, tm, tn);
    return hipGetLastError();
}

template <int CT>
hipError_t launch_typed(const MxGemmParams &p, int x_dt, hipStream_t stream)
{
    if (p.m <= 16) return launch_few<1, CT>(p, x_dt, stream);
    if (p.m <= 32) return launch_few<2, CT>(p, x_dt, stream);
    // the tiled kernels need rows of 128 bytes, and offsets within a tile of 31 bits
    if (p.k <= 128 || mx_pitch(p.k) * 260 > 0x7fffffffLL) return launch_few<4, CT>(p, x_dt, stream);
    // Microseconds, fitted to 50 shapes (m 33 .. 8192, n 1000 .. 14336, k 512 ..
    // 14336), most within a tenth of what was measured:
    // few rows: 80 rows of codes per workgroup, one at 35 GB/s, all at 8.3 TB/s;
    // tiles of 128: a stage of 256 takes a lone workgroup 0.45, and 256 of them
    //   together 0.44 and 2.2 to begin and end;
    // tiles of 256: a stage takes 1.65, a tile's beginning and end 6.
    // Where they differ most: 64 x 14336 x 4096 few 21.9, 128 11.4; 256 x 1000 x
    // 2000 few 5.5, 128 6.9; 8192 x 8192 x 4096 128 152, 256 130; 4300 x 4400 x
    // 640 128 22.4, 256 26.5.
    const double k = (double)p.k, stages = k / 256;
    const double few = (double)((p.m + 63) / 64) * (double)((p.n + 15) / 16);
    const double t128 = (double)((p.m + 127) / 128) * (double)((p.n + 127) / 128);
    const double t256 = (double)((p.m + 255) / 256) * (double)((p.n + 255) / 256);
    const double us_few = 2.0 + std::max(k * 1.16e-3, few * 40.0 * k / 8.3e6);
    const double us_128 = 3.0 + std::max(1.0 + 0.45 * stages, t128 / 256 * (2.2 + 0.44 * stages));
    const double us_256 = 3.0 + std::ceil(t256 / 256) * (6.0 + 1.65 * stages);
    if (us_few <= us_128 && us_few <= us_256) return launch_few<4, CT>(p, x_dt, stream);
    return us_128 <= us_256 ? launch_tile<4, CT>(p, stream) : launch_tile<8, CT>(p, stream);
}

}  // namespace

// Every workgroup of 16 columns quantises the rows it needs, at 6e-5 us a row and
// column of x while up to 384 of them run side by side; a launch that does it
// once costs 4 us. Measured, one launch against two: 14336 x 4096, 4 rows 8.4
// and 10.3 us, 12 rows 12.3 and 11.5; 4096 x 14336, 4 rows 10.0 and 10.9, 6 rows 11.9
// and 11.0; 4096 x 4096, 16 rows 6.8 and 8.2. A row that ends inside a block costs
// 1 us more, as that block is read piece by piece: 1000 x 500, 2 rows 4.1 and
// 7.4, 8 rows 10.3 and 7.1.
bool mx_quantize_inside(long long m, long long n, long long k)
{
    if (m > kMxFewRows) return false;
    const double groups = (double)((n + 15) / 16);
    return (double)m * ((double)k * 6e-5 * std::max(1.0, groups / 384) + (k % 32 ? 1.0 : 0.0)) <= 4.0;
}

hipError_t launch_mxfp4_gemm(const MxGemmParams &p, int c_dt, int x_dt, hipStream_t stream)
{
    return c_dt == kF32 ? launch_typed<kF32>(p, x_dt, stream) : launch_typed<kBF16>(p, x_dt, stream);
}

}  // namespace dps
