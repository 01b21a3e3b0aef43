// Product of an 8-bit block-scaled matrix with a 4-bit or an 8-bit one, C[M, N] =
// A[M, K] . B[N, K]^T with both quantised along K, on gfx950's scaled matrix
// instruction v_mfma_scale_f32_16x16x128_f8f6f4, which takes each operand in its
// own format.
//
// Operand layout (lane l = 16 g + i), measured: in 4 bits the lane holds the 32
// codes of row i, block g of the step's four; in 8 bits the codes 16 g .. 16 g + 15 and
// 64 + 16 g .. 64 + 16 g + 15 of row i, two chunks of 16 bytes. The scale operand's byte of
// lane l is that of block g whatever the format. D register r of lane l:
// D[4 (l / 16) + r][l % 16]. The instruction gets B's rows first, so that a lane
// ends with 4 consecutive columns of one row of C.
//
// With an 8-bit operand the instruction adds the products of 8 consecutive k on a
// grid of 2^-13 of the largest one's octave, cutting the others to it, and
// everything beyond in fp32 (measured). The largest one's own rounding to 8 bits is up to
// 2^-4 of it; bf16 instructions would keep what is cut, at half the rate or less.
#include <algorithm>
#include <cmath>
#include <type_traits>
#include <utility>

#include "mx_gemm_device.h"
#include "mxfp8_internal.h"

namespace dps {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));

constexpr int kE4m3 = 0, kE2m1 = 4;      // the instruction's formats

// a lane's codes of a step of 128: 16 bytes in 4 bits, 32 in 8
template <int BITS> struct Codes { u32x4 lo, hi; };
template <> struct Codes<4> { u32x4 lo; };

template <int BITS>
__device__ __forceinline__ i32x8 operand(const Codes<BITS> &c)
{
    if constexpr (BITS == 8)
        return i32x8{(int)c.lo[0], (int)c.lo[1], (int)c.lo[2], (int)c.lo[3], (int)c.hi[0], (int)c.hi[1], (int)c.hi[2], (int)c.hi[3]};
    else
        return i32x8{(int)c.lo[0], (int)c.lo[1], (int)c.lo[2], (int)c.lo[3], 0, 0, 0, 0};
}
template <int T, int BB>
__device__ __forceinline__ f32x4 mfma(const Codes<BB> &b, unsigned bs, const Codes<8> &a, unsigned as, f32x4 c)
{
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(operand<BB>(b), operand<8>(a), c, BB == 8 ? kE4m3 : kE2m1, kE4m3,
                                                            T, (int)bs, T, (int)as);
}
// step `step` of a row that starts at `row`
template <int BITS>
__device__ __forceinline__ Codes<BITS> codes_at(const unsigned char *row, int step, int g)
{
    Codes<BITS> c;
    const unsigned char *at = row + step * (16 * BITS) + g * 16;
    c.lo = *reinterpret_cast<const u32x4 *>(at);
    if constexpr (BITS == 8) c.hi = *reinterpret_cast<const u32x4 *>(at + 64);
    return c;
}
template <int BITS> __device__ __forceinline__ long long pitch_of(long long k) { return BITS == 8 ? mx8_pitch(k) : mx_pitch(k); }

// A workgroup computes 16 MB rows of C by 16 columns; its 4 waves take
// 512-wide pieces of K in turn, straight from global memory, and their sums
// meet in LDS in a fixed order. Bound by how fast a workgroup gets its 16 rows of B, a cache line of each
// at a time: 8 x 4096 x 14336 with a 4-bit B 10.2 us, its 31 MB at 3.1 TB/s.
template <int MB, int CT, int BB>
__global__ __launch_bounds__(256) void mxfp8_gemm_few_kernel(const MxGemmParams p, unsigned first)
{
    __shared__ f32x4 part[3][MB][64];
    const int lane = threadIdx.x & 63;
    // a scalar, so that what depends on it is skipped by a jump: the matrix
    // instructions run whatever the lane mask says
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int i = lane & 15, g = lane >> 4;
    const unsigned id = first + blockIdx.x, blocks_n = (unsigned)((p.n + 15) >> 4), bm = id / blocks_n;
    const long long n0 = (long long)(id - bm * blocks_n) * 16, m0 = (long long)bm * 16 * MB;
    const long long tiles = mx_scale_tiles(p.k);
    const int steps = (int)((p.k + 127) / 128);
    const unsigned char *brow = p.b + min(n0 + i, p.n - 1) * pitch_of<BB>(p.k);
    // rows past the last are the last one: they are not stored
    long long ra[MB];
#pragma unroll
    for (int b = 0; b < MB; ++b) ra[b] = min(m0 + b * 16 + i, p.m - 1);
    f32x4 acc[MB];
#pragma unroll
    for (int b = 0; b < MB; ++b) acc[b] = f32x4{};
    for (int kt = wave; kt < (int)tiles; kt += 4) {
        const int here = min(4, steps - kt * 4);
        Codes<BB> bw[4];
        const unsigned bs = *reinterpret_cast<const unsigned *>(p.b_scales + ((n0 >> 4) * tiles + kt) * 256 + lane * 4);
#pragma unroll
        for (int t = 0; t < 4; ++t)
            if (t < here) bw[t] = codes_at<BB>(brow, kt * 4 + t, g);
#pragma unroll
        for (int b = 0; b < MB; ++b) {
            Codes<8> aw[4];
            const unsigned as = *reinterpret_cast<const unsigned *>(p.a_scales + ((ra[b] >> 4) * tiles + kt) * 256 +
                                                                    (g * 16 + (int)(ra[b] & 15)) * 4);
            const unsigned char *arow = p.a + ra[b] * mx8_pitch(p.k);
#pragma unroll
            for (int t = 0; t < 4; ++t)
                if (t < here) aw[t] = codes_at<8>(arow, kt * 4 + t, g);
            acc[b] = mfma<0, BB>(bw[0], bs, aw[0], as, acc[b]);
            if (here > 1) acc[b] = mfma<1, BB>(bw[1], bs, aw[1], as, acc[b]);
            if (here > 2) acc[b] = mfma<2, BB>(bw[2], bs, aw[2], as, acc[b]);
            if (here > 3) acc[b] = mfma<3, BB>(bw[3], bs, aw[3], as, acc[b]);
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

template <int MB, int CT, int BB>
hipError_t launch_few(const MxGemmParams &p, hipStream_t stream)
{
    const long long groups = (p.n + 15) / 16 * ((p.m + 16 * MB - 1) / (16 * MB));
    return launch_groups256(groups, [&](unsigned first, unsigned grid) {
        mxfp8_gemm_few_kernel<MB, CT, BB><<<grid, 256, 0, stream>>>(p, first);
    });
}

// ------------------------------------------------------------ tiled kernel

// The matrix instruction with its sums in the accumulation registers for good, as in
// the 4-bit product. Scale byte T of both operands.
template <int T, int BB>
__device__ __forceinline__ void mfma_acc(f32x4 &c, const i32x8 &b8, u32x4 b4, unsigned bs, const i32x8 &a, unsigned as)
{
#define MX8_MFMA(sel)                                                                                          \
    if constexpr (BB == 8)                                                                                     \
        asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 %0, %1, %2, %0, %3, %4 " sel                           \
                     : "+a"(c) : "v"(b8), "v"(a), "v"(bs), "v"(as));                                           \
    else                                                                                                       \
        asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 %0, %1, %2, %0, %3, %4 " sel " cbsz:4"                 \
                     : "+a"(c) : "v"(b4), "v"(a), "v"(bs), "v"(as))
    if constexpr (T == 0) {
        MX8_MFMA("op_sel_hi:[0,0,0]");
    } else if constexpr (T == 1) {
        MX8_MFMA("op_sel:[1,1,0] op_sel_hi:[0,0,0]");
    } else if constexpr (T == 2) {
        MX8_MFMA("op_sel_hi:[1,1,0]");
    } else {
        MX8_MFMA("op_sel:[1,1,0] op_sel_hi:[1,1,0]");
    }
#undef MX8_MFMA
}

// f(0), f(1), ..., each with its number as a type
template <typename F, int... I>
__device__ __forceinline__ void each_of(F f, std::integer_sequence<int, I...>)
{
    (f(std::integral_constant<int, I>{}), ...);
}
template <int N, typename F>
__device__ __forceinline__ void each(F f)
{
    each_of(f, std::make_integer_sequence<int, N>{});
}

// What stands before instruction q of a stage's N: the number of a read, load or scale there, -1 for
// none (k: of those that share a place).
template <int WB, int BB> struct Plan {
    static constexpr int N = WB * WB, loads = WB + WB * BB / 8;
    static constexpr int D = WB == 2 ? 4 : 2;                           // buffers
    static constexpr int x = WB == 8 ? 16 : WB == 4 ? 5 : -1;           // the barrier after the reads of A (WB = 2: none)
    static constexpr int y = WB == 8 ? (BB == 8 ? 34 : 44) : WB == 4 ? 9 : 3;       // the one before the next stage's reads
    static constexpr int scales = D == 4 ? 0 : 2;                       // the stage of four that loads the next four's scales
    static constexpr int read_a_at(int r) { return (r - 2) * 2; }       // fragments 2 .. WB - 1
    static constexpr int load_at(int j) { return WB == 8 ? x + (BB == 8 ? j * 5 / 2 : j * 3) : WB == 4 ? x + j / 2 : y; }
    static constexpr int next_at(int r) { return WB == 8 ? y + (BB == 8 ? r * 3 : r * 2) : WB == 4 ? y + r : y; }
    static constexpr int scale_at(int r) { return WB == 8 ? r : r / 2; }
    static constexpr int find(int (*at)(int), int from, int to, int q, int k)
    {
        for (int r = from; r < to; ++r)
            if (at(r) == q && k-- == 0) return r;
        return -1;
    }
    static constexpr int read_a(int q) { return find(read_a_at, 2, WB, q, 0); }
    static constexpr int load(int q, int k) { return find(load_at, 0, loads, q, k); }
    static constexpr int read_next(int q, int k) { return find(next_at, 0, WB + 2, q, k); }
    static constexpr int scale(int q, int k) { return find(scale_at, 0, 2 * WB, q, k); }
    static constexpr int count_before_y()
    {
        int n = (D - 2) * loads;
        for (int j = 0; j < loads; ++j) n += load_at(j) < y;
        return n;
    }
    static constexpr int newer = count_before_y();                      // loads of stages after the next that y does not wait for
    static_assert(next_at(WB + 1) < N && load_at(loads - 1) < N && scale_at(2 * WB - 1) < y, "within the stage");
    static_assert(WB == 2 || (read_a_at(WB - 1) < x && scale_at(2 * WB - 1) < x), "before the loads");
};

// Tile of 32 WB x 32 WB, 4 waves of 16 WB x 16 WB (WB x WB instructions a stage). A
// stage is 128 of K and goes from global memory straight into one of D LDS buffers
// (buffer_load ... lds, 1 KiB an instruction). In 8 bits a row of a stage is 8
// chunks of 16 bytes, chunk c of row r at position c ^ (r % 8); in 4 bits two rows
// share such a line, row r's chunk c being number 4 (r % 2) + c of line r / 2: the
// 16 rows that a fragment read touches hit distinct banks.
//
// Of stage t a wave holds all fragments of B (two sets, one being read while the other is
// used) and all of A. The instructions of a stage are numbered q; between them stand, with two buffers
// (tiles of 128 and 256):
//   the reads of A's fragments 2 and up of stage t
//   X: every wave has read stage t; the loads of stage t + 2 go into its buffer
//   Y: stage t + 1 is there; its fragments of B and the first two of A are read
// so that a load has a stage and more to arrive. A tile of 64 has 4 instructions a wave and stage, less
// than a load takes, and two fragments of A, read a stage ahead: its buffers are four, and
//   Y: every wave has read stage t, and stage t + 1 is there; the loads of stage t + 4 go into t's
//      buffer, t + 1 is read
// is its only barrier (201 x 4096 x 4096: 8.9 us, with two buffers 14.2 in tiles of 128).
//
// Measured: 4096 x 4096 x 4096 with a 4-bit B 50 to 51 us (2.7 PFLOP/s; B in 8 bits 51 to 52, C in fp32 56 to 62), 8192 x
// 14336 x 4096 321 to 374 by the card's clock (2.6 to 3.0). A loop of these instructions alone reaches 3.7 on uniformly
// random codes and 4.0 on those of a normal distribution, in 4 bits or 8: the 8-bit operand's rate and the card's power
// bound the large product; its matrix units are busy 66 to 74% of the cycles and its waves wait in 13%.
//
// Scales come as one 32-bit load per 16 rows and four stages (512 of K), loaded in
// the third stage of the four before. K is walked in fours of stages; a stage past the
// row's end is loaded from the row's last chunks instead, and gets scale bytes of
// zero on both sides: whatever codes stand there, their products are at most 2^-254 *
// 448^2 and vanish against fp32's smallest 2^-149. Rows past M or N are
// loads of the last row, and their results are not stored.
//
// LOOP: with more tiles of 256 than CUs, 256 workgroups go through them, and load a
// tile's first stages during the last ones of the tile before.
template <int WB, int CT, int BB, bool VEC, bool LOOP>
__global__ __launch_bounds__(256) void mxfp8_gemm_tile_kernel(const MxGemmParams p, int tiles_m, int tiles_n)
{
#ifdef __HIP_DEVICE_COMPILE__                        // the host pass rejects the body's operands, and needs none
    using P = Plan<WB, BB>;
    constexpr int T = 32 * WB;                       // tile side
    constexpr int BSTEP = 16 * BB;                   // bytes of a row of B in a stage
    constexpr int NA = WB, NB = WB * BB / 8;         // a wave's loads a stage
    __shared__ __attribute__((aligned(1024))) unsigned char A0[T * 128], A1[T * 128], B0[T * BSTEP], B1[T * BSTEP];
    constexpr int D = P::D;                          // buffers, each an object of its own: a wait for one is none for another
    __shared__ __attribute__((aligned(1024))) unsigned char A2[D == 4 ? T * 128 : 1], A3[D == 4 ? T * 128 : 1], B2[D == 4 ? T * BSTEP : 1], B3[D == 4 ? T * BSTEP : 1];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wi = wave >> 1, wj = wave & 1, i = lane & 15, g = lane >> 4;
    const int pitch_a = (int)mx8_pitch(p.k), pitch_b = (int)pitch_of<BB>(p.k), ktiles = (int)mx_scale_tiles(p.k);
    const int steps = (int)((p.k + 127) / 128), groups = (steps + 3) / 4;
    // selection of the last four's scale bytes (0x0c selects a zero byte)
    const int rest = steps % 4;
    const unsigned tail = rest == 0 ? 0x03020100u : rest == 1 ? 0x0c0c0c00u : rest == 2 ? 0x0c0c0100u : 0x0c020100u;
    auto abuf = [&](int buf) __attribute__((always_inline)) { return buf == 0 ? A0 : buf == 1 ? A1 : buf == 2 ? A2 : A3; };
    auto bbuf = [&](int buf) __attribute__((always_inline)) { return buf == 0 ? B0 : buf == 1 ? B1 : buf == 2 ? B2 : B3; };

    // the tile that is being loaded: its corner in C and its rows of codes and scales; offsets
    // within them fit 31 bits (checked by the launcher)
    long long lm0, ln0;
    const unsigned char *la, *lb, *lsa, *lsb;
    int last_a, last_b, last_sa, last_sb;
    auto place = [&](int tile) __attribute__((always_inline)) {
        int tm, tn;
        tile_of(tile, tiles_m, tiles_n, tm, tn);
        lm0 = (long long)tm * T;
        ln0 = (long long)tn * T;
        const int rows_a = (int)min((long long)T, p.m - lm0), rows_b = (int)min((long long)T, p.n - ln0);
        la = p.a + lm0 * pitch_a;
        lb = p.b + ln0 * pitch_b;
        lsa = p.a_scales + lm0 / 16 * ktiles * 256;
        lsb = p.b_scales + ln0 / 16 * ktiles * 256;
        last_a = (rows_a - 1) * pitch_a;
        last_b = (rows_b - 1) * pitch_b;
        last_sa = (rows_a - 1) >> 4;
        last_sb = (rows_b - 1) >> 4;
    };
    auto rsrc = [](const unsigned char *base) __attribute__((always_inline)) {
        return __builtin_amdgcn_make_buffer_rsrc((void *)base, (short)0, 0x7fffffff, 0x00020000);
    };
    // lane l of a load fills position l % 8 of line l / 8
    const int line = lane >> 3, slot = (lane & 7) ^ line;
    const int row_a = (wave * 8 * NA + line) * pitch_a, chunk_a = slot * 16;
    const int row_b = BB == 8 ? (wave * 8 * NB + line) * pitch_b : (wave * 16 * NB + 2 * line + (slot >> 2)) * pitch_b;
    const int chunk_b = BB == 8 ? slot * 16 : (slot & 3) * 16;
    // load j of a stage: j < NB B's, else A's j - NB
    auto dtl = [&](int buf, int stage, int j) __attribute__((always_inline)) {
        if (j < NB) {
            const int so = __builtin_amdgcn_readfirstlane(min(stage * BSTEP, pitch_b - BSTEP));
            const int vo = min(row_b + j * (BB == 8 ? 8 : 16) * pitch_b, last_b) + chunk_b;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc(lb), (lds_void *)(bbuf(buf) + (wave * NB + j) * 1024), 16, vo, so, 0, 0);
        } else {
            const int so = __builtin_amdgcn_readfirstlane(min(stage * 128, pitch_a - 128));
            const int vo = min(row_a + (j - NB) * 8 * pitch_a, last_a) + chunk_a;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc(la), (lds_void *)(abuf(buf) + (wave * NA + j - NB) * 1024), 16, vo, so, 0, 0);
        }
    };
    // scales of 16-row group x of this wave's rows (x < WB: A's group x, else B's x - WB), stages 4 kt and on
    auto scale = [&](int x, int kt) __attribute__((always_inline)) {
        const int group = x < WB ? min(wi * WB + x, last_sa) : min(wj * WB + x - WB, last_sb);
        return (unsigned)__builtin_amdgcn_raw_buffer_load_b32(rsrc(x < WB ? lsa : lsb), lane * 4,
                                                              __builtin_amdgcn_readfirstlane((group * ktiles + kt) * 256), 0);
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
    i32x8 af[WB], bf8[BB == 8 ? 2 : 1][BB == 8 ? WB : 1];
    u32x4 bf4[BB == 4 ? 2 : 1][BB == 4 ? WB : 1];
    unsigned sa[WB], sb[WB], ns[2 * WB];

    int tile = blockIdx.x;
    place(tile);
    long long m0 = lm0, n0 = ln0;
#pragma unroll
    for (int d = 0; d < D; ++d)
#pragma unroll
        for (int j = 0; j < NA + NB; ++j) dtl(d, d, j);
#pragma unroll
    for (int x = 0; x < 2 * WB; ++x) ns[x] = scale(x, 0);
    MX_FENCE();
    auto take = [&](unsigned &x, unsigned next, unsigned sel) __attribute__((always_inline)) {
        x = __builtin_amdgcn_perm(0u, next, sel);
        mx_pin(x);
    };
#pragma unroll
    for (int x = 0; x < WB; ++x) {
        take(sa[x], ns[x], groups == 1 ? tail : 0x03020100u);
        take(sb[x], ns[WB + x], groups == 1 ? tail : 0x03020100u);
    }
    mx_settle();
    // fragments: two reads of A's, one or two of B's
    const int at8 = i * 128 + ((g ^ (lane & 7)) << 4);
    const int at4 = (i >> 1) * 128 + ((((i & 1) * 4 + g) ^ (i >> 1)) << 4);
    auto read8 = [&](i32x8 &f, const unsigned char *from) __attribute__((always_inline)) {
        const u32x4 lo = *reinterpret_cast<const u32x4 *>(from + at8), hi = *reinterpret_cast<const u32x4 *>(from + (at8 ^ 64));
        f = __builtin_shufflevector((i32x4)lo, (i32x4)hi, 0, 1, 2, 3, 4, 5, 6, 7);
    };
    auto read_a = [&](int buf, int x) __attribute__((always_inline)) { read8(af[x], abuf(buf) + (wi * WB + x) * 2048); };
    auto read_b = [&](int set, int buf, int x) __attribute__((always_inline)) {
        if constexpr (BB == 8)
            read8(bf8[set][x], bbuf(buf) + (wj * WB + x) * 2048);
        else
            bf4[set][x] = *reinterpret_cast<const u32x4 *>(bbuf(buf) + (wj * WB + x) * 1024 + at4);
    };
    constexpr int N = P::N;
    constexpr int kStores = LOOP && VEC ? N / 2 : 0;
    // loads that Y does not wait for: of the stages after the next one, and the scales issued since
    constexpr auto newer = [](int S) { return P::newer + (D == 4 ? S < 3 : S == 2) * 2 * WB; };
    static_assert(newer(2) < 64 && newer(0) + kStores < 64, "a wait counts at most 63");
    // stage 4 kt + S; `next`: the stage to load, D ahead
    auto stage = [&](auto s_, int next, int next_kt, unsigned sel, bool stores) __attribute__((always_inline)) {
        constexpr int S = decltype(s_)::value, buf = S % D, then = (S + 1) % D, set = S & 1;
        each<N>([&](auto q_) __attribute__((always_inline)) {
            constexpr int q = decltype(q_)::value, a = q / WB, b = q % WB;
            if constexpr (q == P::x) {
                MX_FENCE();
                mx_wait<63, true>();
                __builtin_amdgcn_s_barrier();
                MX_FENCE();
            }
            if constexpr (S == P::scales) {
                if constexpr (P::scale(q, 0) >= 0) ns[P::scale(q, 0)] = scale(P::scale(q, 0), next_kt);
                if constexpr (P::scale(q, 1) >= 0) ns[P::scale(q, 1)] = scale(P::scale(q, 1), next_kt);
            }
            if constexpr (q == P::y) {
                MX_FENCE();
                if (S == 0 && kStores && stores)
                    mx_wait<newer(S) + kStores, false>();
                else
                    mx_wait<newer(S), false>();
                __builtin_amdgcn_s_barrier();
                MX_FENCE();
            }
            if constexpr (P::read_a(q) >= 0) read_a(buf, P::read_a(q));
            each<4>([&](auto k_) __attribute__((always_inline)) {
                constexpr int j = P::load(q, decltype(k_)::value);
                if constexpr (j >= 0) dtl(buf, next, j);
            });
            // the next stage's, in this order: A's fragment 0, B's, A's 1
            auto next_reads = [&](auto k_) __attribute__((always_inline)) {
                constexpr int r = P::read_next(q, decltype(k_)::value);
                if constexpr (r == 0 || r == WB + 1)
                    read_a(then, r == 0 ? 0 : 1);
                else if constexpr (r > 0)
                    read_b(set ^ 1, then, r - 1);
            };
            if constexpr (WB > 2) each<4>(next_reads);
            mfma_acc<S, BB>(acc[a][b], bf8[BB == 8 ? set : 0][BB == 8 ? b : 0], bf4[BB == 4 ? set : 0][BB == 4 ? b : 0], sb[b],
                            af[a], sa[a]);
            // with two fragments the last instruction uses what is read next
            if constexpr (WB == 2) each<4>(next_reads);
            // the next four's scales take their place as soon as this one's have
            // been used, before their first use by WB - 1 instructions
            if constexpr (S == 3) {
                if constexpr (b == 0 && a > 0) take(sa[a - 1], ns[a - 1], sel);
                if constexpr (q > N - WB) take(sb[b - 1], ns[WB + b - 1], sel);
                if constexpr (q == N - 1) {
                    take(sa[WB - 1], ns[WB - 1], sel);
                    take(sb[WB - 1], ns[2 * WB - 1], sel);
                    // with few instructions to a stage the first use follows at once
                    if constexpr (WB == 2) asm volatile("s_nop 3");
                }
            }
            MX_FENCE();
        });
    };
    __builtin_amdgcn_s_waitcnt(0x0F70);
    __syncthreads();
#pragma unroll
    for (int x = 0; x < WB; ++x) read_b(0, 0, x);
    read_a(0, 0);
    read_a(0, 1);
    MX_FENCE();
    const int tiles = tiles_m * tiles_n;
    bool stores = false;
    for (;;) {
        const int following = tile + gridDim.x;
        for (int kt = 0; kt < groups; ++kt) {
            // the last four load the first stages of the workgroup's next tile, which then goes on
            // without a pause (without a next tile, this one's again, to be read by no one)
            const int next = kt + 1 < groups ? kt + 1 : 0;
            const unsigned sel = next + 1 == groups ? tail : 0x03020100u;
            stage(std::integral_constant<int, 0>{}, D == 4 ? 4 * next : 4 * kt + 2, next, 0u, stores);
            stage(std::integral_constant<int, 1>{}, D == 4 ? 4 * next + 1 : 4 * kt + 3, 0, 0u, false);
            if (LOOP && next == 0 && following < tiles) place(following);
            stage(std::integral_constant<int, 2>{}, D == 4 ? 4 * next + 2 : 4 * next, next, 0u, false);
            stage(std::integral_constant<int, 3>{}, D == 4 ? 4 * next + 3 : 4 * next + 1, 0, sel, false);
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
        put_tile<WB, CT, VEC>(p, acc, m0 + wi * 16 * WB, n0 + wj * 16 * WB);
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

template <int WB, int CT, int BB>
hipError_t launch_tile(const MxGemmParams &p, hipStream_t stream)
{
    const int T = 32 * WB;
    const int tm = (int)((p.m + T - 1) / T), tn = (int)((p.n + T - 1) / T);
    constexpr int CUS = 256;
    const bool loop = WB == 8 && tm * tn > CUS;
    const int grid = loop ? CUS : tm * tn;
    // rows of C on 16 bytes: 16-byte stores
    const bool vec = CT == kBF16 && (uintptr_t)p.c % 16 == 0 && p.n % 8 == 0;
    if (vec && loop)
        mxfp8_gemm_tile_kernel<WB, CT, BB, CT == kBF16, WB == 8><<<grid, 256, 0, stream>>>(p, tm, tn);
    else if (vec)
        mxfp8_gemm_tile_kernel<WB, CT, BB, CT == kBF16, false><<<grid, 256, 0, stream>>>(p, tm, tn);
    else if (loop)
        mxfp8_gemm_tile_kernel<WB, CT, BB, false, WB == 8><<<grid, 256, 0, stream>>>(p, tm, tn);
    else
        mxfp8_gemm_tile_kernel<WB, CT, BB, false, false><<<grid, 256, 0, stream>>>(p, tm, tn);
    return hipGetLastError();
}

// Microseconds, fitted to 250 shapes (m 1 .. 4096, n 64 .. 14336, k 128 .. 14336); a half to two thirds of the estimates
// are within a tenth of what was measured. The second figure of a pair is for B in 8 bits:
// few rows: what a workgroup reads of B and of A's rows, one alone and 256 of them together;
// tiles of 64, 128: a stage takes a lone workgroup so long, and 256 of them together so long besides their
//   begin and end; with tiles of 64, which few rows take too, B comes at 4.5 TB/s;
// tiles of 256: a stage takes 1.21 or 1.3, a tile's begin and end 6.
// Where they differ most (us by few rows, 64, 128, 256): 1 x 4096 x 14336 10.9, 25.8; 32 x 14336 x 4096 21.4,
// 11.3; 64 x 14336 x 4096 35.4, 9.5, 15.5; 201 x 4096 x 4096 30.1, 8.9, 14.2, 36.4; 1024 x 4096 x 4096 130, 25.5, 18.9, 38.0;
// 4096 x 4096 x 4096 -, -, 63.4, 47.0.
// Of 402 choices (17 .. 1024 rows, weights in cache) 30 cost more than a tenth over the best of few rows, 64 and 128, and 17
// more than a fifth. Tiles of 128 are taken too early then, with B in 8 bits over wide weights, as its bytes count against
// tiles of 64 alone (us by 128, taken, and by 64: 64 x 14336 x 14336 49.5, 33.2; 64 x 14336 x 4096 17.7, 12.9; 64 x 14336 x
// 2000 10.3, 7.1), with B in 4 bits less often (201 x 4096 x 512 5.6, 4.2; 128 x 14336 x 4096 17.2, 14.0).
template <int CT, int BB>
hipError_t launch_typed(const MxGemmParams &p, hipStream_t stream)
{
    constexpr bool EIGHT = BB == 8;
    // the tiled kernels need offsets within a tile of 31 bits
    if (mx8_pitch(p.k) * 260 > 0x7fffffffLL) return launch_few<2, CT, BB>(p, stream);
    const double m = (double)p.m, n = (double)p.n, k = (double)p.k, stages = 4 * std::ceil(k / 512);
    auto tiles = [&](double side) { return std::ceil(m / side) * std::ceil(n / side) / 256; };
    const double us_few = p.m > 32 ? 1e30
                                   : 2.2 + k * 1e-3 * std::max((EIGHT ? 0.75 : 0.55) + 0.018 * m,
                                                               std::ceil(n / 16) / 256 * ((EIGHT ? 0.94 : 0.48) + 0.026 * m));
    const double us_64 = 3.2 + std::max(std::max((EIGHT ? 0.24 : 0.155) * stages, tiles(64) * (0.55 + (EIGHT ? 0.2 : 0.17) * stages)),
                                        n * k * (EIGHT ? 33 : 17) / 32 / 4.5e6);
    const double us_128 = 3.0 + std::max((EIGHT ? 0.36 : 0.33) * stages, tiles(128) * (1.6 + (EIGHT ? 0.5 : 0.45) * stages));
    const double us_256 = 3.0 + std::ceil(tiles(256)) * (6.0 + (EIGHT ? 1.3 : 1.21) * stages);
    const double us = std::min(std::min(us_few, us_64), std::min(us_128, us_256));
    if (us == us_few) return p.m <= 16 ? launch_few<1, CT, BB>(p, stream) : launch_few<2, CT, BB>(p, stream);
    if (us == us_64) return launch_tile<2, CT, BB>(p, stream);
    return us == us_128 ? launch_tile<4, CT, BB>(p, stream) : launch_tile<8, CT, BB>(p, stream);
}

}  // namespace

hipError_t launch_mxfp8_gemm(const MxGemmParams &p, int b_bits, int c_dt, hipStream_t stream)
{
    if (c_dt == kF32) return b_bits == 8 ? launch_typed<kF32, 8>(p, stream) : launch_typed<kF32, 4>(p, stream);
    return b_bits == 8 ? launch_typed<kBF16, 8>(p, stream) : launch_typed<kBF16, 4>(p, stream);
}

}  // namespace dps
