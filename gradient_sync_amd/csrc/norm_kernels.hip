// Root-mean-square norm of the rows of h = x + residual, and its gradients.
//
//   rstd = 1 / sqrt(mean(h^2) + eps);  y = h rstd w
//   with u = h rstd and g = dy w:  dh = rstd (g - u mean(g u)) + dresidual
//                                  dw = sum over the rows of dy u
//
// A row is read once: a wave (or, for few or long rows, a workgroup) keeps its row in registers
// between the sum and the output. The squares are summed in fp64, so that neither
// a row of large values overflows nor one of small values vanishes; the output in
// 8 bits is quantised from the fp32 values, 4 lanes a block of 32.
#include <algorithm>
#include <type_traits>

#include "mxfp8_device.h"
#include "norm_internal.h"

namespace dps {
namespace {

constexpr int kNT = 256;

// 8 elements of fp32 or bf16 from p on, the first n of them (zero past them)
__device__ __forceinline__ void load8(const char *p, int dt, long long at, int n, float (&v)[8])
{
    if (dt == kF32) {
        const float *s = reinterpret_cast<const float *>(p) + at;
        if (n >= 8) {
            typedef float f32x4_e __attribute__((ext_vector_type(4), aligned(4)));
            const f32x4_e a = reinterpret_cast<const f32x4_e *>(s)[0], b = reinterpret_cast<const f32x4_e *>(s)[1];
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = a[i], v[4 + i] = b[i];
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = i < n ? s[i] : 0.0f;
        }
    } else {
        const unsigned short *s = reinterpret_cast<const unsigned short *>(p) + at;
        if (n >= 8) {
            const mx_u32x4 a = *reinterpret_cast<const mx_u32x4_e *>(s);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[2 * i] = __uint_as_float(a[i] << 16), v[2 * i + 1] = __uint_as_float(a[i] & 0xffff0000u);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = i < n ? __uint_as_float((unsigned)s[i] << 16) : 0.0f;
        }
    }
}
// 8 elements of a row of `cols` as they are stored, from its element `col` on, for `settle` to put in place: past the
// row's end they are the row's last 8, at the far end of which stand the n that are asked for. Such a load has no
// condition, and nothing waits for it before its use: gradients of 8192 x 2500 bf16 41 us against 92 with a condition to each
// element, 8192 x 2501 48 against 115, 16384 x 501 20.2 against 47.9, 100000 x 100 68 against 195. The elements may
// be another thread's: what is written in place of a row comes behind a barrier after its loads, or from the same wave.
enum { kOrdinary, kOnce, kUnder8 };                  // loads: ordinary, nontemporal, of rows of fewer than 8 elements
template <int DT> struct Raw { mx_u32x4 v[DT == kF32 ? 2 : 1]; };
template <int DT, int HOW>
__device__ __forceinline__ Raw<DT> load_row(const char *p, long long row, long long col, long long cols)
{
    Raw<DT> r;
    if constexpr (HOW == kUnder8) {
#pragma unroll
        for (mx_u32x4 &v : r.v) v = mx_u32x4{};
#pragma unroll
        for (int i = 1; i < 8; ++i) {
            const int from = i - 8 + (int)cols;
            if (from < 0) continue;
            if constexpr (DT == kF32)
                r.v[i >> 2][i & 3] = reinterpret_cast<const unsigned *>(p)[row + from];
            else
                r.v[0][i >> 1] |= (unsigned)reinterpret_cast<const unsigned short *>(p)[row + from] << (16 * (i & 1));
        }
    } else {
        const mx_u32x4_e *s = reinterpret_cast<const mx_u32x4_e *>(p + (row + min(col, cols - 8)) * (DT == kF32 ? 4 : 2));
        r.v[0] = HOW == kOnce ? __builtin_nontemporal_load(s) : s[0];
        if constexpr (DT == kF32) r.v[1] = HOW == kOnce ? __builtin_nontemporal_load(s + 1) : s[1];
    }
    return r;
}
// the first n elements in their places, zero past them
template <int DT>
__device__ __forceinline__ void settle(Raw<DT> &r, int n)
{
    if (n >= 8) return;
    constexpr int W = DT == kF32 ? 8 : 4;            // dwords
    const int off = 8 - n;
    unsigned w[W + 4] = {};
#pragma unroll
    for (int i = 0; i < W; ++i) {
        const unsigned x = r.v[i >> 2][i & 3];
        w[i] = n > 0 ? x : 0u;
    }
    const auto pick = [](int from, unsigned a, unsigned b) __attribute__((always_inline)) { return from ? a : b; };
    // by 4 elements, by 2, by 1
#pragma unroll
    for (int i = 0; i < W; ++i) w[i] = pick(off & 4, w[i + (W == 8 ? 4 : 2)], w[i]);
#pragma unroll
    for (int i = 0; i < W; ++i) w[i] = pick(off & 2, w[i + (W == 8 ? 2 : 1)], w[i]);
#pragma unroll
    for (int i = 0; i < W; ++i) w[i] = pick(off & 1, W == 8 ? w[i + 1] : w[i] >> 16 | w[i + 1] << 16, w[i]);
#pragma unroll
    for (int i = 0; i < W; ++i) r.v[i >> 2][i & 3] = w[i];
}
template <int DT>
__device__ __forceinline__ float value(const Raw<DT> &r, int i)
{
    if constexpr (DT == kF32) return __uint_as_float(r.v[i >> 2][i & 3]);
    const unsigned w = r.v[0][i >> 1];
    return __uint_as_float(i & 1 ? w & 0xffff0000u : w << 16);
}
template <int DT, int HOW>
__device__ __forceinline__ void load8_row(const char *p, long long col, long long cols, int n, float (&v)[8])
{
    Raw<DT> r = load_row<DT, HOW == kUnder8 ? kUnder8 : kOrdinary>(p, 0, col, cols);
    settle<DT>(r, n);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = value<DT>(r, i);
}

__device__ __forceinline__ unsigned pack2(float a, float b)
{
    const mx_f32x2 v = {a, b};
    return __builtin_bit_cast(unsigned, __builtin_convertvector(v, mx_bf16x2));
}
__device__ __forceinline__ void store8(char *p, int dt, long long at, int n, const float (&v)[8])
{
    if (dt == kF32) {
        float *d = reinterpret_cast<float *>(p) + at;
        if (n >= 8) {
            typedef float f32x4_e __attribute__((ext_vector_type(4), aligned(4)));
            reinterpret_cast<f32x4_e *>(d)[0] = f32x4_e{v[0], v[1], v[2], v[3]};
            reinterpret_cast<f32x4_e *>(d)[1] = f32x4_e{v[4], v[5], v[6], v[7]};
        } else {
#pragma unroll
            for (int i = 0; i < 7; ++i)
                if (i < n) d[i] = v[i];
        }
    } else {
        unsigned short *d = reinterpret_cast<unsigned short *>(p) + at;
        mx_u32x4 w;
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = pack2(v[2 * i], v[2 * i + 1]);
        if (n >= 8) {
            *reinterpret_cast<mx_u32x4_e *>(d) = w;
        } else {
#pragma unroll
            for (int i = 0; i < 7; ++i)
                if (i < n) d[i] = (unsigned short)(w[i >> 1] >> (16 * (i & 1)));
        }
    }
}
// to the type that the hidden state is kept in
template <int DT>
__device__ __forceinline__ float kept(float x)
{
    if constexpr (DT == kF32) return x;
    return __uint_as_float(pack2(x, x) << 16);
}

// the value of another lane of its row of 16, by a pattern of the data path
template <int CTRL>
__device__ __forceinline__ float moved(float x)
{
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), CTRL, 0xf, 0xf, false));
}
template <int CTRL>
__device__ __forceinline__ double moved(double x)
{
    const int2 v = __builtin_bit_cast(int2, x);
    int2 r;
    r.x = __builtin_amdgcn_update_dpp(0, v.x, CTRL, 0xf, 0xf, false);
    r.y = __builtin_amdgcn_update_dpp(0, v.y, CTRL, 0xf, 0xf, false);
    return __builtin_bit_cast(double, r);
}
// x of the lane's own row of 16 (a pair of rows with HALF) and of its neighbour, added: swapping a value with
// itself leaves one copy with the even row's in both, one with the odd row's
template <bool HALF>
__device__ __forceinline__ unsigned swapped(unsigned x, unsigned &other)
{
    if constexpr (HALF) {
        const auto s = __builtin_amdgcn_permlane32_swap(x, x, false, false);
        other = s[1];
        return s[0];
    } else {
        const auto s = __builtin_amdgcn_permlane16_swap(x, x, false, false);
        other = s[1];
        return s[0];
    }
}
template <bool HALF>
__device__ __forceinline__ float across(float x)
{
    unsigned b;
    const unsigned a = swapped<HALF>(__float_as_uint(x), b);
    return __uint_as_float(a) + __uint_as_float(b);
}
template <bool HALF>
__device__ __forceinline__ double across(double x)
{
    const uint2 v = __builtin_bit_cast(uint2, x);
    uint2 a, b;
    a.x = swapped<HALF>(v.x, b.x);
    a.y = swapped<HALF>(v.y, b.y);
    return __builtin_bit_cast(double, a) + __builtin_bit_cast(double, b);
}
template <bool HALF>
__device__ __forceinline__ unsigned either(unsigned x)
{
    unsigned b;
    const unsigned a = swapped<HALF>(x, b);
    return a | b;
}
// the sum over a wave, in every lane
template <typename T>
__device__ __forceinline__ T wave_sum(T x)
{
    x += moved<0xB1>(x);            // lane ^ 1
    x += moved<0x4E>(x);            // lane ^ 2
    x += moved<0x141>(x);           // mirrored within 8
    x += moved<0x140>(x);           // mirrored within 16
    x = across<false>(x);
    return across<true>(x);
}
// the sum over the TPR threads of a row (a wave, or the whole workgroup), in every one of them. `set` alternates between
// the sums of a workgroup, so that one barrier a sum is enough.
template <int TPR, typename T>
__device__ __forceinline__ T row_sum(T x, int set = 0)
{
    x = wave_sum(x);
    if constexpr (TPR > 64) {
        __shared__ T part[2][TPR / 64];
        part[set][threadIdx.x >> 6] = x;
        __syncthreads();
        x = part[set][0];
#pragma unroll
        for (int i = 1; i < TPR / 64; ++i) x += part[set][i];
    }
    return x;
}
// threads of a workgroup that has TPR a row
template <int TPR> constexpr int kBlock = TPR < kNT ? kNT : TPR;

// 1 / sqrt(mean + eps) as power * (hi + lo), hi in [1, 2)
struct Root {
    float power, hi, lo, rounded;
};
__device__ __forceinline__ Root root_of_mean(double sum, long long cols, double eps)
{
    const double d = sum / (double)cols + eps;
    double r = __builtin_amdgcn_rsq(d);              // to 2^-24 or so; one step of Newton's makes it 2^-47
    if (d < 1e300) r += 0.5 * r * (1.0 - d * r * r);
    Root s;
    s.rounded = (float)r;
    // 2^-128 <= r <= 2^63 of a finite row; zero and NaN go through
    const unsigned e = min(max((unsigned)(__builtin_bit_cast(unsigned long long, r) >> 52), 1023u - 126u), 1023u + 64u);
    s.power = __uint_as_float((e - 1023u + 127u) << 23);
    const double m = r * __builtin_bit_cast(double, (unsigned long long)(2046u - e) << 52);
    s.hi = (float)m;
    s.lo = (float)(m - (double)s.hi);
    return s;
}
// h w / sqrt(mean + eps): of bf16 factors rounded once, of fp32 ones twice. h times the power of two is at
// most sqrt(cols), so that nothing overflows on the way.
__device__ __forceinline__ float normed(float h, float w, const Root &s)
{
    const float t = h * s.power * w;
    return __builtin_fmaf(t, s.hi, t * s.lo);
}

// 8 values of a row (lane's share of chunk `col` .. col + 511) as codes, and the 16 scale bytes of the wave's 512
// columns into their tile: lane 4 b holds the byte of block b, whose place in the tile's 32-bit word
// b % 4 is b / 4, the lane's row of 16.
__device__ __forceinline__ void put8(const RmsNormParams &p, long long row, long long col, const float (&y)[8])
{
    const int lane = threadIdx.x & 63;
    unsigned w[8], top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        w[i] = __float_as_uint(y[i]);
        top = mx_max_f32(top, w[i]);
    }
    const unsigned byte = mx8_scale_byte(mx_max_quad(top));
    const mx_u32x2 code = byte == 255u ? mx_u32x2{0u, 0u} : mx8_pack8(w, mx_scale(byte));
    const long long pitch = mx8_pitch(p.cols);
    if (col < pitch) *reinterpret_cast<mx_u32x2 *>(p.codes + row * pitch + col) = code;
    const unsigned word = either<true>(either<false>(byte << (8 * (lane >> 4))));
    const long long first = col - lane * 8;          // the wave's
    if (lane < 16 && (lane & 3) == 0 && first < p.cols)
        *reinterpret_cast<unsigned *>(p.scales + ((row >> 4) * mx_scale_tiles(p.cols) + (first >> 9)) * 256 +
                                      (((lane >> 2) << 4) + (int)(row & 15)) * 4) = word;
}

template <int DT>
__device__ __forceinline__ void sum8(const RmsNormParams &p, long long row, long long col, int n, float (&h)[8])
{
    load8(p.x, DT, row * p.ldx + col, n, h);
    if (p.residual) {
        float r[8];
        load8(p.residual, DT, row * p.ldr + col, n, r);
#pragma unroll
        for (int i = 0; i < 8; ++i) h[i] = kept<DT>(h[i] + r[i]);
    }
}
__device__ __forceinline__ void out8(const RmsNormParams &p, long long row, long long col, int n, const Root &root,
                                     const float (&h)[8])
{
    float w[8], y[8];
    load8(p.weight, p.w_dt, col, n, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = normed(h[i], w[i], root);
    if (p.y && n > 0) store8(p.y, p.y_dt, row * p.cols + col, n, y);
    if (n < 8) {                                     // a row that is NaN is so up to its end
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = i < n ? y[i] : 0.0f;
    }
    if (p.codes) put8(p, row, col, y);
}

// The first row of workgroup `id`, with RPW a workgroup: workgroups go round-robin to the 8 XCDs, and 16 rows, whose
// scale bytes share lines, are given to workgroups of one XCD, whose L2 puts them together.
template <int RPW>
__device__ __forceinline__ long long swizzled(const RmsNormParams &p, long long id)
{
    constexpr int PER = 16 / RPW;                    // workgroups of 16 rows
    if (p.codes && id < p.rows / 128 * (8 * PER)) {
        const long long in = id % (8 * PER);
        id = id - in + in % 8 * PER + in / 8;
    }
    return id * RPW;
}

// TPR threads a row, NCH chunks of 8 elements a thread. Bound by HBM: 8192 x 4096 bf16 with the residual and
// 8-bit output 45.9 us, its 236 MB at 5.1 TB/s.
template <int DT, int TPR, int NCH>
__global__ __launch_bounds__(kBlock<TPR>) void rms_norm_kernel(const RmsNormParams p, unsigned first)
{
    const int t = threadIdx.x % TPR;
    const long long row = swizzled<kBlock<TPR> / TPR>(p, (long long)first + blockIdx.x) + threadIdx.x / TPR;
    if (row >= p.rows) return;                       // whole waves, or the whole workgroup
    float h[NCH][8];
    double sum = 0;
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
        const long long col = (long long)(c * TPR + t) * 8;
        const int n = (int)min(8LL, max(0LL, p.cols - col));
        sum8<DT>(p, row, col, n, h[c]);
    }
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
        const long long col = (long long)(c * TPR + t) * 8;
        const int n = (int)min(8LL, max(0LL, p.cols - col));
        if (p.hidden && n > 0) store8(p.hidden, DT, row * p.ldh + col, n, h[c]);
#pragma unroll
        for (int i = 0; i < 8; ++i) sum += (double)h[c][i] * (double)h[c][i];
    }
    sum = row_sum<TPR>(sum);
    const Root root = root_of_mean(sum, p.cols, p.eps);
    if (p.rstd && t == 0) p.rstd[row] = root.rounded;
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
        const long long col = (long long)(c * TPR + t) * 8;
        const int n = (int)min(8LL, max(0LL, p.cols - col));
        out8(p, row, col, n, root, h[c]);
    }
}

// Rows of any length, a workgroup a row, read twice.
template <int DT>
__global__ __launch_bounds__(kNT) void rms_norm_long_kernel(const RmsNormParams p, unsigned first)
{
    const long long row = (long long)first + blockIdx.x;
    double sum = 0;
    for (long long at = 0; at < p.cols; at += kNT * 8) {
        const long long col = at + threadIdx.x * 8;
        const int n = (int)min(8LL, max(0LL, p.cols - col));
        float h[8];
        sum8<DT>(p, row, col, n, h);
        if (p.hidden && n > 0) store8(p.hidden, DT, row * p.ldh + col, n, h);
#pragma unroll
        for (int i = 0; i < 8; ++i) sum += (double)h[i] * (double)h[i];
    }
    sum = row_sum<kNT>(sum);
    const Root root = root_of_mean(sum, p.cols, p.eps);
    if (p.rstd && threadIdx.x == 0) p.rstd[row] = root.rounded;
    // each thread's own stores of the hidden state, or x itself, which is not written then
    for (long long at = 0; at < p.cols; at += kNT * 8) {
        const long long col = at + threadIdx.x * 8;
        const int n = (int)min(8LL, max(0LL, p.cols - col));
        float h[8];
        if (p.hidden)
            load8(p.hidden, DT, row * p.ldh + col, n, h);
        else
            load8(p.x, DT, row * p.ldx + col, n, h);
        out8(p, row, col, n, root, h);
    }
}

// f(threads a row, chunks a thread) for rows of `cols` elements: one chunk, or two, four of 8 elements in as
// many threads as that takes, so that a CU has many rows on their way; with many rows a wave to a row of up to
// two. Measured, us for 8192 x 4096 bf16 with the residual and 8-bit output: a wave a row (8 chunks) 66.2, 256 threads (2) 43.9,
// 512 (1) 45.6; its gradients 63.2, 48.9, 47.7. 4096 x 8192: 256 threads (4) 49.4, 512 (2) 44.6; gradients 49.7, 48.7.
template <typename F>
void by_length(long long rows, long long cols, F f)
{
    using std::integral_constant;
    const long long chunks = (cols + 511) / 512;     // of a wave
    if (chunks == 1)
        f(integral_constant<int, 64>{}, integral_constant<int, 1>{});
    else if (chunks == 2 && rows >= 1024)
        f(integral_constant<int, 64>{}, integral_constant<int, 2>{});
    else if (chunks <= 4)
        f(integral_constant<int, 256>{}, integral_constant<int, 1>{});
    else if (chunks <= 8)
        f(integral_constant<int, 512>{}, integral_constant<int, 1>{});
    else if (chunks <= 16)
        f(integral_constant<int, 512>{}, integral_constant<int, 2>{});
    else
        f(integral_constant<int, 1024>{}, integral_constant<int, 2>{});
}
template <int DT>
hipError_t launch_norm(const RmsNormParams &p, hipStream_t stream)
{
    if (p.cols > kNormHeld)
        return launch_groups256(p.rows, [&](unsigned first, unsigned grid) {
            rms_norm_long_kernel<DT><<<grid, kNT, 0, stream>>>(p, first);
        });
    hipError_t e = hipSuccess;
    by_length(p.rows, p.cols, [&](auto tpr, auto nch) {
        constexpr int TPR = decltype(tpr)::value, NCH = decltype(nch)::value, RPW = kBlock<TPR> / TPR;
        const long long groups = (p.rows + RPW - 1) / RPW, most = kMaxGroups256 / (kBlock<TPR> / 256);
        for (long long first = 0; first < groups && e == hipSuccess; first += most) {
            rms_norm_kernel<DT, TPR, NCH><<<(unsigned)std::min(most, groups - first), kBlock<TPR>, 0, stream>>>(p, (unsigned)first);
            e = hipGetLastError();
        }
    });
    return e;
}

// ------------------------------------------------------------ gradients

// Most workgroups whose sums of dw a second launch adds up. 8192 x 4096 bf16: 128 67.7 us, 192 53.1, 256 47.7, 512
// 50.6; 1000 x 2049 fp32: 13.8, 13.4, 12.4, 14.9.
constexpr int kGradGroups = 256;

// The rows of a workgroup follow one another by the grid's size, so that each has its sums
// of dw in registers; the sums of a workgroup's waves meet in LDS. The next row is loaded before this one's sum.
// Bound by HBM: 8192 x 4096 bf16 with the residual 42 to 46 us by the card, its 273 MB, three quarters of them read, at 5.9
// to 6.5 TB/s; with the launch that sums dw 46.7 to 47.7.
template <int DT, int YT, int TPR, int NCH, int HOW>
__device__ __forceinline__ void grad_rows(const RmsNormGradParams &p)
{
    constexpr int RPW = kBlock<TPR> / TPR;
    // 1024 threads have no room for the weight and a row ahead (16384 columns: 128 registers a thread)
    constexpr bool HELD = TPR < 1024, AHEAD = TPR < 1024;
    const int t = threadIdx.x % TPR, sub = threadIdx.x / TPR;
    const long long step = (long long)gridDim.x * RPW;
    const auto weight = [&](long long col, int n, float (&w)[8]) __attribute__((always_inline)) {
        if (p.w_dt == kF32)
            load8_row<kF32, HOW>(p.weight, col, p.cols, n, w);
        else
            load8_row<kBF16, HOW>(p.weight, col, p.cols, n, w);
    };
    float dw[NCH][8], held[NCH][8];
    int n[NCH];
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
        const long long col = (long long)(c * TPR + t) * 8;
        n[c] = (int)min(8LL, max(0LL, p.cols - col));
        if (HELD) weight(col, n[c], held[c]);
#pragma unroll
        for (int i = 0; i < 8; ++i) dw[c][i] = 0;
    }
    Raw<YT> y[NCH];
    Raw<DT> h[NCH], r[NCH];
    float rstd = 0;
    auto load = [&](long long row) __attribute__((always_inline)) {
        rstd = p.rstd[row];
#pragma unroll
        for (int c = 0; c < NCH; ++c) {
            const long long col = (long long)(c * TPR + t) * 8;
            y[c] = load_row<YT, HOW>(p.dy, row * p.lddy, col, p.cols);
            h[c] = load_row<DT, HOW>(p.hidden, row * p.ldh, col, p.cols);
            if (p.dresidual) r[c] = load_row<DT, HOW>(p.dresidual, row * p.lddr, col, p.cols);
        }
    };
    long long row = (long long)blockIdx.x * RPW + sub;
    if (AHEAD && row < p.rows) load(row);
    // a wave with a row of its own goes through its rows alone
    for (int set = 0; row < p.rows; row += step, set ^= 1) {
        float g[NCH][8], u[NCH][8], dot = 0;
        Raw<DT> more[NCH];
        if (!AHEAD) load(row);
        const float s = rstd;
#pragma unroll
        for (int c = 0; c < NCH; ++c) {
            float part = 0, w[8];
            settle<YT>(y[c], n[c]);
            settle<DT>(h[c], n[c]);
            if (p.dresidual) settle<DT>(r[c], n[c]);
            if (!HELD) weight((long long)(c * TPR + t) * 8, n[c], w);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float dy = value<YT>(y[c], i);
                u[c][i] = value<DT>(h[c], i) * s;
                dw[c][i] += dy * u[c][i];
                g[c][i] = dy * (HELD ? held[c][i] : w[i]);
                part += g[c][i] * u[c][i];
            }
            dot += part;
            more[c] = r[c];
        }
        if (AHEAD && row + step < p.rows) load(row + step);
        dot = row_sum<TPR>(dot, set) / (float)p.cols;
#pragma unroll
        for (int c = 0; c < NCH; ++c) {
            const long long col = (long long)(c * TPR + t) * 8;
            float d[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) d[i] = s * (g[c][i] - u[c][i] * dot);
            if (p.dresidual) {
#pragma unroll
                for (int i = 0; i < 8; ++i) d[i] += value<DT>(more[c], i);
            }
            if (n[c] > 0) store8(p.dx, DT, row * p.lddx + col, n[c], d);
        }
    }
    if (!p.dweight) return;
    if constexpr (RPW > 1) {
        __shared__ float sums[RPW - 1][NCH * TPR * 8];
        if (sub > 0) {
#pragma unroll
            for (int c = 0; c < NCH; ++c)
#pragma unroll
                for (int i = 0; i < 8; ++i) sums[sub - 1][(c * 8 + i) * TPR + t] = dw[c][i];
        }
        __syncthreads();
        if (sub > 0) return;
#pragma unroll
        for (int c = 0; c < NCH; ++c)
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
                for (int s = 0; s < RPW - 1; ++s) dw[c][i] += sums[s][(c * 8 + i) * TPR + t];
    }
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
        const long long col = (long long)(c * TPR + t) * 8;
        if (n[c] > 0) store8((char *)p.partial, kF32, blockIdx.x * p.cols + col, n[c], dw[c]);
    }
}

template <int DT, int YT, int TPR, int NCH, bool ONCE>
__global__ __launch_bounds__(kBlock<TPR>) void rms_norm_grad_kernel(const RmsNormGradParams p)
{
    grad_rows<DT, YT, TPR, NCH, ONCE ? kOnce : kOrdinary>(p);
}
// Rows of fewer than 8 elements, which have no last 8 to load. One lane of a wave works, and loads element by element:
// 100000 x 7 bf16 245 to 249 us, 100000 x 100 68.
template <int DT, int YT>
__global__ __launch_bounds__(kNT) void rms_norm_grad_short_kernel(const RmsNormGradParams p)
{
    grad_rows<DT, YT, 64, 1, kUnder8>(p);
}

// dweight[c] = the sum of `parts` rows of partial sums: 64 columns a workgroup, its 16 waves every 16th row, 8
// loads on their way at once
constexpr int kSumWaves = 16;
__global__ __launch_bounds__(64 * kSumWaves) void rms_norm_dweight_kernel(const RmsNormGradParams p, int parts)
{
    __shared__ float part[kSumWaves][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const long long col = min(blockIdx.x * 64LL + lane, p.cols - 1);
    const float *from = p.partial + col;
    float s = 0;
    for (int r0 = wave; r0 < parts; r0 += 8 * kSumWaves) {
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = from[min(r0 + i * kSumWaves, parts - 1) * p.cols];
#pragma unroll
        for (int i = 0; i < 8; ++i) s += r0 + i * kSumWaves < parts ? v[i] : 0.0f;
    }
    part[wave][lane] = s;
    __syncthreads();
    if (wave > 0 || blockIdx.x * 64LL + lane >= p.cols) return;
#pragma unroll
    for (int i = 1; i < kSumWaves; ++i) s += part[i][lane];
    p.dweight[col] = p.accumulate ? p.dweight[col] + s : s;
}

// Rows of any length: the dot products first, a workgroup a row, then 2048 columns of every
// grid.y'th row a workgroup.
template <int DT>
__global__ __launch_bounds__(kNT) void rms_norm_dot_kernel(const RmsNormGradParams p, float *dots, unsigned first)
{
    const long long row = (long long)first + blockIdx.x;
    const float rstd = p.rstd[row];
    float dot = 0;
    for (long long at = 0; at < p.cols; at += kNT * 8) {
        const long long col = at + threadIdx.x * 8;
        const int n = (int)min(8LL, max(0LL, p.cols - col));
        float g[8], u[8], w[8], part = 0;
        load8(p.dy, p.dy_dt, row * p.lddy + col, n, g);
        load8(p.hidden, DT, row * p.ldh + col, n, u);
        load8(p.weight, p.w_dt, col, n, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) part += g[i] * w[i] * (u[i] * rstd);
        dot += part;
    }
    dot = row_sum<kNT>(dot) / (float)p.cols;
    if (threadIdx.x == 0) dots[row] = dot;
}
template <int DT>
__global__ __launch_bounds__(kNT) void rms_norm_grad_long_kernel(const RmsNormGradParams p, const float *dots, int pieces, int parts)
{
    const int piece = blockIdx.x % pieces, part = blockIdx.x / pieces;
    const long long col = piece * (long long)(kNT * 8) + threadIdx.x * 8;
    const int n = (int)min(8LL, max(0LL, p.cols - col));
    if (n <= 0) return;
    float w[8], dw[8] = {};
    load8(p.weight, p.w_dt, col, n, w);
    for (long long row = part; row < p.rows; row += parts) {
        const float rstd = p.rstd[row], dot = dots[row];
        float g[8], u[8], d[8];
        load8(p.dy, p.dy_dt, row * p.lddy + col, n, g);
        load8(p.hidden, DT, row * p.ldh + col, n, u);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            u[i] *= rstd;
            dw[i] += g[i] * u[i];
            d[i] = rstd * (g[i] * w[i] - u[i] * dot);
        }
        if (p.dresidual) {
            float r[8];
            load8(p.dresidual, DT, row * p.lddr + col, n, r);
#pragma unroll
            for (int i = 0; i < 8; ++i) d[i] += r[i];
        }
        store8(p.dx, DT, row * p.lddx + col, n, d);
    }
    if (p.dweight) store8((char *)p.partial, kF32, part * p.cols + col, n, dw);
}

bool held(long long cols) { return cols <= kNormHeld; }
// rows of partial sums of dw
int grad_parts(long long rows, long long cols)
{
    if (!held(cols)) return (int)std::min<long long>(rows, 64);
    int parts = 0;
    by_length(rows, cols, [&](auto tpr, auto) {
        constexpr int TPR = decltype(tpr)::value, RPW = kBlock<TPR> / TPR;
        parts = (int)std::min<long long>(kGradGroups, (rows + RPW - 1) / RPW);
    });
    return parts;
}

// From 128 MiB on, rows of more than a wave are read nontemporal, so that they do not push one another out of the 256
// MiB cache behind the L2s; with rows loaded whole that gives 1% (nontemporal against ordinary, with the residual, in turn
// with others: 8192 x 4096 bf16, 192 MiB, 47.5 us against 48.1, fp32 96.9 against 98.6; 2048 x 4096 bf16, 48 MiB, 17.8 against
// 16.3). Rows of a wave, 65536 x 512: bf16 59.7 against 60.3, fp32 105 against 95.
template <int DT, int YT>
hipError_t launch_grad(const RmsNormGradParams &p, hipStream_t stream)
{
    const bool once = p.rows * p.cols * ((YT == kF32 ? 4 : 2) + (DT == kF32 ? 4 : 2) * (p.dresidual ? 2 : 1)) >= 128LL << 20;
    const int parts = grad_parts(p.rows, p.cols);
    if (p.rows == 0) {
        // dw is the sum of nothing
    } else if (p.cols < 8) {                         // parts are those of a wave a row
        rms_norm_grad_short_kernel<DT, YT><<<parts, kNT, 0, stream>>>(p);
    } else if (held(p.cols)) {
        by_length(p.rows, p.cols, [&](auto tpr, auto nch) {
            constexpr int TPR = decltype(tpr)::value, NCH = decltype(nch)::value;
            if (once && TPR > 64)
                rms_norm_grad_kernel<DT, YT, TPR, NCH, (TPR > 64)><<<parts, kBlock<TPR>, 0, stream>>>(p);
            else
                rms_norm_grad_kernel<DT, YT, TPR, NCH, false><<<parts, kBlock<TPR>, 0, stream>>>(p);
        });
    } else {
        float *dots = p.partial + (p.dweight ? parts * p.cols : 0);
        const hipError_t e = launch_groups256(p.rows, [&](unsigned first, unsigned grid) {
            rms_norm_dot_kernel<DT><<<grid, kNT, 0, stream>>>(p, dots, first);
        });
        if (e != hipSuccess) return e;
        const int pieces = (int)((p.cols + kNT * 8 - 1) / (kNT * 8));
        rms_norm_grad_long_kernel<DT><<<pieces * parts, kNT, 0, stream>>>(p, dots, pieces, parts);
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || !p.dweight) return e;
    rms_norm_dweight_kernel<<<(unsigned)((p.cols + 63) / 64), 64 * kSumWaves, 0, stream>>>(p, parts);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_rms_norm(const RmsNormParams &p, int dt, hipStream_t stream)
{
    return dt == kBF16 ? launch_norm<kBF16>(p, stream) : launch_norm<kF32>(p, stream);
}

size_t rms_norm_grad_ws(long long rows, long long cols, bool dweight)
{
    return (dweight ? (size_t)grad_parts(rows, cols) * cols * 4 : 0) + (held(cols) ? 0 : (size_t)rows * 4);
}

hipError_t launch_rms_norm_grad(const RmsNormGradParams &p, int dt, hipStream_t stream)
{
    if (dt == kBF16) return p.dy_dt == kBF16 ? launch_grad<kBF16, kBF16>(p, stream) : launch_grad<kBF16, kF32>(p, stream);
    return p.dy_dt == kBF16 ? launch_grad<kF32, kBF16>(p, stream) : launch_grad<kF32, kF32>(p, stream);
}

}  // namespace dps
