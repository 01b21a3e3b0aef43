// The optimizer step of a sharded data-parallel update on gfx950: the global
// gradient norm, and AdamW over many tensors in one launch, with the moments in
// fp32 or in 8 bits.
//
// Both walk a list of tensors held in the kernel's arguments, cut into chunks
// of a fixed number of elements; a workgroup takes chunks blockIdx.x,
// blockIdx.x + gridDim.x, ... of all tensors in order. Every load and store of
// a full chunk is as wide as its type allows whatever the tensor's alignment
// (gfx950 takes global accesses of any alignment), so a shard that starts at an
// odd element runs the same code as an aligned one.
#include "optim_internal.h"

#pragma clang fp contract(off)

namespace dps {
namespace {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
// the same with the alignment of one element
typedef float f32x4_e __attribute__((ext_vector_type(4), aligned(4)));
typedef unsigned int u32x4_e __attribute__((ext_vector_type(4), aligned(2)));
typedef unsigned int u32x2_e __attribute__((ext_vector_type(2), aligned(2)));
typedef unsigned int u32_e __attribute__((aligned(1)));

constexpr int kNT = 256;

__device__ __forceinline__ float bf16_at(const char *p, long long i)
{
    return __uint_as_float((unsigned)reinterpret_cast<const unsigned short *>(p)[i] << 16);
}

// ------------------------------------------------------------- gradient norm

// Squares are summed in fp64: v_fma_f64 runs at the rate of an fp32 FMA here,
// so 64 bits cost nothing beside the loads, no square of a finite fp32 gradient
// overflows, and 10^9 terms lose nothing. Each thread holds four sums; a
// workgroup's sum is a fixed tree over its threads, and the last workgroup to
// finish adds the partials in a fixed order: the same bits in every run.
constexpr int kNormChunk = 8192;

template <int DT>
__device__ __forceinline__ void norm_chunk(const char *g, long long left, double (&s)[4])
{
    constexpr int V = DT == kBF16 ? 8 : 4;          // elements per 16-byte load
    constexpr int U = kNormChunk / (kNT * V);
    if (left >= kNormChunk) {
        u32x4 w[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            w[u] = *reinterpret_cast<const u32x4_e *>(g + (u * kNT + (int)threadIdx.x) * 16);
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if constexpr (DT == kBF16) {
                    const double a = __uint_as_float(w[u][j] << 16);
                    const double b = __uint_as_float(w[u][j] & 0xffff0000u);
                    s[j] = __builtin_fma(a, a, s[j]);
                    s[j] = __builtin_fma(b, b, s[j]);
                } else {
                    const double a = __uint_as_float(w[u][j]);
                    s[j] = __builtin_fma(a, a, s[j]);
                }
            }
    } else {
        for (int i = threadIdx.x; i < (int)left; i += kNT) {
            const double a = DT == kBF16 ? bf16_at(g, i) : reinterpret_cast<const float *>(g)[i];
            s[0] = __builtin_fma(a, a, s[0]);
        }
    }
}

__device__ __forceinline__ double block_sum(double x, double *lds)
{
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) x += __shfl_xor(x, d);
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = x;
    __syncthreads();
    x = (lds[0] + lds[1]) + (lds[2] + lds[3]);
    __syncthreads();
    return x;
}

template <int DT>
__global__ __launch_bounds__(kNT) void grad_norm_kernel(const NormParams p)
{
    constexpr int ES = DT == kBF16 ? 2 : 4;
    __shared__ double lds[kNT / 64];
    __shared__ int is_last;
    double s[4] = {0.0, 0.0, 0.0, 0.0};
    const int total = p.first[p.nt];
    int t = 0;
    for (int c = blockIdx.x; c < total; c += gridDim.x) {
        while (c >= p.first[t + 1]) ++t;
        const long long at = (long long)(c - p.first[t]) * kNormChunk;
        norm_chunk<DT>(p.g[t] + at * ES, p.n[t] - at, s);
    }
    const double sum = block_sum((s[0] + s[1]) + (s[2] + s[3]), lds);
    if (threadIdx.x == 0) {
        double *mine = p.partial + blockIdx.x;
        const double all = p.add ? *mine + sum : sum;
        if (!p.finish) {
            *mine = all;
        } else {
            __hip_atomic_store(mine, all, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            // the ticket wraps to zero with the last workgroup, ready for the next call
            const unsigned old = __hip_atomic_fetch_add(p.ticket, 1u, __ATOMIC_ACQ_REL,
                                                        __HIP_MEMORY_SCOPE_AGENT);
            is_last = old == gridDim.x - 1;
        }
    }
    if (!p.finish) return;
    __syncthreads();
    if (!is_last) return;
    double x = 0.0;
    for (int i = threadIdx.x; i < (int)gridDim.x; i += kNT)
        x += __hip_atomic_load(p.partial + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    x = block_sum(x, lds);
    if (threadIdx.x == 0) {
        const double norm = sqrt(x);
        const float nf = (float)norm;
        const bool fine = nf < __builtin_inff();      // false for NaN too
        p.ctrl->norm = nf;
        p.ctrl->scale = !fine ? 0.0f
                        : p.max_norm > 0.0f && norm > (double)p.max_norm ? (float)((double)p.max_norm / norm)
                                                                         : 1.0f;
        if (fine)
            p.ctrl->step += 1;
        else
            p.ctrl->skipped += 1;
        *p.ticket = 0;
    }
}

// --------------------------------------------------------------------- AdamW

// g = scale g;  m = b1 m + (1 - b1) g;  v = b2 v + (1 - b2) g^2;
// p = p (1 - lr wd) - lr / (1 - b1^t) * m / (sqrt(v) / sqrt(1 - b2^t) + eps)
// in fp32 with every operation rounded as written. A thread holds 4 consecutive
// elements per group, so each fp32 access is 16 bytes a lane and a wave covers
// 1 KiB of it.
//
// 8-bit moments: blocks of 128 elements share two fp32 scales. m is held in
// e4m3 as m / (max|m| / 448), and v as its root r = sqrt(v) in e4m3 over
// max r / 448: the root halves v's range in octaves, and the update needs r and
// not v. A positive r is never rounded to zero but up to the smallest code: a
// lost r would leave m over eps, a step of any size, where a raised r only
// makes the step smaller. The update itself uses the new m and r before they
// are rounded. Rounding is to nearest, or at random in proportion to the
// remainder: with b2 near 1 a moment changes by less than half a code per
// step, and to nearest it would stand still relative to its block. 32 lanes of
// a wave hold one block, so the two maxima are register exchanges.
constexpr int kAdamU = 2;                        // groups of 4 elements per thread and chunk
constexpr int kAdamChunk = kNT * 4 * kAdamU;

// largest x (>= 0; a NaN is passed over) of each half of the wave, in all its lanes
__device__ __forceinline__ float half_wave_max(float x)
{
#define DPS_ROR(n)                                                                           \
    x = fmaxf(x, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x120 + n, \
                                                            0xf, 0xf, false)))
    DPS_ROR(8);
    DPS_ROR(4);
    DPS_ROR(2);
    DPS_ROR(1);
#undef DPS_ROR
    const auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return fmaxf(__uint_as_float(s[0]), __uint_as_float(s[1]));
}

// SplitMix64's output function
__device__ __forceinline__ unsigned long long mix64(unsigned long long z)
{
    z = (z ^ (z >> 30)) * 0xBF58476D1CE4E5B9ull;
    z = (z ^ (z >> 27)) * 0x94D049BB133111EBull;
    return z ^ (z >> 31);
}
constexpr unsigned long long kGolden = 0x9E3779B97F4A7C15ull;

// y in [-448, 448] to a value of e4m3, away from zero where the 16 random bits
// reach the remainder: floor(|y| / u + r / 2^16) u with u the step of y's octave
__device__ __forceinline__ float e4m3_stochastic(float y, unsigned r16)
{
    const float a = fabsf(y);
    const unsigned e = max(__float_as_uint(a) >> 23, 121u);      // the lowest octave is 2^-6
    const float up = __uint_as_float((257u - e) << 23), down = __uint_as_float((e - 3u) << 23);
    const float q = floorf(a * up + (float)r16 * 0x1p-16f) * down;
    return copysignf(q > 448.0f ? 448.0f : q, y);                // keeps a NaN
}

__device__ __forceinline__ unsigned pack_e4m3(const float (&x)[4])
{
    const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(x[0], x[1], 0, false);
    return (unsigned)__builtin_amdgcn_cvt_pk_fp8_f32(x[2], x[3], lo, true);
}

__device__ __forceinline__ void unpack_e4m3(unsigned w, float (&x)[4])
{
    const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false);
    const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
    x[0] = lo[0];
    x[1] = lo[1];
    x[2] = hi[0];
    x[3] = hi[1];
}

__device__ __forceinline__ double power(double b, long long t)
{
    double r = 1.0;
    for (; t > 0; t >>= 1) {
        if (t & 1) r *= b;
        b *= b;
    }
    return r;
}

// n (1..4) elements at p[e]; FULL: all four, in one access
template <int DT, bool FULL>
__device__ __forceinline__ void load4(const char *p, long long e, int n, float (&x)[4])
{
    if constexpr (FULL && DT == kF32) {
        const f32x4 w = *reinterpret_cast<const f32x4_e *>(p + 4 * e);
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = w[i];
    } else if constexpr (FULL) {
        const u32x2 w = *reinterpret_cast<const u32x2_e *>(p + 2 * e);
        x[0] = __uint_as_float(w[0] << 16);
        x[1] = __uint_as_float(w[0] & 0xffff0000u);
        x[2] = __uint_as_float(w[1] << 16);
        x[3] = __uint_as_float(w[1] & 0xffff0000u);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            x[i] = i >= n ? 0.0f : DT == kF32 ? reinterpret_cast<const float *>(p)[e + i] : bf16_at(p, e + i);
    }
}

template <int DT, bool FULL>
__device__ __forceinline__ void store4(char *p, long long e, int n, const float (&x)[4])
{
    if constexpr (DT == kF32) {
        if constexpr (FULL) {
            *reinterpret_cast<f32x4_e *>(p + 4 * e) = f32x4{x[0], x[1], x[2], x[3]};
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (i < n) reinterpret_cast<float *>(p)[e + i] = x[i];
        }
    } else {
        const f32x2 a = {x[0], x[1]}, b = {x[2], x[3]};
        const u32x2 w = {__builtin_bit_cast(unsigned, __builtin_convertvector(a, bf16x2)),
                         __builtin_bit_cast(unsigned, __builtin_convertvector(b, bf16x2))};
        if constexpr (FULL) {
            *reinterpret_cast<u32x2_e *>(p + 2 * e) = w;
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (i < n)
                    reinterpret_cast<unsigned short *>(p)[e + i] = (unsigned short)(w[i >> 1] >> (16 * (i & 1)));
        }
    }
}

template <bool FULL>
__device__ __forceinline__ unsigned load_codes(const char *p, long long e, int n)
{
    if constexpr (FULL) return *reinterpret_cast<const u32_e *>(p + e);
    unsigned w = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (i < n) w |= (unsigned)(unsigned char)p[e + i] << (8 * i);
    return w;
}

template <bool FULL>
__device__ __forceinline__ void store_codes(char *p, long long e, int n, unsigned w)
{
    if constexpr (FULL) {
        *reinterpret_cast<u32_e *>(p + e) = w;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < n) p[e + i] = (char)(w >> (8 * i));
    }
}

struct Scalars {
    float clip, step_size, inv_sqrt_bc2;
};

// kAdamU groups of 4 elements per thread from element `at` of tensor t
template <int PT, int GT, bool S8, bool SR, bool FULL>
__device__ __forceinline__ void adam_chunk(const AdamParams &k, const AdamTensor &t, long long at,
                                           const Scalars &c, unsigned long long key)
{
    float p[kAdamU][4], g[kAdamU][4], m[kAdamU][4], v[kAdamU][4];
    unsigned mw[kAdamU], vw[kAdamU];
    f32x2 sc[kAdamU];
    long long e[kAdamU];
    int n[kAdamU];
#pragma unroll
    for (int u = 0; u < kAdamU; ++u) {
        e[u] = at + (u * kNT + (int)threadIdx.x) * 4;
        n[u] = FULL ? 4 : (int)max(0LL, min(4LL, t.n - e[u]));
        load4<GT, FULL>(t.g, e[u], n[u], g[u]);
        load4<PT, FULL>(t.p, e[u], n[u], p[u]);
        if constexpr (S8) {
            mw[u] = load_codes<FULL>(t.m, e[u], n[u]);
            vw[u] = load_codes<FULL>(t.v, e[u], n[u]);
            sc[u] = n[u] > 0 ? reinterpret_cast<const f32x2 *>(t.scales)[e[u] / kStateBlock] : f32x2{0.0f, 0.0f};
        } else {
            load4<kF32, FULL>(t.m, e[u], n[u], m[u]);
            load4<kF32, FULL>(t.v, e[u], n[u], v[u]);
        }
    }
#pragma unroll
    for (int u = 0; u < kAdamU; ++u) {
        float r[4], top_m = 0.0f, top_r = 0.0f;
        if constexpr (S8) {
            unpack_e4m3(mw[u], m[u]);
            unpack_e4m3(vw[u], v[u]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                m[u][i] = m[u][i] * sc[u][0];
                v[u][i] = v[u][i] * sc[u][1];
                v[u][i] = v[u][i] * v[u][i];
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float gi = g[u][i] * c.clip;
            m[u][i] = m[u][i] * k.beta1 + gi * k.one_minus_beta1;
            v[u][i] = v[u][i] * k.beta2 + (gi * gi) * k.one_minus_beta2;
            r[i] = sqrtf(v[u][i]);
            p[u][i] = p[u][i] * k.decay - m[u][i] / (r[i] * c.inv_sqrt_bc2 + k.eps) * c.step_size;
            if constexpr (S8) {
                top_m = fmaxf(top_m, fabsf(m[u][i]));
                top_r = fmaxf(top_r, r[i]);
            }
        }
        store4<PT, FULL>(t.p, e[u], n[u], p[u]);
        if (t.copy) store4<kBF16, FULL>(t.copy, e[u], n[u], p[u]);
        if constexpr (S8) {
            top_m = half_wave_max(top_m);
            top_r = half_wave_max(top_r);
            // a block with nothing above 2^-100 is held as zeros: its
            // reciprocal scale could overflow
            const bool use_m = top_m >= 0x1p-100f, use_r = top_r >= 0x1p-100f;
            const float inv_m = use_m ? 1.0f / top_m * 448.0f : 0.0f, inv_r = use_r ? 1.0f / top_r * 448.0f : 0.0f;
            unsigned long long z[2];
            if constexpr (SR) {
                const unsigned long long pair = (unsigned long long)(e[u] >> 1) + 1;
                z[0] = mix64(key + pair * kGolden);
                z[1] = mix64(key + (pair + 1) * kGolden);
            }
            float ym[4], yr[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                ym[i] = m[u][i] * inv_m;
                yr[i] = r[i] * inv_r;
                if (yr[i] > 0.0f) yr[i] = fmaxf(yr[i], 0x1p-9f);
                if constexpr (SR) {
                    const unsigned half = (unsigned)(z[i >> 1] >> (32 * (i & 1)));
                    ym[i] = e4m3_stochastic(ym[i], half & 0xffffu);
                    yr[i] = e4m3_stochastic(yr[i], half >> 16);
                }
            }
            store_codes<FULL>(t.m, e[u], n[u], pack_e4m3(ym));
            store_codes<FULL>(t.v, e[u], n[u], pack_e4m3(yr));
            if ((threadIdx.x & 31) == 0 && n[u] > 0)
                reinterpret_cast<f32x2 *>(t.scales)[e[u] / kStateBlock] =
                    f32x2{use_m ? top_m * (1.0f / 448.0f) : 0.0f, use_r ? top_r * (1.0f / 448.0f) : 0.0f};
        } else {
            store4<kF32, FULL>(t.m, e[u], n[u], m[u]);
            store4<kF32, FULL>(t.v, e[u], n[u], v[u]);
        }
    }
}

template <int PT, int GT, bool S8, bool SR>
__global__ __launch_bounds__(kNT) void adamw_kernel(const AdamParams k)
{
    Scalars c = {1.0f, k.step_size, k.inv_sqrt_bc2};
    long long step = k.step;
    if (k.ctrl) {
        c.clip = k.ctrl->scale;
        if (c.clip == 0.0f) return;                   // the gradient's norm is not finite
        if (step == 0) {
            step = max(1, k.ctrl->step);
            c.step_size = (float)(k.lr / (1.0 - power(k.dbeta1, step)));
            c.inv_sqrt_bc2 = (float)(1.0 / sqrt(1.0 - power(k.dbeta2, step)));
        }
    }
    unsigned long long key = 0;
    if constexpr (SR) key = mix64(k.seed + (unsigned long long)step * kGolden);
    const int total = k.first[k.nt];
    int t = 0;
    for (int b = blockIdx.x; b < total; b += gridDim.x) {
        while (b >= k.first[t + 1]) ++t;
        const long long at = (long long)(b - k.first[t]) * kAdamChunk;
        unsigned long long tkey = 0;
        if constexpr (SR) tkey = mix64(key + (unsigned long long)(k.index0 + t + 1) * kGolden);
        if (at + kAdamChunk <= k.t[t].n)
            adam_chunk<PT, GT, S8, SR, true>(k, k.t[t], at, c, tkey);
        else
            adam_chunk<PT, GT, S8, SR, false>(k, k.t[t], at, c, tkey);
    }
}

template <int PT, int GT>
hipError_t launch_adamw_typed(const AdamParams &p, bool eight, bool stochastic, hipStream_t stream)
{
    const int grid = min(p.first[p.nt], 2048);
    if (!eight)
        adamw_kernel<PT, GT, false, false><<<grid, kNT, 0, stream>>>(p);
    else if (!stochastic)
        adamw_kernel<PT, GT, true, false><<<grid, kNT, 0, stream>>>(p);
    else
        adamw_kernel<PT, GT, true, true><<<grid, kNT, 0, stream>>>(p);
    return hipGetLastError();
}

}  // namespace

long long norm_chunks(long long n) { return (n + kNormChunk - 1) / kNormChunk; }
long long adam_chunks(long long n) { return (n + kAdamChunk - 1) / kAdamChunk; }

hipError_t launch_grad_norm(const NormParams &p, int dt, int grid, hipStream_t stream)
{
    if (dt == kBF16)
        grad_norm_kernel<kBF16><<<grid, kNT, 0, stream>>>(p);
    else
        grad_norm_kernel<kF32><<<grid, kNT, 0, stream>>>(p);
    return hipGetLastError();
}

hipError_t launch_adamw(const AdamParams &p, int p_dt, int g_dt, bool eight, bool stochastic,
                        hipStream_t stream)
{
    if (p_dt == kF32)
        return g_dt == kF32 ? launch_adamw_typed<kF32, kF32>(p, eight, stochastic, stream)
                            : launch_adamw_typed<kF32, kBF16>(p, eight, stochastic, stream);
    return g_dt == kF32 ? launch_adamw_typed<kBF16, kF32>(p, eight, stochastic, stream)
                        : launch_adamw_typed<kBF16, kBF16>(p, eight, stochastic, stream);
}

}  // namespace dps
