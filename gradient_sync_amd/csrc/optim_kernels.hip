// The optimizer step of a sharded data-parallel update on gfx950: the global
// gradient norm, and AdamW over many tensors in one launch, with the moments in
// fp32 or in 8 bits.
//
// Both walk a list of tensors held in the kernel's arguments, cut into chunks
// of a fixed number of elements; a workgroup takes chunks blockIdx.x,
// blockIdx.x + gridDim.x, ... of all tensors in order (the norm), or one chunk
// (AdamW). Every load and store of
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

// Everything here is read once and written once per step: nontemporal, whatever
// the alignment (the norm of 200M fp32 values: 117 us in place of 131; AdamW with
// fp32 states and a copy, 200M elements 953 for 1035, 40M 187 for 209, up to 4M the
// same. Steps of 7M to 20M elements one after the other, whose tensors then stay in
// the 256 MB Infinity Cache, are 5 to 11% slower for it, 14M 66 us for 59: between the
// steps of a training run its other work passes through that cache).
#define DPS_ONCE(V)                                                                          \
    __device__ __forceinline__ V load_once(const V *p) { return __builtin_nontemporal_load(p); } \
    __device__ __forceinline__ void store_once(V *p, V v) { __builtin_nontemporal_store(v, p); }
DPS_ONCE(f32x4_e)
DPS_ONCE(u32x4_e)
DPS_ONCE(u32x2_e)
DPS_ONCE(u32_e)
#undef DPS_ONCE

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
// Bound by reading the gradients: 200M bf16 values in 62 us (6.45 TB/s), 200M fp32
// ones in 117 (6.8 TB/s), 10M fp32 ones in 12.3 (3.3 TB/s: the launch, the finish, and
// 1,224 chunks over 512 workgroups, three for some and two for others).
constexpr int kNormChunk = 8192;

template <int DT>
__device__ __forceinline__ void add_squares(u32x4 w, double (&s)[4])
{
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if constexpr (DT == kBF16) {
            const double a = __uint_as_float(w[j] << 16), b = __uint_as_float(w[j] & 0xffff0000u);
            s[j] = __builtin_fma(a, a, s[j]);
            s[j] = __builtin_fma(b, b, s[j]);
        } else {
            const double a = __uint_as_float(w[j]);
            s[j] = __builtin_fma(a, a, s[j]);
        }
    }
}

template <int DT>
__device__ __forceinline__ void norm_chunk(const char *g, long long left, double (&s)[4])
{
    constexpr int V = DT == kBF16 ? 8 : 4;          // elements per 16-byte load
    constexpr int U = kNormChunk / (kNT * V);
    if (left >= kNormChunk) {
        u32x4 w[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            w[u] = load_once(reinterpret_cast<const u32x4_e *>(g + (u * kNT + (int)threadIdx.x) * 16));
#pragma unroll
        for (int u = 0; u < U; ++u) add_squares<DT>(w[u], s);
    } else {
        // whole vectors, then the last few elements one a thread
        const int whole = (int)left / V;
        u32x4 w[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int at = u * kNT + (int)threadIdx.x;
            w[u] = at < whole ? load_once(reinterpret_cast<const u32x4_e *>(g + at * 16)) : u32x4_e{};
        }
        const int i = whole * V + (int)threadIdx.x;
        const double a = i >= (int)left ? 0.0 : DT == kBF16 ? bf16_at(g, i) : reinterpret_cast<const float *>(g)[i];
        s[0] = __builtin_fma(a, a, s[0]);
#pragma unroll
        for (int u = 0; u < U; ++u) add_squares<DT>(w[u], s);
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
            // What the workgroups hand over are the partials alone, and each is
            // stored and loaded as a device-wide atomic, past the caches of one
            // XCD. So the ticket has to wait for the store, but need not release:
            // a release writes back, and an acquire drops, the XCD's whole cache,
            // 1,226 times in a norm of 40 MB (39.6 us with, 21.8 without; 512
            // workgroups in place of 1,226 take it to 13).
            __hip_atomic_store(mine, all, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            __builtin_amdgcn_s_waitcnt(0);
            asm volatile("" ::: "memory");
            const unsigned old = __hip_atomic_fetch_add(p.ticket, 1u, __ATOMIC_RELAXED,
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
        // zero is what tells the update to skip: a factor too small for fp32 is its
        // smallest number
        p.ctrl->scale = !fine ? 0.0f
                        : p.max_norm > 0.0 && norm > p.max_norm ? fmaxf((float)(p.max_norm / norm), 0x1p-149f)
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
// p = p (1 - lr wd) - m / (sqrt(v) * (1 / sqrt(1 - b2^t)) + eps) * (lr / (1 - b1^t))
// in fp32 with every operation rounded as written (with 8-bit states the quotient
// is the exception, see there). A thread holds 4 consecutive
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
//
// Bound by HBM: 200M elements in 64 shards (fp32 p, bf16 g and copy) take 981
// us with fp32 states (5.7 TB/s; 976-1037 in one run) and 585-634 with 8-bit ones,
// stochastically rounded (5.1-5.5 TB/s); with bf16 p and g and stochastic rounding the
// vector units bound it, at the clock that power leaves (474-555 us, 3.6-4.3 TB/s;
// to nearest 385). One chunk per workgroup: workgroups that go through several load
// nothing while they compute and store (1245 us against 1005, fp32 states).
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
// reach the remainder: floor(|y| / u + r / 2^16) u with u the step of y's octave.
// e4m3 keeps 3 of fp32's 23 fraction bits, so from its lowest octave up that is
// an addition to the other 20 and a mask; a value below 2^-6 is first moved into
// that octave, where u is the same. 448 has none of those 20 bits, and no more than
// a few of them set for a rounding above it: nothing is carried past 448. A NaN is
// brought to the lowest quiet one first, so that the addition leaves it a NaN.
__device__ __forceinline__ float e4m3_stochastic(float y, unsigned r16)
{
    const float a = fabsf(y), move = a < 0x1p-6f ? 0x1p-6f : 0.0f;
    const unsigned bits = (min(__float_as_uint(a + move), 0x7fc00000u) + (r16 << 4)) & 0xfff00000u;
    return copysignf(__uint_as_float(bits) - move, y);
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

// sqrt(x) rounded to nearest: the hardware's root is off by at most one place, and
// the sign of x - s (s -+ one place) tells. Below 2^-96 that residual would lose
// digits, and the hardware takes a subnormal x for zero (a root of 2^-149 for one
// of 2^-64: a step 2^85 times too long where eps is smaller), so such an x is
// scaled by 2^32 first, its root by 2^-16 (200M elements with stochastically rounded
// 8-bit states: bf16 parameters 463 to 474 us, fp32 ones 541 to 546). Zeros, infinities and NaNs pass through, as their neighbours
// give NaN residuals.
__device__ __forceinline__ float root(float x)
{
    const bool small = x < 0x1p-96f;
    const float y = small ? x * 0x1p32f : x;
    const float s = __builtin_amdgcn_sqrtf(y);
    const float down = __uint_as_float(__float_as_uint(s) - 1u), up = __uint_as_float(__float_as_uint(s) + 1u);
    const float rd = __builtin_fmaf(-down, s, y), ru = __builtin_fmaf(-up, s, y);
    const float t = rd <= 0.0f ? down : s;
    const float r = ru > 0.0f ? up : t;
    return small ? r * 0x1p-16f : r;
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

// 4 elements at p[e] in one access (FULL), or the first n of them and zeros: every
// load of a short chunk is issued, from the tensor's last element where there is
// none, as a load behind a branch would be waited for before the next one
template <int DT, bool FULL>
__device__ __forceinline__ void load4(const char *p, long long e, int n, long long last, float (&x)[4])
{
    if constexpr (FULL && DT == kF32) {
        const f32x4 w = load_once(reinterpret_cast<const f32x4_e *>(p + 4 * e));
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = w[i];
    } else if constexpr (FULL) {
        const u32x2 w = load_once(reinterpret_cast<const u32x2_e *>(p + 2 * e));
        x[0] = __uint_as_float(w[0] << 16);
        x[1] = __uint_as_float(w[0] & 0xffff0000u);
        x[2] = __uint_as_float(w[1] << 16);
        x[3] = __uint_as_float(w[1] & 0xffff0000u);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const long long at = min(e + i, last);
            const float v = DT == kF32 ? reinterpret_cast<const float *>(p)[at] : bf16_at(p, at);
            x[i] = i < n ? v : 0.0f;
        }
    }
}

template <int DT, bool FULL>
__device__ __forceinline__ void store4(char *p, long long e, int n, const float (&x)[4])
{
    if constexpr (DT == kF32) {
        if constexpr (FULL) {
            store_once(reinterpret_cast<f32x4_e *>(p + 4 * e), f32x4_e{x[0], x[1], x[2], x[3]});
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
            store_once(reinterpret_cast<u32x2_e *>(p + 2 * e), u32x2_e(w));
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (i < n)
                    reinterpret_cast<unsigned short *>(p)[e + i] = (unsigned short)(w[i >> 1] >> (16 * (i & 1)));
        }
    }
}

template <bool FULL>
__device__ __forceinline__ unsigned load_codes(const char *p, long long e, int n, long long last)
{
    if constexpr (FULL) return load_once(reinterpret_cast<const u32_e *>(p + e));
    unsigned w = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const unsigned v = (unsigned char)p[min(e + i, last)];
        w |= (i < n ? v : 0u) << (8 * i);
    }
    return w;
}

template <bool FULL>
__device__ __forceinline__ void store_codes(char *p, long long e, int n, unsigned w)
{
    if constexpr (FULL) {
        store_once(reinterpret_cast<u32_e *>(p + e), u32_e(w));
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < n) p[e + i] = (char)(w >> (8 * i));
    }
}

struct Scalars {
    float clip, step_size, inv_sqrt_bc2;
    long long step;
};

// clip = 0: the gradient's norm is not finite, nothing is to change
__device__ __forceinline__ Scalars scalars(const AdamParams &k)
{
    Scalars c = {1.0f, k.step_size, k.inv_sqrt_bc2, k.step};
    if (k.ctrl) {
        c.clip = k.ctrl->scale;
        if (c.step == 0) {
            // as the host does it for a given step, in fp64 and rounded once: even
            // lanes lr / (1 - beta1^t), odd lanes 1 / sqrt(1 - beta2^t)
            c.step = max(1, k.ctrl->step);
            double b1 = k.dbeta1, b2 = k.dbeta2;
#ifdef __HIP_DEVICE_COMPILE__
            asm volatile("" : "+s"(b1), "+s"(b2));    // scalars: chosen by address, they would wait for the loads above
#endif
            const bool odd = threadIdx.x & 1;
            const double left = 1.0 - power(odd ? b2 : b1, c.step);
            const int x = __float_as_int((float)((odd ? 1.0 : k.lr) / (odd ? sqrt(left) : left)));
            c.step_size = __int_as_float(__builtin_amdgcn_readlane(x, 0));
            c.inv_sqrt_bc2 = __int_as_float(__builtin_amdgcn_readlane(x, 1));
        }
    }
    return c;
}

// kAdamU groups of 4 elements per thread from element `at` of tensor t
template <int PT, int GT, bool S8, bool SR, bool FULL>
__device__ __forceinline__ void adam_chunk(const AdamParams &k, const AdamTensor &t, int index, long long at)
{
    float p[kAdamU][4], g[kAdamU][4], m[kAdamU][4], v[kAdamU][4];
    unsigned mw[kAdamU], vw[kAdamU];
    f32x2 sc[kAdamU];
    long long e[kAdamU];
    int n[kAdamU];
    const long long last = t.n - 1;
#pragma unroll
    for (int u = 0; u < kAdamU; ++u) {
        e[u] = at + (u * kNT + (int)threadIdx.x) * 4;
        n[u] = FULL ? 4 : (int)max(0LL, min(4LL, t.n - e[u]));
        load4<GT, FULL>(t.g, e[u], n[u], last, g[u]);
        load4<PT, FULL>(t.p, e[u], n[u], last, p[u]);
        if constexpr (S8) {
            mw[u] = load_codes<FULL>(t.m, e[u], n[u], last);
            vw[u] = load_codes<FULL>(t.v, e[u], n[u], last);
            sc[u] = reinterpret_cast<const f32x2 *>(t.scales)[min(e[u], last) / kStateBlock];
        } else {
            load4<kF32, FULL>(t.m, e[u], n[u], last, m[u]);
            load4<kF32, FULL>(t.v, e[u], n[u], last, v[u]);
        }
    }
    // after the loads have been issued: they take longer than this
    const Scalars c = scalars(k);
    if (c.clip == 0.0f) return;
    float r[kAdamU][4], top[kAdamU][2];
#pragma unroll
    for (int u = 0; u < kAdamU; ++u) {
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
        top[u][0] = top[u][1] = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float gi = g[u][i] * c.clip;
            m[u][i] = m[u][i] * k.beta1 + gi * k.one_minus_beta1;
            v[u][i] = v[u][i] * k.beta2 + (gi * gi) * k.one_minus_beta2;
            r[u][i] = root(v[u][i]);
            // A denominator below the normal numbers counts as 2^-126 (its quotient
            // could overflow); a maximum would pass a NaN over, and take a step over
            // 2^-126 in its place.
            float den = r[u][i] * c.inv_sqrt_bc2 + k.eps;
            den = den < 0x1p-126f ? 0x1p-126f : den;
            // With fp32 states the quotient is rounded as written (200M elements: 925
            // us, with a reciprocal 954). With 8-bit ones it is a product with the
            // hardware's reciprocal, 2 places off at most: the m and r that enter
            // hold 4 bits, and a division costs where the vector units bound it
            // (200M elements, bf16 parameters: 511 us for 480).
            float quotient;
            if constexpr (S8)
                quotient = m[u][i] * __builtin_amdgcn_rcpf(den);
            else
                quotient = m[u][i] / den;
            p[u][i] = p[u][i] * k.decay - quotient * c.step_size;
            if constexpr (S8) {
                top[u][0] = fmaxf(top[u][0], fabsf(m[u][i]));
                top[u][1] = fmaxf(top[u][1], r[u][i]);
            }
        }
        store4<PT, FULL>(t.p, e[u], n[u], p[u]);
        if (t.copy) store4<kBF16, FULL>(t.copy, e[u], n[u], p[u]);
        if constexpr (!S8) {
            store4<kF32, FULL>(t.m, e[u], n[u], m[u]);
            store4<kF32, FULL>(t.v, e[u], n[u], v[u]);
        }
    }
    if constexpr (S8) {
        static_assert(kAdamU == 2, "four reciprocals fill the four lanes of a quad");
#pragma unroll
        for (int u = 0; u < kAdamU; ++u) {
            top[u][0] = half_wave_max(top[u][0]);
            top[u][1] = half_wave_max(top[u][1]);
        }
        // The four scales that a thread's groups need are the same in all of a
        // block's lanes: lane j of every four divides for number j, and the
        // quad shares the results. A block with nothing above 2^-100 is held as
        // zeros, as its reciprocal scale could overflow.
        const int j = threadIdx.x & 3;
        const float mine = j < 2 ? (j == 0 ? top[0][0] : top[0][1]) : (j == 2 ? top[1][0] : top[1][1]);
        const bool use = mine >= 0x1p-100f;
        const int inverse = __float_as_int(use ? 1.0f / mine * 448.0f : 0.0f);
        const float scale = use ? mine * (1.0f / 448.0f) : 0.0f;
#define DPS_QUAD(n) __int_as_float(__builtin_amdgcn_update_dpp(0, inverse, (n) * 0x55, 0xf, 0xf, false))
        const float inv[kAdamU][2] = {{DPS_QUAD(0), DPS_QUAD(1)}, {DPS_QUAD(2), DPS_QUAD(3)}};
#undef DPS_QUAD
        // number j of a block's first four lanes: scale j & 1 of group j / 2
        {
            const long long first = e[0] - 4 * (long long)j, at = j < 2 ? first : first + kNT * 4;
            if ((threadIdx.x & 31) < 4 && at < t.n) t.scales[at / kStateBlock * 2 + (j & 1)] = scale;
        }
        unsigned long long key = 0;
        if constexpr (SR) {
            key = mix64(k.seed + (unsigned long long)c.step * kGolden);
            key = mix64(key + (unsigned long long)(k.index0 + index + 1) * kGolden);
            key += ((unsigned long long)at / 2 + 1) * kGolden + (unsigned long long)threadIdx.x * (2 * kGolden);
        }
#pragma unroll
        for (int u = 0; u < kAdamU; ++u) {
            unsigned long long z[2];
            if constexpr (SR) {
                // counters of the thread's two pairs of elements
                z[0] = mix64(key + u * (kNT * 2 * kGolden));
                z[1] = mix64(key + (u * kNT * 2 + 1) * kGolden);
            }
            float ym[4], yr[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                ym[i] = m[u][i] * inv[u][0];
                yr[i] = r[u][i] * inv[u][1];
                if (yr[i] > 0.0f) yr[i] = fmaxf(yr[i], 0x1p-9f);
                if constexpr (SR) {
                    const unsigned half = (unsigned)(z[i >> 1] >> (32 * (i & 1)));
                    ym[i] = e4m3_stochastic(ym[i], half & 0xffffu);
                    yr[i] = e4m3_stochastic(yr[i], half >> 16);
                }
            }
            store_codes<FULL>(t.m, e[u], n[u], pack_e4m3(ym));
            store_codes<FULL>(t.v, e[u], n[u], pack_e4m3(yr));
        }
    }
}

template <int PT, int GT, bool S8, bool SR>
__global__ __launch_bounds__(kNT) void adamw_kernel(const AdamParams k, unsigned first)
{
    const int b = (int)(first + blockIdx.x);
    // the last tensor that starts at or before this chunk, by halves (one tensor a
    // lane, a vector load and a ballot: 4% slower at 200M elements)
    int t = 0;
#pragma unroll
    for (int half = kAdamTensors / 2; half > 0; half >>= 1)
        if (t + half < k.nt && b >= k.first[t + half]) t += half;
    const long long at = (long long)(b - k.first[t]) * kAdamChunk;
    if (at + kAdamChunk <= k.t[t].n)
        adam_chunk<PT, GT, S8, SR, true>(k, k.t[t], t, at);
    else
        adam_chunk<PT, GT, S8, SR, false>(k, k.t[t], t, at);
}

template <int PT, int GT>
hipError_t launch_adamw_typed(const AdamParams &p, bool eight, bool stochastic, hipStream_t stream)
{
    // fp32 states: LDS that the kernel does not use keeps a CU at two workgroups,
    // 7 KiB a wave on their way, and their streams apart (fp32 parameters, 200M elements:
    // 925 us for 985 with eight; 80M 360 for 379; 7M 34.8 for 35.2), but
    // not where eight a CU take every chunk at once (2M: 9.5 us for 10.9; 4M 19.3 for
    // 19.8; 1M, at most two a CU anyway, 6.7 and 6.7). With 8-bit states a wave computes
    // longer and every one helps (200M elements: 578 us for 722).
    constexpr int kCUs = 256, kPerCU = 8;
    const unsigned lds = !eight && p.first[p.nt] > kPerCU * kCUs ? 80u << 10 : 0u;
    return launch_groups256(p.first[p.nt], [&](unsigned first, unsigned grid) {
        if (!eight)
            adamw_kernel<PT, GT, false, false><<<grid, kNT, lds, stream>>>(p, first);
        else if (!stochastic)
            adamw_kernel<PT, GT, true, false><<<grid, kNT, 0, stream>>>(p, first);
        else
            adamw_kernel<PT, GT, true, true><<<grid, kNT, 0, stream>>>(p, first);
    });
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
