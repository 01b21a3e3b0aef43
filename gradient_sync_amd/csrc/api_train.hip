// extern "C" entry points of the optimizer step and of the 4-bit block-scaled
// product: argument validation and kernel dispatch on the caller's stream. The
// contract of every call is stated in include/dpsync.h.
#include <math.h>
#include <stdint.h>
#include <string.h>

#include <algorithm>
#include <new>

#include "dpsync.h"
#include "mxfp4_internal.h"
#include "optim_internal.h"

static_assert(sizeof(dp_step_ctrl_t) == sizeof(dps::StepCtrl), "control block layouts differ");
static_assert(DP_GRAD_NORM_WS_BYTES >= dps::kNormWsBytes, "norm workspace too small");
static_assert(DP_STATE_BLOCK == dps::kStateBlock, "state block sizes differ");

namespace {

constexpr int64_t kMaxDim = (int64_t)1 << 24;
// Elements of a product: its tiles of 128 x 128 are then fewer than a launch's
// workgroups, edges included (2^23 + 2^18 of 2^24 - 1).
constexpr int64_t kMaxOut = (int64_t)1 << 37;

struct Range {
    uintptr_t lo, hi;
    bool written;
};

// Adds [p, p + bytes) to `r`.
void add(Range *r, size_t &n, const void *p, size_t bytes, bool written)
{
    if (bytes) r[n++] = Range{(uintptr_t)p, (uintptr_t)p + bytes, written};
}

// true when a written range overlaps any other
bool aliased(Range *r, size_t n)
{
    std::sort(r, r + n, [](const Range &a, const Range &b) { return a.lo < b.lo; });
    uintptr_t any = 0, written = 0;
    for (size_t i = 0; i < n; ++i) {
        if (r[i].lo < (r[i].written ? any : written)) return true;
        any = std::max(any, r[i].hi);
        if (r[i].written) written = std::max(written, r[i].hi);
    }
    return false;
}

bool aligned(const void *p, uintptr_t a) { return p && (uintptr_t)p % a == 0; }

// NULL entries are allowed where the tensor is empty
bool tensors_ok(const void *const *a, const int64_t *counts, int nt, int es)
{
    if (!a) return false;
    for (int i = 0; i < nt; ++i)
        if (counts[i] > 0 && !aligned(a[i], (uintptr_t)es)) return false;
    return true;
}

bool counts_ok(const int64_t *counts, int nt)
{
    if (nt < 0 || nt > DP_MAX_TENSORS || !counts) return false;
    for (int i = 0; i < nt; ++i)
        if (counts[i] < 0 || counts[i] > ((int64_t)1 << 40)) return false;
    return true;
}

bool float_dt(int dt) { return dt == DP_F32 || dt == DP_BF16; }

dp_status_t run_adamw(int nt, const int64_t *counts, void *const *params, int p_dt,
                      const void *const *grads, int g_dt, void *const *m, void *const *v,
                      float *const *scales, void *const *copies, const dp_adamw_opts_t *o,
                      const dp_step_ctrl_t *ctrl, void *stream, bool eight)
{
    if (!counts_ok(counts, nt) || !o) return DP_ERR_INVALID_ARG;
    if (!float_dt(p_dt) || !float_dt(g_dt)) return DP_ERR_UNSUPPORTED;
    if (copies && p_dt != DP_F32) return DP_ERR_UNSUPPORTED;
    const bool stochastic = (o->flags & DP_ADAMW_STOCHASTIC) != 0;
    if ((o->flags & ~DP_ADAMW_STOCHASTIC) || o->reserved) return DP_ERR_INVALID_ARG;
    if (stochastic && !eight) return DP_ERR_UNSUPPORTED;
    if (!(isfinite(o->lr) && o->lr >= 0 && o->beta1 >= 0 && o->beta1 < 1 && o->beta2 >= 0 &&
          o->beta2 < 1 && isfinite(o->eps) && o->eps >= 0 && isfinite(o->weight_decay) &&
          o->weight_decay >= 0))
        return DP_ERR_INVALID_ARG;
    if (o->step < 0 || (o->step == 0 && !ctrl)) return DP_ERR_INVALID_ARG;
    if (ctrl && !aligned(ctrl, 4)) return DP_ERR_INVALID_ARG;
    const int pe = dps::elem_size(p_dt), ge = dps::elem_size(g_dt), se = eight ? 1 : 4;
    if (!tensors_ok((const void *const *)params, counts, nt, pe) || !tensors_ok(grads, counts, nt, ge) ||
        !tensors_ok((const void *const *)m, counts, nt, se) ||
        !tensors_ok((const void *const *)v, counts, nt, se) ||
        (eight && !tensors_ok((const void *const *)scales, counts, nt, 8)) ||
        (copies && !tensors_ok((const void *const *)copies, counts, nt, 2)))
        return DP_ERR_INVALID_ARG;

    Range few[6 * 64 + 1];
    Range *r = nt <= 64 ? few : new (std::nothrow) Range[6 * (size_t)nt + 1];
    if (!r) return DP_ERR_INVALID_ARG;
    size_t nr = 0;
    for (int i = 0; i < nt; ++i) {
        const size_t n = (size_t)counts[i];
        add(r, nr, params[i], n * pe, true);
        add(r, nr, grads[i], n * ge, false);
        add(r, nr, m[i], n * se, true);
        add(r, nr, v[i], n * se, true);
        if (eight) add(r, nr, scales[i], (n + DP_STATE_BLOCK - 1) / DP_STATE_BLOCK * 8, true);
        if (copies) add(r, nr, copies[i], n * 2, true);
    }
    if (ctrl) add(r, nr, ctrl, sizeof(*ctrl), false);
    const bool bad = aliased(r, nr);
    if (r != few) delete[] r;
    if (bad) return DP_ERR_ALIAS;

    dps::AdamParams p;
    memset(&p, 0, sizeof(p));
    p.beta1 = (float)o->beta1;
    p.beta2 = (float)o->beta2;
    p.one_minus_beta1 = (float)(1.0 - o->beta1);
    p.one_minus_beta2 = (float)(1.0 - o->beta2);
    p.eps = (float)o->eps;
    p.decay = (float)(1.0 - o->lr * o->weight_decay);
    if (o->step > 0) {
        p.step_size = (float)(o->lr / (1.0 - pow(o->beta1, (double)o->step)));
        p.inv_sqrt_bc2 = (float)(1.0 / sqrt(1.0 - pow(o->beta2, (double)o->step)));
    }
    p.lr = o->lr;
    p.dbeta1 = o->beta1;
    p.dbeta2 = o->beta2;
    p.step = o->step;
    p.seed = o->seed;
    p.ctrl = (const dps::StepCtrl *)ctrl;
    for (int i = 0; i < nt;) {
        p.nt = 0;
        p.index0 = i;
        long long chunks = 0;
        for (; i < nt && p.nt < dps::kAdamTensors; ++i) {
            const long long more = dps::adam_chunks(counts[i]);
            if (chunks + more > 0x7fffffffLL - 4096) break;
            dps::AdamTensor &t = p.t[p.nt];
            t.p = (char *)params[i];
            t.g = (const char *)grads[i];
            t.m = (char *)m[i];
            t.v = (char *)v[i];
            t.copy = copies ? (char *)copies[i] : nullptr;
            t.scales = eight ? scales[i] : nullptr;
            t.n = counts[i];
            p.first[p.nt++] = (int)chunks;
            chunks += more;
        }
        p.first[p.nt] = (int)chunks;
        if (!chunks) continue;
        const hipError_t e = dps::launch_adamw(p, p_dt, g_dt, eight, stochastic, (hipStream_t)stream);
        if (e != hipSuccess) return (dp_status_t)dps::hip_failure_code(e);
    }
    return DP_OK;
}

bool mx_dims_ok(int64_t rows, int64_t cols) { return rows >= 0 && cols >= 0 && rows <= kMaxDim && cols <= kMaxDim; }

// a quantised operand: 16-byte aligned codes, 4-byte aligned scales
bool mx_operand_ok(const void *codes, const void *scales) { return aligned(codes, 16) && aligned(scales, 4); }

}  // namespace

extern "C" {

dp_status_t dp_grad_norm(int nt, const int64_t *counts, const void *const *grads, int dt,
                         double max_norm, dp_step_ctrl_t *ctrl, void *workspace, void *stream)
{
    if (!counts_ok(counts, nt)) return DP_ERR_INVALID_ARG;
    if (!float_dt(dt)) return DP_ERR_UNSUPPORTED;
    const int es = dps::elem_size(dt);
    if (!tensors_ok(grads, counts, nt, es) || !aligned(ctrl, 4) || !aligned(workspace, 8) ||
        !(max_norm >= 0) || !isfinite(max_norm))
        return DP_ERR_INVALID_ARG;
    const uintptr_t c0 = (uintptr_t)ctrl, c1 = c0 + sizeof(*ctrl);
    const uintptr_t w0 = (uintptr_t)workspace, w1 = w0 + DP_GRAD_NORM_WS_BYTES;
    if (c0 < w1 && w0 < c1) return DP_ERR_ALIAS;
    long long most = 1, all = 0;
    for (int i = 0; i < nt; ++i) {
        const uintptr_t lo = (uintptr_t)grads[i], hi = lo + (uintptr_t)counts[i] * es;
        if (counts[i] && ((lo < c1 && c0 < hi) || (lo < w1 && w0 < hi))) return DP_ERR_ALIAS;
        all += dps::norm_chunks(counts[i]);
        if ((i + 1) % dps::kNormTensors == 0 || i + 1 == nt) {
            if (all > 0x7fffffffLL - 4096) return DP_ERR_INVALID_ARG;
            most = std::max(most, all);
            all = 0;
        }
    }
    const int grid = (int)std::min<long long>(most, dps::kNormMaxGrid);
    dps::NormParams p;
    memset(&p, 0, sizeof(p));
    p.partial = (double *)workspace;
    p.ticket = (unsigned *)((char *)workspace + dps::kNormMaxGrid * sizeof(double));
    p.ctrl = (dps::StepCtrl *)ctrl;
    p.max_norm = max_norm;
    int i = 0;
    do {
        p.nt = 0;
        long long chunks = 0;
        for (; i < nt && p.nt < dps::kNormTensors; ++i) {
            p.g[p.nt] = (const char *)grads[i];
            p.n[p.nt] = counts[i];
            p.first[p.nt++] = (int)chunks;
            chunks += dps::norm_chunks(counts[i]);
        }
        p.first[p.nt] = (int)chunks;
        p.finish = i == nt;
        const hipError_t e = dps::launch_grad_norm(p, dt, grid, (hipStream_t)stream);
        if (e != hipSuccess) return (dp_status_t)dps::hip_failure_code(e);
        p.add = 1;
    } while (i < nt);
    return DP_OK;
}

dp_status_t dp_adamw(int nt, const int64_t *counts, void *const *params, int p_dt,
                     const void *const *grads, int g_dt, float *const *m, float *const *v,
                     void *const *copies, const dp_adamw_opts_t *opts, const dp_step_ctrl_t *ctrl,
                     void *stream)
{
    return run_adamw(nt, counts, params, p_dt, grads, g_dt, (void *const *)m, (void *const *)v, nullptr,
                     copies, opts, ctrl, stream, false);
}

dp_status_t dp_adamw8(int nt, const int64_t *counts, void *const *params, int p_dt,
                      const void *const *grads, int g_dt, uint8_t *const *m, uint8_t *const *v,
                      float *const *scales, void *const *copies, const dp_adamw_opts_t *opts,
                      const dp_step_ctrl_t *ctrl, void *stream)
{
    return run_adamw(nt, counts, params, p_dt, grads, g_dt, (void *const *)m, (void *const *)v, scales,
                     copies, opts, ctrl, stream, true);
}

size_t dp_mxfp4_code_bytes(int64_t rows, int64_t cols)
{
    return mx_dims_ok(rows, cols) ? (size_t)(rows * dps::mx_pitch(cols)) : 0;
}

size_t dp_mxfp4_scale_bytes(int64_t rows, int64_t cols)
{
    return mx_dims_ok(rows, cols) ? (size_t)((rows + 15) / 16 * dps::mx_scale_tiles(cols) * 256) : 0;
}

dp_status_t dp_mxfp4_quantize(const void *src, int64_t rows, int64_t cols, int64_t ld, int dt,
                              void *codes, void *scales, void *codes_t, void *scales_t, void *stream)
{
    if (!mx_dims_ok(rows, cols) || ld < cols || ld > ((int64_t)1 << 40)) return DP_ERR_INVALID_ARG;
    if (!float_dt(dt)) return DP_ERR_UNSUPPORTED;
    if (rows == 0 || cols == 0) return DP_OK;
    if ((!codes && !codes_t) || !codes != !scales || !codes_t != !scales_t) return DP_ERR_INVALID_ARG;
    const int es = dps::elem_size(dt);
    if (!aligned(src, (uintptr_t)es) || (codes && !mx_operand_ok(codes, scales)) ||
        (codes_t && !mx_operand_ok(codes_t, scales_t)) ||
        (codes_t && (rows + 127) / 128 * ((cols + 127) / 128) > dps::kMaxGroups256) ||
        (!codes_t && (rows + 15) / 16 * dps::mx_scale_tiles(cols) > dps::kMaxGroups256))
        return DP_ERR_INVALID_ARG;
    Range r[5];
    size_t n = 0;
    add(r, n, src, ((size_t)(rows - 1) * ld + cols) * es, false);
    if (codes) {
        add(r, n, codes, dp_mxfp4_code_bytes(rows, cols), true);
        add(r, n, scales, dp_mxfp4_scale_bytes(rows, cols), true);
    }
    if (codes_t) {
        add(r, n, codes_t, dp_mxfp4_code_bytes(cols, rows), true);
        add(r, n, scales_t, dp_mxfp4_scale_bytes(cols, rows), true);
    }
    if (aliased(r, n)) return DP_ERR_ALIAS;
    dps::MxQuantParams p = {(const char *)src, rows, cols, ld, (unsigned char *)codes,
                            (unsigned char *)scales, (unsigned char *)codes_t, (unsigned char *)scales_t};
    const hipError_t e = dps::launch_mxfp4_quantize(p, dt, (hipStream_t)stream);
    return (dp_status_t)dps::hip_failure_code(e);
}

dp_status_t dp_mxfp4_dequantize(const void *codes, const void *scales, int64_t rows, int64_t cols,
                                void *dst, int64_t ld, int dt, void *stream)
{
    if (!mx_dims_ok(rows, cols) || ld < cols || ld > ((int64_t)1 << 40)) return DP_ERR_INVALID_ARG;
    if (!float_dt(dt)) return DP_ERR_UNSUPPORTED;
    if (rows == 0 || cols == 0) return DP_OK;
    const int es = dps::elem_size(dt);
    if (!mx_operand_ok(codes, scales) || !aligned(dst, (uintptr_t)es) ||
        rows * ((cols + 7) / 8) > (int64_t)0x7fffffff * 128)
        return DP_ERR_INVALID_ARG;
    Range r[3];
    size_t n = 0;
    add(r, n, codes, dp_mxfp4_code_bytes(rows, cols), false);
    add(r, n, scales, dp_mxfp4_scale_bytes(rows, cols), false);
    add(r, n, dst, ((size_t)(rows - 1) * ld + cols) * es, true);
    if (aliased(r, n)) return DP_ERR_ALIAS;
    dps::MxExpandParams p = {(const unsigned char *)codes, (const unsigned char *)scales, (char *)dst, rows, cols, ld};
    const hipError_t e = dps::launch_mxfp4_dequantize(p, dt, (hipStream_t)stream);
    return (dp_status_t)dps::hip_failure_code(e);
}

dp_status_t dp_gemm_mxfp4(const void *a, const void *a_scales, const void *b, const void *b_scales,
                          void *c, int64_t m, int64_t n, int64_t kk, int c_dt, int accumulate,
                          void *stream)
{
    if (!mx_dims_ok(m, n) || m * n > kMaxOut || kk < 1 || kk > kMaxDim) return DP_ERR_INVALID_ARG;
    if (!float_dt(c_dt) || (accumulate && c_dt != DP_F32)) return DP_ERR_UNSUPPORTED;
    if (m == 0 || n == 0) return DP_OK;
    const int es = dps::elem_size(c_dt);
    if (!mx_operand_ok(a, a_scales) || !mx_operand_ok(b, b_scales) || !aligned(c, (uintptr_t)es))
        return DP_ERR_INVALID_ARG;
    Range r[5];
    size_t nr = 0;
    add(r, nr, a, dp_mxfp4_code_bytes(m, kk), false);
    add(r, nr, a_scales, dp_mxfp4_scale_bytes(m, kk), false);
    add(r, nr, b, dp_mxfp4_code_bytes(n, kk), false);
    add(r, nr, b_scales, dp_mxfp4_scale_bytes(n, kk), false);
    add(r, nr, c, (size_t)m * n * es, true);
    if (aliased(r, nr)) return DP_ERR_ALIAS;
    dps::MxGemmParams p;
    memset(&p, 0, sizeof(p));
    p.a = (const unsigned char *)a;
    p.a_scales = (const unsigned char *)a_scales;
    p.b = (const unsigned char *)b;
    p.b_scales = (const unsigned char *)b_scales;
    p.c = (char *)c;
    p.m = m;
    p.n = n;
    p.k = kk;
    p.accumulate = accumulate != 0;
    const hipError_t e = dps::launch_mxfp4_gemm(p, c_dt, -1, (hipStream_t)stream);
    return (dp_status_t)dps::hip_failure_code(e);
}

size_t dp_mxfp4_linear_ws_bytes(int64_t m, int64_t n, int64_t kk)
{
    if (!mx_dims_ok(m, kk) || !mx_dims_ok(m, n) || dps::mx_quantize_inside(m, n, kk)) return 0;
    return (dp_mxfp4_code_bytes(m, kk) + 255) / 256 * 256 + dp_mxfp4_scale_bytes(m, kk);
}

dp_status_t dp_mxfp4_linear(const void *x, int64_t ldx, int x_dt, const void *w,
                            const void *w_scales, void *y, int64_t m, int64_t n, int64_t kk,
                            int y_dt, void *workspace, void *stream)
{
    if (!mx_dims_ok(m, n) || m * n > kMaxOut || kk < 1 || kk > kMaxDim || ldx < kk || ldx > ((int64_t)1 << 40))
        return DP_ERR_INVALID_ARG;
    if (!float_dt(x_dt) || !float_dt(y_dt)) return DP_ERR_UNSUPPORTED;
    if (m == 0 || n == 0) return DP_OK;
    const int xe = dps::elem_size(x_dt), ye = dps::elem_size(y_dt);
    const size_t ws = dp_mxfp4_linear_ws_bytes(m, n, kk);
    if (!aligned(x, (uintptr_t)xe) || !mx_operand_ok(w, w_scales) || !aligned(y, (uintptr_t)ye) ||
        (ws && !aligned(workspace, 16)))
        return DP_ERR_INVALID_ARG;
    Range r[5];
    size_t nr = 0;
    add(r, nr, x, ((size_t)(m - 1) * ldx + kk) * xe, false);
    add(r, nr, w, dp_mxfp4_code_bytes(n, kk), false);
    add(r, nr, w_scales, dp_mxfp4_scale_bytes(n, kk), false);
    add(r, nr, y, (size_t)m * n * ye, true);
    if (ws) add(r, nr, workspace, ws, true);
    if (aliased(r, nr)) return DP_ERR_ALIAS;
    dps::MxGemmParams p;
    memset(&p, 0, sizeof(p));
    p.b = (const unsigned char *)w;
    p.b_scales = (const unsigned char *)w_scales;
    p.c = (char *)y;
    p.m = m;
    p.n = n;
    p.k = kk;
    if (!ws) {
        p.x = (const char *)x;
        p.ldx = ldx;
        const hipError_t e = dps::launch_mxfp4_gemm(p, y_dt, x_dt, (hipStream_t)stream);
        return (dp_status_t)dps::hip_failure_code(e);
    }
    unsigned char *codes = (unsigned char *)workspace;
    unsigned char *scales = codes + (dp_mxfp4_code_bytes(m, kk) + 255) / 256 * 256;
    dps::MxQuantParams q = {(const char *)x, m, kk, ldx, codes, scales, nullptr, nullptr};
    hipError_t e = dps::launch_mxfp4_quantize(q, x_dt, (hipStream_t)stream);
    if (e != hipSuccess) return (dp_status_t)dps::hip_failure_code(e);
    p.a = codes;
    p.a_scales = scales;
    e = dps::launch_mxfp4_gemm(p, y_dt, -1, (hipStream_t)stream);
    return (dp_status_t)dps::hip_failure_code(e);
}

}  // extern "C"
