// Calls the optimizer and 4-bit entry points with AddressSanitizer and
// UndefinedBehaviorSanitizer in a host build whose launches are stand-ins: they
// check what a kernel would be given (tables, chunk prefixes, grids) instead of
// running one. The device pointers are fake addresses that are never
// dereferenced. Exit status 0 when everything holds.
#include <stdio.h>
#include <string.h>

#include <vector>

#include "dpsync.h"
#include "mxfp4_internal.h"
#include "optim_internal.h"

static int failures = 0, launches = 0;
static long long elements = 0, last_index = 0;
static bool finished = false;

#define EXPECT(c)                                              \
    do {                                                       \
        if (!(c)) {                                            \
            fprintf(stderr, "FAIL line %d: %s\n", __LINE__, #c); \
            ++failures;                                        \
        }                                                      \
    } while (0)

namespace dps {

int hip_failure_code(hipError_t e) { return e == hipSuccess ? DP_OK : DP_ERR_HIP; }
long long norm_chunks(long long n) { return (n + 8191) / 8192; }
long long adam_chunks(long long n) { return (n + 2047) / 2048; }

hipError_t launch_grad_norm(const NormParams &p, int, int grid, hipStream_t)
{
    EXPECT(p.nt >= 0 && p.nt <= kNormTensors && grid >= 1 && grid <= kNormMaxGrid && p.first[0] == 0);
    for (int i = 0; i < p.nt; ++i) {
        EXPECT(p.first[i + 1] - p.first[i] == norm_chunks(p.n[i]));
        elements += p.n[i];
    }
    EXPECT((p.add != 0) == (launches > 0));
    EXPECT(!finished);
    finished = p.finish;
    ++launches;
    return hipSuccess;
}

hipError_t launch_adamw(const AdamParams &p, int, int, bool eight, bool, hipStream_t)
{
    EXPECT(p.nt >= 1 && p.nt <= kAdamTensors && p.first[0] == 0 && p.first[p.nt] > 0);
    EXPECT(p.index0 == last_index);
    last_index += p.nt;
    for (int i = 0; i < p.nt; ++i) {
        EXPECT(p.first[i + 1] - p.first[i] == adam_chunks(p.t[i].n));
        EXPECT(!eight || p.t[i].n == 0 || p.t[i].scales);
        elements += p.t[i].n;
    }
    ++launches;
    return hipSuccess;
}

hipError_t launch_mxfp4_quantize(const MxQuantParams &, int, hipStream_t) { ++launches; return hipSuccess; }
hipError_t launch_mxfp4_dequantize(const MxExpandParams &, int, hipStream_t) { ++launches; return hipSuccess; }
hipError_t launch_mxfp4_gemm(const MxGemmParams &p, int, int x_dt, hipStream_t)
{
    EXPECT(x_dt < 0 ? p.a && p.a_scales : p.x != nullptr);
    ++launches;
    return hipSuccess;
}
bool mx_quantize_inside(long long m, long long, long long) { return m <= 4; }

}  // namespace dps

static void fresh()
{
    launches = 0;
    elements = last_index = 0;
    finished = false;
}

int main()
{
    char *at = (char *)((uintptr_t)1 << 40);
    for (int nt : {0, 1, 2, 63, 64, 65, 127, 128, 129, 300, 5000}) {
        std::vector<int64_t> n(nt);
        std::vector<void *> p(nt), g(nt), m(nt), v(nt), c(nt), s(nt);
        long long all = 0;
        char *next = at;
        auto take = [&](size_t bytes) { char *r = next; next += (bytes + 255) / 256 * 256; return r; };
        for (int i = 0; i < nt; ++i) {
            n[i] = i % 7 == 3 ? 0 : 1 + (int64_t)i * i * 37 % 40000;
            all += n[i];
            for (auto *a : {&p, &g, &m, &v, &c, &s}) (*a)[i] = n[i] ? take(n[i] * 4) : nullptr;
        }
        void *ctrl = take(16), *ws = take(DP_GRAD_NORM_WS_BYTES);
        fresh();
        EXPECT(dp_grad_norm(nt, n.data(), g.data(), DP_F32, 1.0, (dp_step_ctrl_t *)ctrl, ws, nullptr) ==
               (nt ? DP_OK : n.data() && g.data() ? DP_OK : DP_ERR_INVALID_ARG));
        if (nt) EXPECT(finished && elements == all && launches == (nt + 127) / 128);
        dp_adamw_opts_t o = {1e-3, 0.9, 0.999, 1e-8, 0.01, 3, 7, 0, 0};
        if (!nt) continue;
        fresh();
        EXPECT(dp_adamw(nt, n.data(), p.data(), DP_F32, g.data(), DP_BF16, (float *const *)m.data(),
                        (float *const *)v.data(), c.data(), &o, (dp_step_ctrl_t *)ctrl, nullptr) == DP_OK);
        EXPECT(elements == all);
        o.flags = DP_ADAMW_STOCHASTIC;
        o.step = 0;
        fresh();
        EXPECT(dp_adamw8(nt, n.data(), p.data(), DP_BF16, g.data(), DP_F32, (uint8_t *const *)m.data(),
                         (uint8_t *const *)v.data(), (float *const *)s.data(), nullptr, &o, (dp_step_ctrl_t *)ctrl,
                         nullptr) == DP_OK);
        EXPECT(elements == all);
        if (nt > 70) {
            // an overlap between tensors far apart in the list, and nothing launched for it
            void *was = v[nt - 2];
            v[nt - 2] = (char *)p[1] + 4;
            n[nt - 2] = 8;
            fresh();
            EXPECT(dp_adamw(nt, n.data(), p.data(), DP_F32, g.data(), DP_F32, (float *const *)m.data(),
                            (float *const *)v.data(), nullptr, &o, nullptr, nullptr) != DP_OK);
            EXPECT(launches == 0);
            v[nt - 2] = was;
        }
    }
    char *a = at, *b = at + (1ll << 36), *c = at + (2ll << 36), *d = at + (3ll << 36), *e = at + (4ll << 36);
    const int64_t big = (int64_t)1 << 24;
    fresh();
    EXPECT(dp_mxfp4_quantize(a, 100, 70, 71, DP_BF16, b, c, d, e, nullptr) == DP_OK);
    EXPECT(dp_mxfp4_quantize(a, big, big, big, DP_F32, b, c, nullptr, nullptr, nullptr) != DP_OK);
    EXPECT(dp_mxfp4_quantize(a, INT64_MAX, 1, 1, DP_F32, b, c, nullptr, nullptr, nullptr) == DP_ERR_INVALID_ARG);
    EXPECT(dp_mxfp4_dequantize(a, b, 33, 65, c, 65, DP_BF16, nullptr) == DP_OK);
    EXPECT(dp_mxfp4_dequantize(a, b, big, big, c, big, DP_F32, nullptr) != DP_OK);
    EXPECT(dp_gemm_mxfp4(a, b, c, d, e, 300, 200, 100, DP_F32, 1, nullptr) == DP_OK);
    EXPECT(dp_gemm_mxfp4(a, b, c, d, e, big, big, 100, DP_F32, 0, nullptr) == DP_ERR_INVALID_ARG);
    EXPECT(launches == 3);
    EXPECT(dp_mxfp4_linear_ws_bytes(4, 100, 1000) == 0 && dp_mxfp4_linear_ws_bytes(5, 100, 1000) > 0);
    fresh();
    EXPECT(dp_mxfp4_linear(a, 1000, DP_BF16, b, c, d, 4, 100, 1000, DP_F32, nullptr, nullptr) == DP_OK && launches == 1);
    EXPECT(dp_mxfp4_linear(a, 1000, DP_BF16, b, c, d, 5, 100, 1000, DP_F32, nullptr, nullptr) == DP_ERR_INVALID_ARG);
    EXPECT(dp_mxfp4_linear(a, 1000, DP_BF16, b, c, d, 5, 100, 1000, DP_F32, e, nullptr) == DP_OK && launches == 3);
    printf("%d failures\n", failures);
    return failures ? 1 : 0;
}
