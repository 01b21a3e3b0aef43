// Overlapping buffers and other refusals of the optimizer and 4-bit entry
// points, each with the status it must give, under AddressSanitizer and
// UndefinedBehaviorSanitizer in a host build whose launches are stand-ins:
// nothing may be launched for a refused call. Lists beyond 64 tensors take the
// range table from the heap, shorter ones from the stack; both are gone through.
// The device pointers are fake addresses that are never dereferenced. Exit status
// 0 when everything holds.
#include <stdio.h>
#include <string.h>

#include <vector>

#include "dpsync.h"
#include "mxfp4_internal.h"
#include "optim_internal.h"

static int failures = 0, launches = 0;

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
hipError_t launch_grad_norm(const NormParams &, int, int, hipStream_t) { ++launches; return hipSuccess; }
hipError_t launch_adamw(const AdamParams &, int, int, bool, bool, hipStream_t) { ++launches; return hipSuccess; }
hipError_t launch_mxfp4_quantize(const MxQuantParams &, int, hipStream_t) { ++launches; return hipSuccess; }
hipError_t launch_mxfp4_dequantize(const MxExpandParams &, int, hipStream_t) { ++launches; return hipSuccess; }
hipError_t launch_mxfp4_gemm(const MxGemmParams &, int, int, hipStream_t) { ++launches; return hipSuccess; }
bool mx_quantize_inside(long long m, long long, long long) { return m <= 4; }

}  // namespace dps

struct Lists {
    std::vector<int64_t> n;
    std::vector<void *> p, g, m, v, c, s;
    char *next = (char *)((uintptr_t)1 << 40);
    char *ctrl, *ws;
    dp_adamw_opts_t o = {1e-3, 0.9, 0.999, 1e-8, 0.01, 3, 7, 0, 0};

    char *take(size_t bytes)
    {
        char *r = next;
        next += (bytes + 255) / 256 * 256;
        return r;
    }
    explicit Lists(int nt) : n(nt), p(nt), g(nt), m(nt), v(nt), c(nt), s(nt)
    {
        for (int i = 0; i < nt; ++i) {
            n[i] = 10 + 37 * (i % 11);
            for (auto *a : {&p, &g, &m, &v, &c, &s}) (*a)[i] = take(n[i] * 4);
        }
        ctrl = take(16);
        ws = take(DP_GRAD_NORM_WS_BYTES);
    }
    dp_status_t adamw()
    {
        launches = 0;
        return dp_adamw((int)n.size(), n.data(), p.data(), DP_F32, g.data(), DP_F32, (float *const *)m.data(),
                        (float *const *)v.data(), c.data(), &o, (dp_step_ctrl_t *)ctrl, nullptr);
    }
    dp_status_t adamw8()
    {
        launches = 0;
        return dp_adamw8((int)n.size(), n.data(), p.data(), DP_F32, g.data(), DP_F32, (uint8_t *const *)m.data(),
                         (uint8_t *const *)v.data(), (float *const *)s.data(), c.data(), &o, (dp_step_ctrl_t *)ctrl, nullptr);
    }
    dp_status_t norm()
    {
        launches = 0;
        return dp_grad_norm((int)n.size(), n.data(), g.data(), DP_F32, 1.0, (dp_step_ctrl_t *)ctrl, ws, nullptr);
    }
};

int main()
{
    for (int nt : {2, 63, 64, 65, 100, 3000}) {
        const int a = 0, z = nt - 1;
        Lists ok(nt);
        EXPECT(ok.adamw() == DP_OK && launches == (nt + 63) / 64);
        EXPECT(ok.adamw8() == DP_OK && launches == (nt + 63) / 64);
        EXPECT(ok.norm() == DP_OK && launches == (nt + 127) / 128);
        // each written buffer of the last tensor on each buffer of the first, by its last element
        auto end = [](const Lists &x, const std::vector<void *> &b, int at, size_t es) { return (char *)b[at] + (x.n[at] - 1) * es; };
        for (int from = 0; from < 4; ++from)
            for (int to = 0; to < 5; ++to) {
                Lists x(nt);
                std::vector<void *> *written[] = {&x.p, &x.m, &x.v, &x.c}, *any[] = {&x.p, &x.g, &x.m, &x.v, &x.c};
                (*written[from])[z] = end(x, *any[to], a, to == 4 ? 2 : 4);
                if ((uintptr_t)(*written[from])[z] % 4) (*written[from])[z] = (char *)(*written[from])[z] - 2;
                EXPECT(x.adamw() == DP_ERR_ALIAS && launches == 0);
            }
        {
            Lists x(nt);                             // a gradient that another tensor's update writes
            x.g[z] = end(x, x.m, a, 4);
            EXPECT(x.adamw() == DP_ERR_ALIAS && launches == 0);
        }
        {
            Lists x(nt);                             // gradients are only read: they may be shared
            x.g[z] = x.g[a];
            x.n[z] = x.n[a] = 5;
            EXPECT(x.adamw() == DP_OK && x.norm() == DP_OK);
        }
        {
            Lists x(nt);                             // side by side is no overlap
            x.n[a] = 10;
            x.n[z] = 16;
            x.v[z] = (char *)x.v[a] + 40;
            x.m[z] = (char *)x.m[a] + 40;
            EXPECT(x.adamw() == DP_OK && x.adamw8() == DP_OK);
        }
        for (int which = 0; which < 4; ++which) {    // 8-bit: scales and codes
            Lists x(nt);
            if (which == 0) x.s[z] = x.m[a];
            if (which == 1) x.s[z] = (char *)x.s[a] + (x.n[a] - 1) / DP_STATE_BLOCK * 8;
            if (which == 2) x.m[z] = (char *)x.v[a] + x.n[a] - 1;
            if (which == 3) x.v[z] = (char *)x.g[a] + 1;
            EXPECT(x.adamw8() == DP_ERR_ALIAS && launches == 0);
        }
        {
            Lists x(nt);                             // the step control is read
            x.ctrl = (char *)x.p[z] + 4;
            EXPECT(x.adamw() == DP_ERR_ALIAS && launches == 0);
            x.ctrl = (char *)x.g[z];
            EXPECT(x.norm() == DP_ERR_ALIAS && launches == 0);
        }
        {
            Lists x(nt);
            x.ws = (char *)x.g[z] - DP_GRAD_NORM_WS_BYTES + 8;
            EXPECT(x.norm() == DP_ERR_ALIAS && launches == 0);
        }
        {
            Lists x(nt);                             // other refusals
            x.v[z] = nullptr;
            EXPECT(x.adamw() == DP_ERR_INVALID_ARG && x.adamw8() == DP_ERR_INVALID_ARG);
            x = Lists(nt);
            x.n[z] = -1;
            EXPECT(x.adamw() == DP_ERR_INVALID_ARG && x.norm() == DP_ERR_INVALID_ARG);
            x = Lists(nt);
            x.o.flags = DP_ADAMW_STOCHASTIC;
            EXPECT(x.adamw() == DP_ERR_UNSUPPORTED && launches == 0 && x.adamw8() == DP_OK);
            x.o.step = 0;
            EXPECT(x.adamw8() == DP_OK);
            x.ctrl = nullptr;
            EXPECT(x.adamw8() == DP_ERR_INVALID_ARG && launches == 0);
        }
    }
    char *a = (char *)((uintptr_t)1 << 40), *b = a + (1ll << 36), *c = a + (2ll << 36), *d = a + (3ll << 36), *e = a + (4ll << 36);
    const int64_t big = (int64_t)1 << 24;
    launches = 0;
    EXPECT(dp_mxfp4_quantize(a, big, big, big, DP_F32, b, c, nullptr, nullptr, nullptr) == DP_ERR_INVALID_ARG);
    EXPECT(dp_mxfp4_quantize(a, 100, 70, 71, DP_F32, a + 99 * 71 * 4, c, nullptr, nullptr, nullptr) == DP_ERR_INVALID_ARG);
    EXPECT(dp_mxfp4_quantize(a, 100, 70, 71, DP_F32, a + 28112, c, nullptr, nullptr, nullptr) == DP_ERR_ALIAS);
    EXPECT(dp_mxfp4_quantize(a, 100, 70, 71, DP_F32, b, c, b + 64, e, nullptr) == DP_ERR_ALIAS);
    EXPECT(dp_mxfp4_dequantize(a, b, big, big, c, big, DP_F32, nullptr) == DP_ERR_INVALID_ARG);
    EXPECT(dp_mxfp4_dequantize(a, b, 33, 65, a + 33 * 64 - 2, 65, DP_BF16, nullptr) == DP_ERR_ALIAS);
    EXPECT(dp_gemm_mxfp4(a, b, c, d, d + 252, 300, 200, 100, DP_F32, 0, nullptr) == DP_ERR_ALIAS);
    EXPECT(dp_gemm_mxfp4(a, b, c, d, e, big, big, 100, DP_F32, 0, nullptr) == DP_ERR_INVALID_ARG);
    EXPECT(dp_mxfp4_linear(a, 1000, DP_BF16, b, c, d, 5, 100, 1000, DP_F32, d + 16, nullptr) == DP_ERR_ALIAS);
    EXPECT(dp_mxfp4_linear(a, 1000, DP_BF16, b, c, a + 1998, 4, 100, 1000, DP_BF16, nullptr, nullptr) == DP_ERR_ALIAS);
    EXPECT(launches == 0);
    printf("%d failures\n", failures);
    return failures ? 1 : 0;
}
