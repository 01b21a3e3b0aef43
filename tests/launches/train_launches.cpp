// Loads libdpsync.so (its path is the argument) and stands in for the HIP
// runtime's launch: a launch is checked against the runtime's limit, fewer than
// 2^32 work-items, and counted, and nothing runs. The device pointers are fake
// addresses that are never dereferenced. Exit status 0 when everything holds.
#include <dlfcn.h>
#include <hip/hip_runtime.h>
#include <stdio.h>
#include <string.h>

#include <vector>

#include "dpsync.h"
#include "optim_internal.h"

static int failures = 0, launches = 0;
static long long groups = 0, tensors_index = 0;
static dim3 grid_, block_;
static size_t shared_;
static hipStream_t stream_;
static bool parts = false, adam = false, eight_bits = false;

#define EXPECT(c)                                              \
    do {                                                       \
        if (!(c)) {                                            \
            fprintf(stderr, "FAIL line %d: %s\n", __LINE__, #c); \
            ++failures;                                        \
        }                                                      \
    } while (0)

extern "C" {

hipError_t __hipPushCallConfiguration(dim3 grid, dim3 block, size_t shared, hipStream_t stream)
{
    grid_ = grid, block_ = block, shared_ = shared, stream_ = stream;
    return hipSuccess;
}
hipError_t __hipPopCallConfiguration(dim3 *grid, dim3 *block, size_t *shared, hipStream_t *stream)
{
    *grid = grid_, *block = block_, *shared = shared_, *stream = stream_;
    return hipSuccess;
}
hipError_t hipLaunchKernel(const void *, dim3 grid, dim3 block, void **args, size_t shared, hipStream_t)
{
    EXPECT(grid.x >= 1 && (unsigned long long)grid.x * block.x < 1ull << 32);
    EXPECT(grid.y == 1 && grid.z == 1 && block.y == 1 && block.z == 1);
    if (adam) {
        // launches of one table of tensors follow one another without a gap; the next table starts again
        const dps::AdamParams *p = (const dps::AdamParams *)args[0];
        const unsigned first = *(const unsigned *)args[1];
        if (p->index0 != tensors_index) groups = 0;
        tensors_index = p->index0;
        EXPECT(first == groups && first + (long long)grid.x <= p->first[p->nt]);
        // fp32 states: two workgroups a CU, except where eight take all the chunks at once
        EXPECT(shared == (!eight_bits && p->first[p->nt] > 2048 ? 80u << 10 : 0u));
    } else if (parts) {
        // the last argument is the first workgroup's number
        EXPECT(*(const unsigned *)args[1] == groups || *(const unsigned *)args[2] == groups);
    }
    groups += grid.x;
    ++launches;
    return hipSuccess;
}
hipError_t hipGetLastError() { return hipSuccess; }

}  // extern "C"

static void fresh()
{
    launches = 0;
    groups = tensors_index = 0;
}

int main(int, char **argv)
{
    void *lib = dlopen(argv[1], RTLD_NOW);
    if (!lib) {
        fprintf(stderr, "%s\n", dlerror());
        return 2;
    }
#define CALL(name) ((decltype(&name))dlsym(lib, #name))
    char *a = (char *)((uintptr_t)1 << 44), *b = a + (1ll << 42), *c = a + (2ll << 42), *d = a + (3ll << 42), *e = a + (4ll << 42);
    const int64_t one = 1;

    // AdamW: 2^35 elements and more are 2^24 chunks of 2048
    adam = true;
    for (int64_t n : {one, one << 20, 2048 * 2048 * one, 2048 * 2048 * one + 1, (one << 35) - 2048, one << 35, (one << 35) + 5, one << 37}) {
        void *p = a, *g = b, *m = c, *v = d, *s = e;
        dp_adamw_opts_t o = {1e-3, 0.9, 0.999, 1e-8, 0.01, 3, 7, 0, 0};
        for (bool eight : {false, true}) {
            fresh();
            eight_bits = eight;
            if (eight) {
                o.flags = DP_ADAMW_STOCHASTIC;
                EXPECT(CALL(dp_adamw8)(1, &n, &p, DP_BF16, &g, DP_BF16, (uint8_t **)&m, (uint8_t **)&v, (float **)&s, nullptr, &o, nullptr, nullptr) == DP_OK);
            } else {
                EXPECT(CALL(dp_adamw)(1, &n, &p, DP_F32, &g, DP_F32, (float **)&m, (float **)&v, nullptr, &o, nullptr, nullptr) == DP_OK);
            }
            EXPECT(groups == (n + 2047) / 2048);
            EXPECT(launches == (groups + (1 << 24) - 2) / ((1 << 24) - 1));
        }
    }
    {
        // 100 tensors, the first 64 of them beyond one launch
        std::vector<int64_t> n(100, one << 30);
        std::vector<void *> p(100), g(100, b), m(100), v(100);
        for (int i = 0; i < 100; ++i) p[i] = c + (one << 34) * i, m[i] = d + (one << 34) * i, v[i] = e + (one << 34) * i;
        dp_adamw_opts_t o = {1e-3, 0.9, 0.999, 1e-8, 0.01, 3, 7, 0, 0};
        fresh();
        eight_bits = false;
        EXPECT(CALL(dp_adamw)(100, n.data(), p.data(), DP_F32, g.data(), DP_F32, (float **)m.data(), (float **)v.data(), nullptr, &o, nullptr, nullptr) == DP_OK);
        EXPECT(launches == 5 && tensors_index == 64 && groups == 36ll << 19);   // 2^25 chunks in three, 36 x 2^19 in two
    }
    adam = false;

    // expansion: a thread takes 8 elements
    parts = true;
    for (int64_t rows : {one, one << 20, one << 21, (one << 21) + 1, one << 24}) {
        fresh();
        EXPECT(CALL(dp_mxfp4_dequantize)(a, c, rows, 1 << 14, e, 1 << 14, DP_BF16, nullptr) == DP_OK);
        EXPECT(groups == rows * 8);
        EXPECT(launches == (groups + (1 << 24) - 2) / ((1 << 24) - 1));
    }
    // product of short rows: workgroups of 64 x 16 outputs, any sizes that are accepted
    for (int64_t m : {one << 10, one << 17, (one << 17) + 1, one << 20, one << 24})
        for (int64_t n : {one << 13, (one << 13) + 1, one << 17}) {
            fresh();
            const dp_status_t s = CALL(dp_gemm_mxfp4)(a, b, c, d, e, m, n, 64, DP_BF16, 0, nullptr);
            EXPECT(s == (m * n <= one << 37 ? DP_OK : DP_ERR_INVALID_ARG));
            if (s == DP_OK) EXPECT(groups == (m + 63) / 64 * ((n + 15) / 16));
        }
    parts = false;
    // tiled product, narrow and square, up to the largest output
    for (int64_t m : {one << 6, (one << 13) + 1, one << 19, one << 24})
        for (int64_t n : {one << 6, one << 13, one << 18, one << 24}) {
            fresh();
            const dp_status_t s = CALL(dp_gemm_mxfp4)(a, b, c, d, e, m, n, 512, DP_BF16, 0, nullptr);
            EXPECT(s == (m * n <= one << 37 ? DP_OK : DP_ERR_INVALID_ARG));
            EXPECT((launches > 0) == (s == DP_OK));
        }
    // quantisation: pieces of 16 x 512 along the rows, of 128 x 128 otherwise
    struct { int64_t rows, cols; bool t, fine; } q[] = {
        {one << 24, 8192 - 512, false, true}, {one << 24, 8192, false, false}, {1, one << 24, false, true},
        {one << 24, 128 * 127, true, true}, {one << 24, 128 * 128, true, false}, {(one << 20) - 128, 128 << 11, true, true},
        {one << 20, 128 << 11, true, false}};
    for (const auto &x : q) {
        fresh();
        const dp_status_t s = CALL(dp_mxfp4_quantize)(a, x.rows, x.cols, x.cols, DP_BF16, b, c, x.t ? d : nullptr, x.t ? e : nullptr, nullptr);
        EXPECT(s == (x.fine ? DP_OK : DP_ERR_INVALID_ARG) && launches == (x.fine ? 1 : 0));
    }
    printf("%d failures\n", failures);
    return failures ? 1 : 0;
}
