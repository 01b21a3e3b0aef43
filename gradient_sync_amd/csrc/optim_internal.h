// Internal declarations of the optimizer kernels (global gradient norm and
// AdamW over many tensors), shared by optim_kernels.hip and the entry points.
#pragma once

#include "dps_internal.h"

namespace dps {

// Workspace of the norm: one partial sum per workgroup, then the ticket that
// tells the last workgroup to finish.
constexpr int kNormMaxGrid = 512;
constexpr size_t kNormWsBytes = kNormMaxGrid * sizeof(double) + 64;

// Device-side step control, laid out as dp_step_ctrl_t.
struct StepCtrl {
    float norm, scale;
    int step, skipped;
};

constexpr int kNormTensors = 128;
struct NormParams {
    const char *g[kNormTensors];
    long long n[kNormTensors];
    int first[kNormTensors + 1];    // first chunk of tensor i in this launch
    int nt;
    int add;                        // add to the partials of an earlier launch
    int finish;                     // the call's last launch: the last workgroup sums up
    double max_norm;
    double *partial;
    unsigned *ticket;
    StepCtrl *ctrl;
};
long long norm_chunks(long long n);
// grid: the same for every launch of a call
hipError_t launch_grad_norm(const NormParams &p, int dt, int grid, hipStream_t stream);

constexpr int kAdamTensors = 64;
constexpr int kStateBlock = 128;    // elements that share an 8-bit state's scales
struct AdamTensor {
    char *p;
    const char *g;
    char *m, *v;
    char *copy;                     // bf16, or NULL
    float *scales;                  // 8-bit states: (m scale, sqrt(v) scale) per block
    long long n;
};
struct AdamParams {
    AdamTensor t[kAdamTensors];
    int first[kAdamTensors + 1];
    int nt;
    int index0;                     // number of t[0] within the call (seeds the rounding)
    float beta1, beta2, one_minus_beta1, one_minus_beta2, eps, decay;
    float step_size, inv_sqrt_bc2;  // used when step > 0
    double lr, dbeta1, dbeta2;      // used when step == 0 (step taken from ctrl)
    long long step;
    unsigned long long seed;
    const StepCtrl *ctrl;           // or NULL
};
long long adam_chunks(long long n);
hipError_t launch_adamw(const AdamParams &p, int p_dt, int g_dt, bool eight, bool stochastic,
                        hipStream_t stream);

}  // namespace dps
