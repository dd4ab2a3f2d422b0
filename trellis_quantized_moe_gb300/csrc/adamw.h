// AdamW over many tensors: kernel arguments and launchers (internal).
#pragma once
#include <cuda_runtime_api.h>
#include <stdint.h>

#include "../../include/exl3.h"

namespace exl3 {

constexpr int kAdamwBlock = EXL3_ADAMW_BLOCK;
constexpr size_t kAdamwWorkspace = 256;

// What the step's first kernel leaves in the workspace, after the error word.
struct AdamwScalars {
    int32_t error, run;             // run: 1 when the step is made, 0 when it is left out
    float decay;                    // 1 - rate wd
    float rate;                     // - rate / (1 - beta1^t)
    float root;                     // 1 / sqrt(1 - beta2^t)
    float grad;                     // grad_scale
    float second;                   // grad_scale sqrt(1 - beta2)
    uint32_t seed;                  // of the step's random roundings
};

struct AdamwArgs {
    exl3_adamw_tensors t;
    double lr, weight_decay, log_beta1, log_beta2;
    float b1, b2, c1, c2, root_b2, eps;     // c1 = 1 - beta1, c2 = 1 - beta2, root_b2 = sqrt(beta2)
    const float *lr_scale, *grad_scale;
    int32_t *step;
    AdamwScalars *out;
};

cudaError_t adamw_set_attributes();
cudaError_t launch_adamw(const AdamwArgs &a, cudaStream_t s);

}  // namespace exl3
