// Router kernel arguments and launchers (internal).
#pragma once
#include <cuda_runtime_api.h>
#include <stdint.h>

#include "../../include/exl3.h"

namespace exl3 {

struct RouterArgs {
    const void *logits;
    int logits_dtype, M, E, topk, renorm, num_sms;
    int32_t *ids;
    void *rw;
    int rw_dtype;
    float *stats;
    const uint8_t *valid;
    int32_t *counts;
    float *loss;
    float *mean;                    // workspace: f32 [E], mean probability of each expert
    // backward
    const void *d_rw;
    const float *d_loss;
    void *d_logits;
};

size_t router_workspace_bytes(int M, int E);
cudaError_t launch_router_forward(const RouterArgs &a, cudaStream_t s);
cudaError_t launch_router_backward(const RouterArgs &a, cudaStream_t s);

}  // namespace exl3
