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
    float *psum;                    // workspace: f32 [ctas][E], each CTA's sum of probabilities
    int32_t *pcount;                // workspace: int32 [ctas][E + 1], its counts and valid rows
    // backward
    const void *d_rw;
    const float *d_loss;
    void *d_logits;
};

// CTAs of the balance pass at most: two of 16 warps per SM.
constexpr int kRouterCtas = 304;
constexpr int kRouterWarps = 16;
// Balance of at most this many rows: one CTA does it all, two rows a warp, with
// no second kernel (288 experts, fp32, the forward pass: 16 rows 4.5 us, 32 rows
// 7.1; 48 rows 9.6 so and 8.6 with the join, 64 rows 12.1 and 8.6, 128 rows 22.2
// and 8.6).
constexpr int kRouterOneCta = 32;

inline int router_balance_ctas(int M)
{
    if (M <= kRouterOneCta)
        return M > 0;
    const int n = (M + kRouterWarps - 1) / kRouterWarps;
    return n < kRouterCtas ? n : kRouterCtas;
}

size_t router_workspace_bytes(int M, int E);
cudaError_t router_set_attributes();
cudaError_t launch_router_forward(const RouterArgs &a, cudaStream_t s);
cudaError_t launch_router_backward(const RouterArgs &a, cudaStream_t s);

}  // namespace exl3
