// Dispatch and combine: kernel arguments and launchers (internal).
#pragma once
#include <cuda_runtime_api.h>
#include <stdint.h>

#include "../../include/exl3.h"

namespace exl3 {

constexpr int kPlanCluster = 16;        // CTAs of one cluster at most
constexpr int kPlanCtas = 128;          // CTAs by themselves at most
constexpr int kPlanCounts = 65536;      // their counts at most, but one of each

// Threads of a CTA of the plan for R routes.  Few of them where there are few routes:
// barriers, counters to clear and to add up go by the warps (192 experts, 256 / 512 /
// 1024 threads: 8 routes 2.0 / 2.4 / 3.6 us, 2040 3.4 / 4.0 / 5.2, 8000 4.6 / 4.8 / 5.4,
// 16000 5.6 / 5.6 / 6.0 (1024 experts 10.6 / 9.4 / 10.0), 32000 9.2 / 7.3 / 7.5, 524288
// 59 / 39 / 17).
inline int dispatch_plan_threads(int R) { return R <= 8192 ? 256 : R <= 32768 ? 512 : 1024; }

// CTAs that share R routes of E experts: up to 32768 routes in one cluster, a power of
// two that leaves each at most 512 routes (or 16 of them).  Above, one for each 1024
// routes, up to 128, fewer for many experts, as each reads all CTAs' counts (524288
// routes, 128 / 64 / 32 CTAs: 192 experts 17 / 24 / - us, 1024 experts 47 / 40 / 53).
inline int dispatch_plan_ctas(int R, int E)
{
    if (R <= 32768) {
        int n = 1;
        while (n < kPlanCluster && R > n * 512)
            n *= 2;
        return n;
    }
    const int all = (R + 1023) / 1024, fit = kPlanCounts / (E + 1), most = fit > kPlanCtas ? kPlanCtas : fit;
    return all < most ? all : most;
}

// Workspace: its first word is the call's error word; then int [ctas][E + 2], the
// CTAs' counts, where they are no cluster.  The bytes are a bound that never falls
// as M, topk or E grows, though the CTAs get fewer for many experts: what counts is
// that ctas (E + 1) <= kPlanCounts and ctas <= kPlanCtas.
constexpr int kPlanHeader = 64;

inline size_t dispatch_plan_bytes(int R, int E)
{
    const int n = R <= 32768 ? 0 : R >= kPlanCtas * 1024 ? kPlanCtas : (R + 1023) / 1024;
    const int all = n * (E + 2), most = kPlanCounts + n;
    return ((size_t)(kPlanHeader + (all < most ? all : most)) * 4 + 255) / 256 * 256;
}

struct DispatchPlanArgs {
    const void *ids;
    int R, E, ctas, threads;
    int32_t *offsets, *packed, *slots, *experts, *hdr, *counts;
};

struct RowsArgs {
    int M, topk, width, dtype, rw_dtype;
    const int32_t *slots;
    const void *x;                  // dispatch: rows of the tokens; combine: base; backward: d_out
    const void *y;                  // rows in expert order
    const void *rw;
    void *rows;                     // written rows in expert order
    void *out;                      // combine: rows of the tokens; backward: d_rw
};

cudaError_t dispatch_set_attributes();
cudaError_t launch_dispatch_plan(const DispatchPlanArgs &a, int ids_dtype, cudaStream_t s);
cudaError_t launch_dispatch(const RowsArgs &a, cudaStream_t s);
cudaError_t launch_combine(const RowsArgs &a, cudaStream_t s);
cudaError_t launch_combine_backward(const RowsArgs &a, cudaStream_t s);

}  // namespace exl3
