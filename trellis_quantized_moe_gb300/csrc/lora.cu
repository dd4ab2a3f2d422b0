// The adapters' three products over rows grouped by adapter (include/exl3.h,
// "adapters"): shrink (x A^T, and dy B^T in the backward pass), expand
// (h B, and dh A) and outer (dA, dB).
#include "common.cuh"
#include "lora.h"

namespace exl3 {

namespace {

constexpr int kThreads = 256;

EXL3_DEV float load16(const uint16_t *p, int dtype)
{
    return load_act(p, 0, dtype);
}

EXL3_DEV void store16(void *p, size_t i, int dtype, float v)
{
    if (dtype == EXL3_BF16)
        static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(v);
    else
        static_cast<__half *>(p)[i] = __float2half_rn(v);
}

__global__ void __launch_bounds__(kThreads) k_lora_check(LoraCheckArgs a)
{
    const LoraPlanLayout L = lora_plan_layout(a.M, a.N);
    int err = 0;
    if (a.plan[kLpMagic] != kLoraMagic || a.plan[kLpM] != a.M || a.plan[kLpN] != a.N) {
        err = EXL3_DERR_PLAN;
    } else {
        err = a.plan[kLpError];
        const int32_t *off = a.plan + L.offsets / 4;
        for (int i = threadIdx.x; i < a.N; i += kThreads) {
            if (off[i] == off[i + 1] && !a.GA)
                continue;
            const int r = a.rank[i];
            bool bad = r < 0 || r > a.max_rank;
            if (r > 0) {
                bad |= !a.A[i] || (a.A[i] & 15) || !a.B[i] || (a.B[i] & 15);
                if (a.GA)
                    bad |= !a.GA[i] || (a.GA[i] & 15) || !a.GB[i] || (a.GB[i] & 15);
            }
            err |= bad ? EXL3_DERR_TABLE : 0;
        }
    }
    err = __syncthreads_or(err & EXL3_DERR_TABLE) ? err | EXL3_DERR_TABLE : err;
    if (threadIdx.x == 0)
        a.hdr[kHdrError] = err;
}

// adapter of slot s: the group whose span holds it (N: none)
EXL3_DEV int slot_adapter(const int32_t *off, int N, int s)
{
    int lo = 0, hi = N;                       // last g with off[g] <= s
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (off[mid] <= s)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

// one block per slot, one warp per adapter row
__global__ void __launch_bounds__(kThreads) k_lora_shrink(LoraArgs a)
{
    if (a.hdr[kHdrError])
        return;
    const LoraPlanLayout L = lora_plan_layout(a.M, a.N);
    const int s = blockIdx.x, lane = threadIdx.x & 31;
    const int g = slot_adapter(a.plan + L.offsets / 4, a.N, s);
    const int r = g < a.N ? a.rank[g] : 0;
    const size_t row = (size_t)a.plan[L.perm / 4 + s] * a.width;
    for (int j = threadIdx.x >> 5; j < a.h_cols; j += kThreads / 32) {
        float v = 0.0f;
        if (j < r) {
            const uint16_t *w = reinterpret_cast<const uint16_t *>(a.W[g]) + (size_t)j * a.width;
            for (int i = lane; i < a.width; i += 32)
                v = fmaf(load_act(a.x, row + i, a.act_dtype), load16(w + i, a.act_dtype), v);
#pragma unroll
            for (int m = 16; m; m >>= 1)
                v += __shfl_xor_sync(0xffffffffu, v, m);
            if (a.scaled)
                v *= a.scale[g];
        }
        if (lane == 0)
            store16(a.h, (size_t)s * a.h_cols + j, a.act_dtype, v);
    }
}

// one block per slot, a thread per output
__global__ void __launch_bounds__(kThreads) k_lora_expand(LoraArgs a)
{
    const int s = blockIdx.x;
    if (a.hdr[kHdrError]) {
        for (int n = threadIdx.x; n < a.width; n += kThreads)
            store16(a.y, (size_t)s * a.width + n, a.act_dtype, 0.0f);
        return;
    }
    const LoraPlanLayout L = lora_plan_layout(a.M, a.N);
    const int g = slot_adapter(a.plan + L.offsets / 4, a.N, s);
    const int r = g < a.N ? a.rank[g] : 0;
    const float alpha = g < a.N && a.scaled ? a.scale[g] : 1.0f;
    const uint16_t *w = r ? reinterpret_cast<const uint16_t *>(a.W[g]) : nullptr;
    const size_t row = (size_t)a.plan[L.perm / 4 + s] * a.width;
    for (int n = threadIdx.x; n < a.width; n += kThreads) {
        float v = 0.0f;
        for (int j = 0; j < r; j++)
            v = fmaf(load_act(a.h, (size_t)s * a.h_cols + j, a.act_dtype),
                     load16(w + (size_t)j * a.width + n, a.act_dtype), v);
        const float b = a.base ? load_act(a.base, row + n, a.act_dtype) : 0.0f;
        store16(a.y, row + n, a.act_dtype, fmaf(alpha, v, b));
    }
}

// one block per (adapter, rank row), a thread per column
__global__ void __launch_bounds__(kThreads) k_lora_outer(LoraArgs a)
{
    if (a.hdr[kHdrError])
        return;
    const LoraPlanLayout L = lora_plan_layout(a.M, a.N);
    const int g = blockIdx.x, j = blockIdx.y;
    if (j >= a.rank[g])
        return;
    const int s0 = a.plan[L.offsets / 4 + g], s1 = a.plan[L.offsets / 4 + g + 1];
    const float alpha = a.scaled ? a.scale[g] : 1.0f;
    void *out = reinterpret_cast<void *>(a.G[g]);
    for (int n = threadIdx.x; n < a.width; n += kThreads) {
        float v = 0.0f;
        for (int s = s0; s < s1; s++)
            v = fmaf(load_act(a.h, (size_t)s * a.h_cols + j, a.act_dtype),
                     load_act(a.x, (size_t)a.plan[L.perm / 4 + s] * a.width + n, a.act_dtype), v);
        store16(out, (size_t)j * a.width + n, a.act_dtype, alpha * v);
    }
}

}  // namespace

cudaError_t launch_lora_check(const LoraCheckArgs &a, cudaStream_t s)
{
    k_lora_check<<<1, kThreads, 0, s>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_lora_shrink(const LoraArgs &a, cudaStream_t s)
{
    k_lora_shrink<<<a.M, kThreads, 0, s>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_lora_expand(const LoraArgs &a, cudaStream_t s)
{
    k_lora_expand<<<a.M, kThreads, 0, s>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_lora_outer(const LoraArgs &a, cudaStream_t s)
{
    k_lora_outer<<<dim3(a.N, a.max_rank), kThreads, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace exl3
