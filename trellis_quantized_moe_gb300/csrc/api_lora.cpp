// C ABI of the adapters (include/exl3.h, "adapters"): checks and launches.
#include <cuda_runtime.h>

#include "host.h"
#include "lora.h"

using namespace exl3;

namespace {

bool sizes_ok(int M, int N, int in_f, int out_f, int max_rank)
{
    return M >= 0 && M < (1 << 30) && N >= 1 && N <= EXL3_MAX_ADAPTERS && in_f > 0 && out_f > 0 &&
           in_f % kHb == 0 && out_f % kHb == 0 && in_f < (1 << 24) && out_f < (1 << 24) && max_rank >= 1 &&
           max_rank <= EXL3_MAX_RANK;
}

int check_adapters(const exl3_adapters *ad)
{
    if (!ad || !ad->A || !ad->B)
        return EXL3_E_NULL;
    if (!aligned(ad->A, 8) || !aligned(ad->B, 8) || !aligned(ad->rank, 4) || !aligned(ad->scale, 4))
        return EXL3_E_ALIGN;
    return EXL3_OK;
}

// What forward and backward share: dtype, tables, sizes, plan, workspace.
int check_call(int act_dtype, int M, const exl3_adapters *ad, const void *plan, void *ws, size_t ws_bytes)
{
    int rc = check_adapters(ad);
    if (rc != EXL3_OK)
        return rc;
    if (!ad->rank || !ad->scale || !plan || !ws)
        return EXL3_E_NULL;
    if (!is_act_dtype(act_dtype))
        return EXL3_E_DTYPE;
    if (!sizes_ok(M, ad->N, ad->in_features, ad->out_features, ad->max_rank))
        return EXL3_E_SHAPE;
    if (!aligned(plan, 256) || !aligned(ws, 256))
        return EXL3_E_ALIGN;
    if (ws_bytes < lora_ws_layout(M, ad->N, ad->in_features, ad->out_features, ad->max_rank).total)
        return EXL3_E_WORKSPACE;
    return EXL3_OK;
}

LoraArgs common_args(int act_dtype, int M, const exl3_adapters *ad, const void *plan, void *ws, int sms)
{
    LoraArgs a{};
    a.plan = static_cast<const int32_t *>(plan);
    a.M = M;
    a.N = ad->N;
    a.act_dtype = act_dtype;
    a.max_rank = ad->max_rank;
    a.h_cols = lora_h_cols(ad->max_rank);
    a.num_sms = sms;
    a.rank = ad->rank;
    a.scale = ad->scale;
    a.hdr = static_cast<int32_t *>(ws);
    return a;
}

LoraCheckArgs table_check(int M, const exl3_adapters *ad, const exl3_adapters *grads, const void *plan, void *ws)
{
    LoraCheckArgs c{};
    c.plan = static_cast<const int32_t *>(plan);
    c.M = M;
    c.N = ad->N;
    c.max_rank = ad->max_rank;
    c.A = ad->A;
    c.B = ad->B;
    c.GA = grads ? grads->A : nullptr;
    c.GB = grads ? grads->B : nullptr;
    c.rank = ad->rank;
    c.hdr = static_cast<int32_t *>(ws);
    return c;
}

}  // namespace

extern "C" {

size_t exl3_lora_plan_bytes(int M, int N)
{
    return sizes_ok(M, N, kHb, kHb, 1) ? lora_plan_layout(M, N).total : 0;
}

int exl3_lora_h_cols(int max_rank)
{
    return max_rank >= 1 && max_rank <= EXL3_MAX_RANK ? lora_h_cols(max_rank) : 0;
}

size_t exl3_lora_workspace_bytes(int M, int N, int in_features, int out_features, int max_rank)
{
    if (!sizes_ok(M, N, in_features, out_features, max_rank))
        return 0;
    return lora_ws_layout(M, N, in_features, out_features, max_rank).total;
}

int exl3_lora_plan(const void *ids, int ids_dtype, int M, int N, void *plan, size_t plan_bytes,
                   cudaStream_t stream)
{
    if (!plan || (M > 0 && !ids))
        return EXL3_E_NULL;
    if (ids_dtype != EXL3_I32 && ids_dtype != EXL3_I64)
        return EXL3_E_DTYPE;
    if (!sizes_ok(M, N, kHb, kHb, 1))
        return EXL3_E_SHAPE;
    if (!aligned(plan, 256) || !aligned(ids, ids_dtype == EXL3_I64 ? 8 : 4))
        return EXL3_E_ALIGN;
    if (plan_bytes < lora_plan_layout(M, N).total)
        return EXL3_E_WORKSPACE;
    int dev, sms;
    const int rc = setup_device(stream, &dev, &sms);
    if (rc != EXL3_OK)
        return rc;
    if (!on_device(plan, dev) || (M > 0 && !on_device(ids, dev)))
        return EXL3_E_DEVICE;
    LoraPlanArgs a{};
    a.ids = ids;
    a.M = M;
    a.N = N;
    a.plan = static_cast<int32_t *>(plan);
    return launch_lora_plan(a, ids_dtype, stream) == cudaSuccess ? EXL3_OK : EXL3_E_CUDA;
}

int exl3_lora_forward(const void *x, int act_dtype, int M, const exl3_adapters *ad, const void *plan,
                      const void *base, void *y, void *h, void *ws, size_t ws_bytes, cudaStream_t stream)
{
    int rc = check_call(act_dtype, M, ad, plan, ws, ws_bytes);
    if (rc != EXL3_OK)
        return rc;
    if (M > 0 && (!x || !y))
        return EXL3_E_NULL;
    if (!aligned(x, 16) || !aligned(base, 16) || !aligned(y, 16) || !aligned(h, 16))
        return EXL3_E_ALIGN;
    int dev, sms;
    rc = setup_device(stream, &dev, &sms);
    if (rc != EXL3_OK)
        return rc;
    const void *ptrs[] = {x, base, y, h, plan, ws, ad->A, ad->B, ad->rank, ad->scale};
    for (const void *p : ptrs)
        if (p && !on_device(p, dev))
            return EXL3_E_DEVICE;
    if (M == 0)
        return EXL3_OK;
    const LoraWsLayout L = lora_ws_layout(M, ad->N, ad->in_features, ad->out_features, ad->max_rank);
    if (launch_lora_check(table_check(M, ad, nullptr, plan, ws), stream) != cudaSuccess)
        return EXL3_E_CUDA;
    LoraArgs a = common_args(act_dtype, M, ad, plan, ws, sms);
    a.h = h ? h : static_cast<uint8_t *>(ws) + L.h;
    a.x = x;
    a.W = ad->A;
    a.width = ad->in_features;
    if (launch_lora_shrink(a, stream) != cudaSuccess)
        return EXL3_E_CUDA;
    a.W = ad->B;
    a.width = ad->out_features;
    a.scaled = 1;
    a.base = base;
    a.y = y;
    return launch_lora_expand(a, stream) == cudaSuccess ? EXL3_OK : EXL3_E_CUDA;
}

int exl3_lora_backward(const void *dy, const void *x, const void *h, int act_dtype, int M,
                       const exl3_adapters *ad, const void *plan, const void *dx_base, void *dx,
                       const exl3_adapters *grads, void *ws, size_t ws_bytes, cudaStream_t stream)
{
    int rc = check_call(act_dtype, M, ad, plan, ws, ws_bytes);
    if (rc != EXL3_OK)
        return rc;
    if ((!dx && !grads) || (M > 0 && (!dy || (grads && (!x || !h)))))
        return EXL3_E_NULL;
    if (grads) {
        rc = check_adapters(grads);
        if (rc != EXL3_OK)
            return rc;
        if (grads->N != ad->N || grads->in_features != ad->in_features ||
            grads->out_features != ad->out_features)
            return EXL3_E_SHAPE;
    }
    if (!aligned(dy, 16) || !aligned(x, 16) || !aligned(h, 16) || !aligned(dx_base, 16) || !aligned(dx, 16))
        return EXL3_E_ALIGN;
    int dev, sms;
    rc = setup_device(stream, &dev, &sms);
    if (rc != EXL3_OK)
        return rc;
    const void *ptrs[] = {dy, x, h, dx_base, dx, plan, ws, ad->A, ad->B, ad->rank, ad->scale,
                          grads ? grads->A : nullptr, grads ? grads->B : nullptr};
    for (const void *p : ptrs)
        if (p && !on_device(p, dev))
            return EXL3_E_DEVICE;
    if (M == 0 && !grads)
        return EXL3_OK;
    const LoraWsLayout L = lora_ws_layout(M, ad->N, ad->in_features, ad->out_features, ad->max_rank);
    if (launch_lora_check(table_check(M, ad, grads, plan, ws), stream) != cudaSuccess)
        return EXL3_E_CUDA;
    LoraArgs a = common_args(act_dtype, M, ad, plan, ws, sms);
    void *dh = static_cast<uint8_t *>(ws) + L.h;
    if (M > 0) {
        a.h = dh;
        a.x = dy;
        a.W = ad->B;
        a.width = ad->out_features;
        a.scaled = 1;
        if (launch_lora_shrink(a, stream) != cudaSuccess)
            return EXL3_E_CUDA;
    }
    if (M > 0 && dx) {
        a.W = ad->A;
        a.width = ad->in_features;
        a.scaled = 0;
        a.base = dx_base;
        a.y = dx;
        if (launch_lora_expand(a, stream) != cudaSuccess)
            return EXL3_E_CUDA;
    }
    if (grads) {
        a.h = dh;
        a.x = x;
        a.G = grads->A;
        a.width = ad->in_features;
        a.scaled = 0;
        if (launch_lora_outer(a, stream) != cudaSuccess)
            return EXL3_E_CUDA;
        a.h = const_cast<void *>(h);
        a.x = dy;
        a.G = grads->B;
        a.width = ad->out_features;
        a.scaled = 1;
        if (launch_lora_outer(a, stream) != cudaSuccess)
            return EXL3_E_CUDA;
    }
    return EXL3_OK;
}

}  // extern "C"
