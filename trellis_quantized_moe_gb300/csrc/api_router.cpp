// C ABI of the router (include/exl3.h, "router"): checks and launches.
#include <cuda_runtime.h>

#include "host.h"
#include "router.h"

using namespace exl3;

namespace {

int check_sizes(int logits_dtype, int rw_dtype, int M, int E, int topk)
{
    if (!is_float_dtype(logits_dtype) || !is_float_dtype(rw_dtype))
        return EXL3_E_DTYPE;
    if (M < 0 || (long long)M * topk >= (1ll << 30))
        return EXL3_E_SHAPE;
    if (E < 1 || E > EXL3_MAX_EXPERTS || topk < 1 || topk > E || topk > EXL3_ROUTER_MAX_TOPK)
        return EXL3_E_ROUTING;
    return EXL3_OK;
}

}  // namespace

extern "C" {

size_t exl3_router_workspace_bytes(int M, int E)
{
    if (M < 0 || E < 1 || E > EXL3_MAX_EXPERTS)
        return 0;
    return router_workspace_bytes(M, E);
}

int exl3_router_forward(const void *logits, int logits_dtype, int M, int E, int topk, int renorm,
                        int32_t *ids, void *rw, int rw_dtype, float *stats, const uint8_t *valid,
                        int32_t *counts, float *loss, void *ws, size_t ws_bytes, cudaStream_t stream)
{
    int rc = check_sizes(logits_dtype, rw_dtype, M, E, topk);
    if (rc != EXL3_OK)
        return rc;
    if ((M > 0 && (!logits || !ids || !rw)) || !counts != !loss || (counts && !ws))
        return EXL3_E_NULL;
    if (!aligned(logits, 16) || !aligned(ids, 4) || !aligned(rw, float_size(rw_dtype)) || !aligned(stats, 8) ||
        !aligned(counts, 4) || !aligned(loss, 4) || (counts && !aligned(ws, 256)))
        return EXL3_E_ALIGN;
    int dev, sms;
    rc = setup_device(stream, &dev, &sms);
    if (rc != EXL3_OK)
        return rc;
    const void *ptrs[] = {logits, ids, rw, stats, counts ? valid : nullptr, counts, loss, counts ? ws : nullptr};
    for (const void *p : ptrs)
        if (p && !on_device(p, dev))
            return EXL3_E_DEVICE;
    if (counts && ws_bytes < router_workspace_bytes(M, E))
        return EXL3_E_WORKSPACE;
    RouterArgs a{};
    a.logits = logits;
    a.logits_dtype = logits_dtype;
    a.M = M;
    a.E = E;
    a.topk = topk;
    a.renorm = renorm != 0;
    a.num_sms = sms;
    a.ids = ids;
    a.rw = rw;
    a.rw_dtype = rw_dtype;
    a.stats = stats;
    a.valid = valid;
    a.counts = counts;
    a.loss = loss;
    if (counts) {
        a.psum = static_cast<float *>(ws);
        a.pcount = reinterpret_cast<int32_t *>(a.psum + (size_t)router_balance_ctas(M) * E);
    }
    return launch_router_forward(a, stream) == cudaSuccess ? EXL3_OK : EXL3_E_CUDA;
}

int exl3_router_backward(const void *logits, int logits_dtype, int M, int E, int topk, int renorm,
                         const int32_t *ids, const float *stats, const void *d_rw, int rw_dtype,
                         const uint8_t *valid, const int32_t *counts, const float *d_loss, void *d_logits,
                         cudaStream_t stream)
{
    int rc = check_sizes(logits_dtype, rw_dtype, M, E, topk);
    if (rc != EXL3_OK)
        return rc;
    if ((M > 0 && (!logits || !ids || !stats || !d_logits)) || !counts != !d_loss || (!d_rw && !d_loss))
        return EXL3_E_NULL;
    if (!aligned(logits, 16) || !aligned(d_logits, 16) || !aligned(ids, 4) || !aligned(stats, 8) ||
        !aligned(d_rw, float_size(rw_dtype)) || !aligned(counts, 4) || !aligned(d_loss, 4))
        return EXL3_E_ALIGN;
    int dev, sms;
    rc = setup_device(stream, &dev, &sms);
    if (rc != EXL3_OK)
        return rc;
    const void *ptrs[] = {logits, ids, stats, d_rw, counts ? valid : nullptr, counts, d_loss, d_logits};
    for (const void *p : ptrs)
        if (p && !on_device(p, dev))
            return EXL3_E_DEVICE;
    if (M == 0)
        return EXL3_OK;
    RouterArgs a{};
    a.logits = logits;
    a.logits_dtype = logits_dtype;
    a.M = M;
    a.E = E;
    a.topk = topk;
    a.renorm = renorm != 0;
    a.num_sms = sms;
    a.ids = const_cast<int32_t *>(ids);
    a.stats = const_cast<float *>(stats);
    a.rw_dtype = rw_dtype;
    a.d_rw = d_rw;
    a.valid = valid;
    a.counts = const_cast<int32_t *>(counts);
    a.d_loss = d_loss;
    a.d_logits = d_logits;
    return launch_router_backward(a, stream) == cudaSuccess ? EXL3_OK : EXL3_E_CUDA;
}

}  // extern "C"
