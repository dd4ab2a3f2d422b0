// C ABI of the optimiser (include/exl3.h, "optimiser"): checks and launches.
#include <cfloat>
#include <cmath>
#include <cuda_runtime.h>

#include "adamw.h"
#include "host.h"

using namespace exl3;

extern "C" {

size_t exl3_adamw_workspace_bytes(void) { return kAdamwWorkspace; }

int exl3_adamw(const exl3_adamw_tensors *t, double lr, double beta1, double beta2, double eps, double weight_decay,
               const float *lr_scale, const float *grad_scale, int32_t *step, void *ws, size_t ws_bytes,
               cudaStream_t stream)
{
    if (!t || !t->param || !t->grad || !t->m || !t->v || !t->numel || !t->first || !step || !ws)
        return EXL3_E_NULL;
    const bool codes = t->state_dtype == EXL3_E4M3 || t->state_dtype == EXL3_E4M3_RANDOM;
    if (!is_float_dtype(t->param_dtype) || (t->grad_dtype != t->param_dtype && t->grad_dtype != EXL3_F32) ||
        (!codes && t->state_dtype != EXL3_F32) || (t->master && t->param_dtype == EXL3_F32))
        return EXL3_E_DTYPE;
    if (codes ? !t->m_scale || !t->v_scale : t->m_scale || t->v_scale)
        return EXL3_E_NULL;
    if (t->N < 1 || t->blocks < 0 || t->blocks >= (1ll << 33))
        return EXL3_E_SHAPE;
    // what is rounded to float here stays in range there (the rate and its products are
    // known on the device); a NaN fails every comparison
    const auto scalar = [](double x) { return x >= 0 && x <= 1e30; };
    const auto beta = [](double x) { return x >= 0 && (float)x < 1.0f && (float)(1.0 - x) > 0.0f; };
    if (!scalar(lr) || !scalar(weight_decay) || !scalar(eps) || !((float)eps >= FLT_MIN) || !beta(beta1) || !beta(beta2))
        return EXL3_E_VALUE;
    const void *tables[] = {t->param, t->grad, t->m, t->v, t->m_scale, t->v_scale, t->master, t->numel, t->first};
    for (const void *p : tables)
        if (!aligned(p, 8))
            return EXL3_E_ALIGN;
    if (!aligned(lr_scale, 4) || !aligned(grad_scale, 4) || !aligned(step, 4) || !aligned(ws, 256))
        return EXL3_E_ALIGN;
    if (ws_bytes < kAdamwWorkspace)
        return EXL3_E_WORKSPACE;
    int dev, sms;
    const int rc = setup_device(stream, &dev, &sms);
    if (rc != EXL3_OK)
        return rc;
    for (const void *p : tables)
        if (p && !on_device(p, dev))
            return EXL3_E_DEVICE;
    const void *ptrs[] = {lr_scale, grad_scale, step, ws};
    for (const void *p : ptrs)
        if (p && !on_device(p, dev))
            return EXL3_E_DEVICE;
    AdamwArgs a{};
    a.t = *t;
    a.lr = lr;
    a.weight_decay = weight_decay;
    a.log_beta1 = std::log(beta1);
    a.log_beta2 = std::log(beta2);
    a.b1 = (float)beta1;
    a.b2 = (float)beta2;
    a.c1 = (float)(1.0 - beta1);
    a.c2 = (float)(1.0 - beta2);
    a.root_b2 = (float)std::sqrt(beta2);
    a.eps = (float)eps;
    a.lr_scale = lr_scale;
    a.grad_scale = grad_scale;
    a.step = step;
    a.out = static_cast<AdamwScalars *>(ws);
    return launch_adamw(a, stream) == cudaSuccess ? EXL3_OK : EXL3_E_CUDA;
}

}  // extern "C"
