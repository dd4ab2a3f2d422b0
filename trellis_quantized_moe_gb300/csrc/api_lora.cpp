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
           max_rank <= EXL3_MAX_RANK &&
           ((long long)M / 64 + N) * ((in_f + out_f) / 64) < (1ll << 31);   // work items are counted in 32 bits
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
int check_call(int act_dtype, int M, const exl3_adapters *ad, const void *plan, size_t plan_bytes, void *ws,
               size_t ws_bytes)
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
    if (plan_bytes < lora_plan_layout(M, ad->N).total ||
        ws_bytes < lora_ws_layout(M, ad->N, ad->in_features, ad->out_features, ad->max_rank).total)
        return EXL3_E_WORKSPACE;
    return EXL3_OK;
}

// One CTA per SM shares a product's work; the workspace knows kLoraCtas of them.
int product_ctas(int sms) { return sms < kLoraCtas ? sms : kLoraCtas; }

// Rows up to which one launch does both products.  It reads a weight once per
// eight rows (from L2), the products' own kernels once per 128, at the price of
// two launches and partial sums between them.  GPU time of a call, one launch /
// two (bf16, us): 5120 -> 1536, rank 16: 1 row 4.3 / 10.8, 512 rows 7.2 / 13.8,
// 1024 rows 10.8 / 16.7, 1500 rows 17.5 / 17.7, 2048 rows 19.6 / 19.5, 4096 rows
// 37.6 / 25.3; rank 64: 1024 rows 19.7 / 20.7, 1500 rows 33.1 / 21.6; 1536 ->
// 5120: rank 16, 1024 rows 13.3 / 17.7, 1500 rows 23.2 / 19.0.  Its registers hold
// less of a wide adapter: 2048 -> 2048, rank 128: 512 rows 17.9 / 19.6, 1024 rows
// 26.0 / 21.1.
int rows_max(int max_rank) { return max_rank <= 64 ? 1024 : 512; }

// h = h_scale * W1 x, y = base + y_scale * h W2 of a batch (scale_h: the
// adapter's scale goes to h instead of y), and the check of the tables.
struct Products {
    const void *x;
    const int64_t *W1, *W2;
    int in_width, out_width, scale_h;
    const void *base;
    void *y, *h;
};

LoraRowsArgs rows_args(const Products &p, int act_dtype, int M, const exl3_adapters *ad, const exl3_adapters *grads,
                       const void *plan, void *ws)
{
    LoraRowsArgs a{};
    a.plan = static_cast<const int32_t *>(plan);
    a.M = M;
    a.N = ad->N;
    a.act_dtype = act_dtype;
    a.max_rank = ad->max_rank;
    a.h_cols = lora_h_cols(ad->max_rank);
    a.in_width = p.in_width;
    a.out_width = p.out_width;
    a.scale_h = p.scale_h;
    a.x = p.x;
    a.W1 = p.W1;
    a.W2 = p.W2;
    a.GA = grads ? grads->A : nullptr;
    a.GB = grads ? grads->B : nullptr;
    a.rank = ad->rank;
    a.scale = ad->scale;
    a.base = p.base;
    a.y = p.y;
    a.h = p.h;
    a.hdr = static_cast<int32_t *>(ws);
    return a;
}

// The first product and its join.
cudaError_t run_shrink(const Products &p, int act_dtype, int M, const exl3_adapters *ad, const exl3_adapters *grads,
                       const void *plan, void *ws, const LoraWsLayout &L, int ctas, cudaStream_t stream)
{
    LoraShrinkArgs sh{};
    sh.plan = static_cast<const int32_t *>(plan);
    sh.M = M;
    sh.N = ad->N;
    sh.act_dtype = act_dtype;
    sh.max_rank = ad->max_rank;
    sh.h_cols = lora_h_cols(ad->max_rank);
    sh.width = p.in_width;
    sh.x = p.x;
    sh.W = p.W1;
    sh.rank = ad->rank;
    sh.part = reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + L.part);
    sh.A = ad->A;
    sh.B = ad->B;
    sh.GA = grads ? grads->A : nullptr;
    sh.GB = grads ? grads->B : nullptr;
    sh.hdr = static_cast<int32_t *>(ws);
    const cudaError_t e = launch_lora_shrink(sh, ctas, stream);
    if (e != cudaSuccess)
        return e;
    LoraJoinArgs jn{};
    jn.plan = sh.plan;
    jn.M = M;
    jn.N = sh.N;
    jn.act_dtype = act_dtype;
    jn.h_cols = sh.h_cols;
    jn.scale_h = p.scale_h;
    jn.part = sh.part;
    jn.shrink_width = sh.width;
    jn.shrink_ctas = ctas;
    jn.rank = ad->rank;
    jn.scale = ad->scale;
    jn.h = p.h;
    jn.hdr = sh.hdr;
    return launch_lora_join(jn, stream);
}

// The second product.
cudaError_t run_expand(const Products &p, int act_dtype, int M, const exl3_adapters *ad, const void *plan, void *ws,
                       int ctas, cudaStream_t stream)
{
    LoraExpandArgs ex{};
    ex.plan = static_cast<const int32_t *>(plan);
    ex.M = M;
    ex.N = ad->N;
    ex.act_dtype = act_dtype;
    ex.h_cols = lora_h_cols(ad->max_rank);
    ex.width = p.out_width;
    ex.scale_h = p.scale_h;
    ex.h = p.h;
    ex.W = p.W2;
    ex.rank = ad->rank;
    ex.scale = ad->scale;
    ex.base = p.base;
    ex.y = p.y;
    ex.hdr = static_cast<int32_t *>(ws);
    return launch_lora_expand(ex, ctas, stream);
}

LoraOuterArgs outer_args(int act_dtype, int M, const exl3_adapters *ad, const void *plan, void *ws,
                         const LoraWsLayout &L, int ctas)
{
    LoraOuterArgs o{};
    o.plan = static_cast<const int32_t *>(plan);
    o.M = M;
    o.N = ad->N;
    o.act_dtype = act_dtype;
    o.h_cols = lora_h_cols(ad->max_rank);
    o.ctas = ctas;
    o.rank = ad->rank;
    o.scale = ad->scale;
    o.part = reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + L.part);
    o.hdr = static_cast<int32_t *>(ws);
    return o;
}

}  // namespace

extern "C" {

size_t exl3_lora_plan_bytes(int M, int N)
{
    return sizes_ok(M, N, kHb, kHb, 1) ? lora_plan_layout(M, N).total : 0;
}

int exl3_lora_h_cols(int max_rank)
{
    return max_rank >= 1 && max_rank <= EXL3_MAX_RANK ? lora_h_pitch(lora_h_cols(max_rank)) : 0;
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
                      size_t plan_bytes, const void *base, void *y, void *h, void *ws, size_t ws_bytes, cudaStream_t stream)
{
    int rc = check_call(act_dtype, M, ad, plan, plan_bytes, ws, ws_bytes);
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
    const Products p{x, ad->A, ad->B, ad->in_features, ad->out_features, 0, base, y,
                     h ? h : static_cast<uint8_t *>(ws) + L.h};
    const int ctas = product_ctas(sms);
    cudaError_t e;
    if (M <= rows_max(ad->max_rank)) {
        e = launch_lora_rows(rows_args(p, act_dtype, M, ad, nullptr, plan, ws), sms, stream);
    } else {
        e = run_shrink(p, act_dtype, M, ad, nullptr, plan, ws, L, ctas, stream);
        if (e == cudaSuccess)
            e = run_expand(p, act_dtype, M, ad, plan, ws, ctas, stream);
    }
    return e == cudaSuccess ? EXL3_OK : EXL3_E_CUDA;
}

int exl3_lora_backward(const void *dy, const void *x, const void *h, int act_dtype, int M,
                       const exl3_adapters *ad, const void *plan, size_t plan_bytes, const void *dx_base, void *dx,
                       const exl3_adapters *grads, void *ws, size_t ws_bytes, cudaStream_t stream)
{
    int rc = check_call(act_dtype, M, ad, plan, plan_bytes, ws, ws_bytes);
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
    const int ctas = product_ctas(sms);
    void *dh = static_cast<uint8_t *>(ws) + L.h;
    const Products p{dy, ad->B, ad->A, ad->out_features, ad->in_features, 1, dx_base, dx, dh};
    LoraOuterArgs o = outer_args(act_dtype, M, ad, plan, ws, L, ctas);
    if (grads) {
        o.p[0] = {x, dh, grads->A, ad->in_features, 0};
        o.p[1] = {dy, h, grads->B, ad->out_features, 1};
    }
    cudaError_t e;
    if (M <= rows_max(ad->max_rank)) {
        e = launch_lora_rows(rows_args(p, act_dtype, M, ad, grads, plan, ws), sms, stream);
        if (e == cudaSuccess && grads)
            e = launch_lora_outer(o, stream);
    } else {
        // the weights' gradients first, while dy is in L2 (8192 rows, ranks 64
        // and 128: 1 us)
        e = run_shrink(p, act_dtype, M, ad, grads, plan, ws, L, ctas, stream);
        if (e == cudaSuccess && grads)
            e = launch_lora_outer(o, stream);
        if (e == cudaSuccess && dx)
            e = run_expand(p, act_dtype, M, ad, plan, ws, ctas, stream);
    }
    return e == cudaSuccess ? EXL3_OK : EXL3_E_CUDA;
}

}  // extern "C"
