// Router: softmax top-k with route weights, balance loss and per-expert
// counts, and the gradient of the logits (include/exl3.h, "router").
//
// Forward, one warp per row: the row's maximum m and s = sum exp(l - m) give
// p_e = exp(l_e - m) / s (kept as the pair: m + log s in fp32 would lose s for
// large |m|); the chosen experts follow one
// another in the order (logit descending, expert ascending), so each is the
// first entry after the previous one.
// Backward, with G_e = dL/dp_e (balance term on valid rows, plus the route
// weights' gradient where they are plain probabilities):
//   dl_e = p_e (G_e - sum_j p_j G_j),
// and renormalised weights w, which depend on the chosen logits only, add
// w_i (d_i - sum_j w_j d_j) at the chosen experts.
#include "common.cuh"
#include "router.h"

namespace exl3 {

namespace {

constexpr int kWarps = 8;

EXL3_DEV float warp_sum(float v)
{
#pragma unroll
    for (int m = 16; m; m >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, m);
    return v;
}

EXL3_DEV void store_float(void *p, size_t i, int dtype, float v)
{
    if (dtype == EXL3_F32)
        static_cast<float *>(p)[i] = v;
    else if (dtype == EXL3_BF16)
        static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(v);
    else
        static_cast<__half *>(p)[i] = __float2half_rn(v);
}

// Unsigned keys in the order of the logits: NaN lowest, then -inf .. +inf,
// with -0 and +0 equal.
EXL3_DEV uint32_t order_key(float l)
{
    if (isnan(l))
        return 0;
    const uint32_t u = __float_as_uint(l + 0.0f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__global__ void __launch_bounds__(kWarps * 32) k_router_forward(RouterArgs a)
{
    const int lane = threadIdx.x & 31;
    const int t = blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (t >= a.M)
        return;
    const size_t row = (size_t)t * a.E;
    float m = -INFINITY;
    for (int e = lane; e < a.E; e += 32)
        m = fmaxf(m, load_act(a.logits, row + e, a.logits_dtype));
#pragma unroll
    for (int d = 16; d; d >>= 1)
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    const float ref = m == -INFINITY ? 0.0f : m;
    float s = 0.0f;
    for (int e = lane; e < a.E; e += 32)
        s += expf(load_act(a.logits, row + e, a.logits_dtype) - ref);
    s = warp_sum(s);
    if (lane == 0 && a.stats)
        reinterpret_cast<float2 *>(a.stats)[t] = make_float2(ref, s);
    // the pairs (key, ~expert) are distinct and ordered as the choice is
    uint64_t prev = ~0ull;
    float w[EXL3_ROUTER_MAX_TOPK], total = 0.0f;
    for (int j = 0; j < a.topk; j++) {
        uint64_t best = 0;
        for (int e = lane; e < a.E; e += 32) {
            const uint64_t k = ((uint64_t)order_key(load_act(a.logits, row + e, a.logits_dtype)) << 32) |
                               (uint32_t)~e;
            if (k < prev && k > best)
                best = k;
        }
#pragma unroll
        for (int d = 16; d; d >>= 1) {
            const uint64_t o = __shfl_xor_sync(0xffffffffu, best, d);
            best = o > best ? o : best;
        }
        prev = best;
        const int e = (int)~(uint32_t)best;
        w[j] = s == 0.0f ? 0.0f : expf(load_act(a.logits, row + e, a.logits_dtype) - ref) / s;
        total += w[j];
        if (lane == 0)
            a.ids[(size_t)t * a.topk + j] = e;
    }
    if (lane == 0) {
        const float norm = a.renorm ? (total == 0.0f ? 1.0f : total) : 1.0f;
        for (int j = 0; j < a.topk; j++)
            store_float(a.rw, (size_t)t * a.topk + j, a.rw_dtype, w[j] / norm);
    }
}

// One block per expert: its count over valid rows, its mean probability, and
// (block E) the number of valid rows.
__global__ void __launch_bounds__(256) k_router_balance(RouterArgs a)
{
    __shared__ float sp[256];
    __shared__ int sc[256], sv[256];
    const int e = blockIdx.x;
    float p = 0.0f;
    int c = 0, v = 0;
    for (int t = threadIdx.x; t < a.M; t += 256) {
        if (a.valid && !a.valid[t])
            continue;
        v++;
        if (e == a.E)
            continue;
        const float2 st = reinterpret_cast<const float2 *>(a.stats)[t];
        p += st.y == 0.0f ? 0.0f : expf(load_act(a.logits, (size_t)t * a.E + e, a.logits_dtype) - st.x) / st.y;
        for (int j = 0; j < a.topk; j++)
            c += a.ids[(size_t)t * a.topk + j] == e;
    }
    sp[threadIdx.x] = p;
    sc[threadIdx.x] = c;
    sv[threadIdx.x] = v;
    for (int h = 128; h; h >>= 1) {
        __syncthreads();
        if (threadIdx.x < h) {
            sp[threadIdx.x] += sp[threadIdx.x + h];
            sc[threadIdx.x] += sc[threadIdx.x + h];
            sv[threadIdx.x] += sv[threadIdx.x + h];
        }
    }
    if (threadIdx.x == 0) {
        a.counts[e] = e == a.E ? sv[0] : sc[0];
        if (e < a.E)
            a.mean[e] = sv[0] ? sp[0] / (float)sv[0] : 0.0f;
    }
}

__global__ void __launch_bounds__(32) k_router_loss(RouterArgs a)
{
    float v = 0.0f;
    for (int e = threadIdx.x; e < a.E; e += 32)
        v += (float)a.counts[e] * a.mean[e];
    v = warp_sum(v);
    const int T = a.counts[a.E];
    if (threadIdx.x == 0)
        *a.loss = T ? (float)a.E / ((float)a.topk * (float)T) * v : 0.0f;
}

__global__ void __launch_bounds__(kWarps * 32) k_router_backward(RouterArgs a)
{
    const int lane = threadIdx.x & 31;
    const int t = blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (t >= a.M)
        return;
    const size_t row = (size_t)t * a.E, rk = (size_t)t * a.topk;
    const float2 st = reinterpret_cast<const float2 *>(a.stats)[t];
    float cg = 0.0f;                // balance gradient of p_e is cg * c_e
    if (a.counts && (!a.valid || a.valid[t])) {
        const float T = (float)a.counts[a.E];
        if (T > 0.0f)
            cg = *a.d_loss * (float)a.E / ((float)a.topk * T * T);
    }
    auto prob = [&](int e) {
        return st.y == 0.0f ? 0.0f : expf(load_act(a.logits, row + e, a.logits_dtype) - st.x) / st.y;
    };
    float total = 0.0f, dot = 0.0f;          // over the chosen: sum p, sum p d
    if (a.d_rw)
        for (int j = 0; j < a.topk; j++) {
            const int e = a.ids[rk + j];
            if ((unsigned)e >= (unsigned)a.E)
                continue;
            const float p = prob(e);
            total += p;
            dot += p * load_act(a.d_rw, rk + j, a.rw_dtype);
        }
    const float inv = a.renorm ? (total == 0.0f ? 0.0f : 1.0f / total) : 1.0f;
    float pg = 0.0f;
    if (a.counts)
        for (int e = lane; e < a.E; e += 32)
            pg += prob(e) * (cg * (float)a.counts[e]);
    pg = warp_sum(pg);
    if (!a.renorm)
        pg += dot;
    for (int e = lane; e < a.E; e += 32) {
        const float p = prob(e);
        float d = p * ((a.counts ? cg * (float)a.counts[e] : 0.0f) - pg);
        if (a.d_rw)
            for (int j = 0; j < a.topk; j++)
                if (a.ids[rk + j] == e) {
                    const float g = load_act(a.d_rw, rk + j, a.rw_dtype);
                    d += a.renorm ? p * inv * (g - dot * inv) : p * g;
                }
        store_float(a.d_logits, row + e, a.logits_dtype, d);
    }
}

}  // namespace

size_t router_workspace_bytes(int M, int E)
{
    (void)M;
    return (((size_t)E + 1 + 2 * (size_t)M) * 4 + 255) / 256 * 256;
}

cudaError_t launch_router_forward(const RouterArgs &a, cudaStream_t s)
{
    if (a.M > 0)
        k_router_forward<<<(a.M + kWarps - 1) / kWarps, kWarps * 32, 0, s>>>(a);
    if (a.counts) {
        k_router_balance<<<a.E + 1, 256, 0, s>>>(a);
        k_router_loss<<<1, 32, 0, s>>>(a);
    }
    return cudaGetLastError();
}

cudaError_t launch_router_backward(const RouterArgs &a, cudaStream_t s)
{
    if (a.M > 0)
        k_router_backward<<<(a.M + kWarps - 1) / kWarps, kWarps * 32, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace exl3
