// Router: softmax top-k with route weights, balance loss and per-expert
// counts, and the gradient of the logits (include/exl3.h, "router").
//
// A warp owns a row: lane l holds the logits of experts l, l + 32, ... in
// registers, so the row is read once.  Forward: m = max l, s = sum exp(l - m),
// p_e = exp(l_e - m) / s (kept as the pair: m + log s in fp32 would lose s for
// large |m|); then topk rounds of a warp-wide maximum over order-preserving
// integer keys, ties to the lower expert.  Backward, with G_e = dL/dp_e
// (balance term on valid rows, plus the route weights' gradient where they are
// plain probabilities):
//   dl_e = p_e (G_e - sum_j p_j G_j),
// and renormalised weights w, which depend on the chosen logits only, add
// w_i (d_i - sum_j w_j d_j) at the chosen experts.
//
// What bounds it: not HBM but the instructions of the topk rounds (about 30
// per round and row at 192 experts).
#include <type_traits>

#include "common.cuh"
#include "router.h"

namespace exl3 {

namespace {

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

// Keys in the order of the logits, never 0 (0: no expert, or taken): NaN
// lowest, then -inf .. +inf, with -0 and +0 equal.
EXL3_DEV uint32_t order_key(float l)
{
    const uint32_t u = __float_as_uint(l + 0.0f);
    const uint32_t k = u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
    return isnan(l) ? 1u : k;
}

EXL3_DEV float key_logit(uint32_t k)
{
    return k == 1u ? __uint_as_float(0x7FC00000u)
                   : __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

// A row's logits, lane l: experts l + 32 i (absent ones: `pad`).
template <int V>
EXL3_DEV void load_row(const void *p, size_t row, int E, int dtype, float pad, float (&v)[V])
{
    const int lane = threadIdx.x & 31;
    if (dtype == EXL3_F32) {
#pragma unroll
        for (int i = 0; i < V; i++)
            v[i] = lane + 32 * i < E ? static_cast<const float *>(p)[row + lane + 32 * i] : pad;
    } else if (dtype == EXL3_BF16) {
#pragma unroll
        for (int i = 0; i < V; i++)
            v[i] = lane + 32 * i < E
                       ? __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[row + lane + 32 * i])
                       : pad;
    } else {
#pragma unroll
        for (int i = 0; i < V; i++)
            v[i] = lane + 32 * i < E ? __half2float(static_cast<const __half *>(p)[row + lane + 32 * i]) : pad;
    }
}

// counts, T and loss from one expert's totals per thread: thread e of the CTA
// holds c and p of expert e0 + e; returns the CTA's part of sum c_e p_e in
// thread 0 (fixed order).
__device__ float block_dot(float v, float *scratch)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    v = warp_sum(v);
    if (lane == 0)
        scratch[warp] = v;
    __syncthreads();
    float t = threadIdx.x < nw ? scratch[threadIdx.x] : 0.0f;
    if (warp == 0)
        t = warp_sum(t);
    __syncthreads();
    return t;
}

EXL3_DEV float loss_of(const RouterArgs &a, float dot, int T)
{
    const float n = (float)T;
    return T ? (float)a.E / ((float)a.topk * n) * (dot / n) : 0.0f;
}

// V: experts per lane.  BAL: counts and probability sums as well; each CTA
// leaves its own in the workspace (rows are dealt to warps in a fixed way and
// everything is added in a fixed order), or finishes alone (one CTA).
template <int V, bool BAL>
__global__ void __launch_bounds__(kRouterWarps * 32) k_router_forward(RouterArgs a)
{
    extern __shared__ float sm[];                  // BAL: [E + 1] counts, then [warps][E] sums
    __shared__ float scratch[32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    const int E = a.E, k = a.topk;
    int32_t *cnt = reinterpret_cast<int32_t *>(sm);
    float psum[V];
    int nvalid = 0;
    if (BAL) {
        grid_dep_launch();
        for (int e = threadIdx.x; e <= E; e += blockDim.x)
            cnt[e] = 0;
#pragma unroll
        for (int i = 0; i < V; i++)
            psum[i] = 0.0f;
        __syncthreads();
    }
    for (int t = blockIdx.x * nw + warp; t < a.M; t += gridDim.x * nw) {
        float l[V];
        load_row<V>(a.logits, (size_t)t * E, E, a.logits_dtype, -INFINITY, l);
        uint32_t key[V], best = 0;
        int slot = 0;
#pragma unroll
        for (int i = V - 1; i >= 0; i--) {
            key[i] = lane + 32 * i < E ? order_key(l[i]) : 0u;
            if (key[i] >= best) {
                best = key[i];
                slot = i;
            }
        }
        const uint32_t top = __reduce_max_sync(0xffffffffu, best);
        const float m = key_logit(top);
        const float ref = m == -INFINITY ? 0.0f : m;           // NaN where every logit is NaN
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < V; i++) {
            l[i] = __expf(l[i] - ref);
            s += l[i];
        }
        s = warp_sum(s);
        const float inv = s == 0.0f ? 0.0f : 1.0f / s;
        if (a.stats && lane == 0)
            reinterpret_cast<float2 *>(a.stats)[t] = make_float2(ref, s);
        bool ok = false;
        if (BAL) {
            ok = !a.valid || a.valid[t] != 0;
            if (ok) {
                nvalid++;
#pragma unroll
                for (int i = 0; i < V; i++)
                    psum[i] += l[i] * inv;
            }
        }
        // round j: the warp's best key, the lowest expert that has it; lane j
        // keeps the pair, the owner drops it
        uint32_t mine = 0;
        int id = 0;
        for (int j = 0; j < k; j++) {
            const uint32_t b = j == 0 ? top : __reduce_max_sync(0xffffffffu, best);
            const int e = __reduce_min_sync(0xffffffffu, best == b ? slot * 32 + lane : 0x7FFFFFFF);
            if (lane == j) {
                mine = b;
                id = e;
            }
            if (lane == (e & 31)) {
                const int out = e >> 5;
                best = 0;
#pragma unroll
                for (int i = V - 1; i >= 0; i--) {
                    key[i] = i == out ? 0u : key[i];
                    if (key[i] >= best) {
                        best = key[i];
                        slot = i;
                    }
                }
            }
        }
        float w = lane < k ? __expf(key_logit(mine) - ref) * inv : 0.0f;
        if (a.renorm) {
            const float total = warp_sum(w);
            w = total == 0.0f ? 0.0f : w / total;
        }
        if (lane < k) {
            a.ids[(size_t)t * k + lane] = id;
            store_float(a.rw, (size_t)t * k + lane, a.rw_dtype, w);
            if (BAL && ok)
                atomicAdd(cnt + id, 1);
        }
    }
    if (!BAL)
        return;
    // the CTA's sums, warps in order
    float *rows = sm + E + 1;
#pragma unroll
    for (int i = 0; i < V; i++)
        if (lane + 32 * i < E)
            rows[warp * E + lane + 32 * i] = psum[i];
    if (lane == 0)
        atomicAdd(cnt + E, nvalid);
    __syncthreads();
    float dot = 0.0f;
    for (int e = threadIdx.x; e < E; e += blockDim.x) {
        float p = 0.0f;
        for (int w = 0; w < nw; w++)
            p += rows[w * E + e];
        if (gridDim.x == 1) {
            a.counts[e] = cnt[e];
            dot += (float)cnt[e] * p;
        } else {
            a.psum[(size_t)blockIdx.x * E + e] = p;
            a.pcount[(size_t)blockIdx.x * (E + 1) + e] = cnt[e];
        }
    }
    if (gridDim.x == 1) {
        dot = block_dot(dot, scratch);
        if (threadIdx.x == 0) {
            a.counts[E] = cnt[E];
            *a.loss = loss_of(a, dot, cnt[E]);
        }
    } else if (threadIdx.x == 0) {
        a.pcount[(size_t)blockIdx.x * (E + 1) + E] = cnt[E];
    }
}

// Joins the CTAs' counts and sums: a cluster of kJoin CTAs, each an eighth of
// the experts; 1024 / 32 = 32 threads per expert, whose parts are added in order.
constexpr int kJoin = 8, kJoinThreads = 1024;

EXL3_DEV void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__global__ void __cluster_dims__(kJoin, 1, 1) __launch_bounds__(kJoinThreads) k_router_join(RouterArgs a, int n)
{
    __shared__ float sp[kJoinThreads], scratch[32], parts[kJoin];
    __shared__ int sc[kJoinThreads], T;
    const int E = a.E, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    cluster_sync();                                // CTA 0's shared memory may be written from here on
    grid_dep_wait();
    if (warp == 0) {
        int t = 0;
        for (int g = lane; g < n; g += 32)
            t += a.pcount[(size_t)g * (E + 1) + E];
        t = __reduce_add_sync(0xffffffffu, t);
        if (lane == 0)
            T = t;
    }
    const int per = (E + kJoin - 1) / kJoin, e0 = blockIdx.x * per, e1 = min(E, e0 + per);
    float dot = 0.0f;
    for (int base = e0; base < e1; base += 32) {   // 32 experts at a time, 32 threads each
        const int e = base + lane;
        float p = 0.0f;
        int c = 0;
        if (e < e1)
#pragma unroll 10
            for (int g = warp; g < n; g += 32) {
                p += a.psum[(size_t)g * E + e];
                c += a.pcount[(size_t)g * (E + 1) + e];
            }
        sp[threadIdx.x] = p;
        sc[threadIdx.x] = c;
        __syncthreads();
        if (warp == 0 && e < e1) {
            for (int w = 1; w < 32; w++) {
                p += sp[w * 32 + lane];
                c += sc[w * 32 + lane];
            }
            a.counts[e] = c;
            dot += (float)c * p;
        }
        __syncthreads();
    }
    dot = block_dot(dot, scratch);
    // every CTA's part into CTA 0 of the cluster
    if (threadIdx.x == 0) {
        uint32_t dst;
        asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(dst) : "r"(smem_addr(parts + blockIdx.x)));
        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(dst), "f"(dot) : "memory");
    }
    cluster_sync();
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        float v = 0.0f;
        for (int i = 0; i < kJoin; i++)
            v += parts[i];
        a.counts[E] = T;
        *a.loss = loss_of(a, v, T);
    }
}

constexpr int kBackWarps = 8;

template <int V>
__global__ void __launch_bounds__(kBackWarps * 32) k_router_backward(RouterArgs a)
{
    extern __shared__ float sm[];                  // [warps][E]: the row's gradients at chosen experts
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int E = a.E, k = a.topk;
    float *at = sm + warp * E;
    for (int e = lane; e < E; e += 32)
        at[e] = 0.0f;
    __syncwarp();
    float g[V];                                    // balance gradient of p_e on valid rows
    {
        float cg = 0.0f;
        if (a.counts) {
            const float T = (float)a.counts[E];
            cg = T > 0.0f ? *a.d_loss * (float)E / ((float)k * T * T) : 0.0f;
        }
#pragma unroll
        for (int i = 0; i < V; i++)
            g[i] = a.counts && lane + 32 * i < E ? cg * (float)a.counts[lane + 32 * i] : 0.0f;
    }
    for (int t = blockIdx.x * kBackWarps + warp; t < a.M; t += gridDim.x * kBackWarps) {
        const size_t row = (size_t)t * E;
        const float2 st = reinterpret_cast<const float2 *>(a.stats)[t];
        const float inv = st.y == 0.0f ? 0.0f : 1.0f / st.y;
        const bool bal = a.counts && (!a.valid || a.valid[t] != 0);
        int id = -1;
        float d = 0.0f, pj = 0.0f;
        if (a.d_rw && lane < k) {
            id = a.ids[(size_t)t * k + lane];
            d = load_act(a.d_rw, (size_t)t * k + lane, a.rw_dtype);
            if ((unsigned)id >= (unsigned)E)
                id = -1;
        }
        float p[V];
        load_row<V>(a.logits, row, E, a.logits_dtype, -INFINITY, p);
        if (a.d_rw) {
            float add = d;
            if (a.renorm) {                        // w_j (d_j - sum w d), beside the softmax's own term
                pj = id >= 0 ? __expf(load_act(a.logits, row + id, a.logits_dtype) - st.x) * inv : 0.0f;
                const float total = warp_sum(pj);
                const float w = total == 0.0f ? 0.0f : pj / total;
                const float wd = warp_sum(id >= 0 ? w * d : 0.0f);
                add = w * (d - wd);
            }
            if (id >= 0)
                atomicAdd(at + id, add);           // distinct ids: one addend each
            __syncwarp();
        }
        float pg = 0.0f;
#pragma unroll
        for (int i = 0; i < V; i++) {
            p[i] = inv == 0.0f ? 0.0f : __expf(p[i] - st.x) * inv;
            float G = bal ? g[i] : 0.0f;
            if (a.d_rw && !a.renorm && lane + 32 * i < E)
                G += at[lane + 32 * i];
            pg = fmaf(p[i], G, pg);
        }
        pg = warp_sum(pg);
#pragma unroll
        for (int i = 0; i < V; i++) {
            const int e = lane + 32 * i;
            if (e < E) {
                const float own = a.d_rw ? at[e] : 0.0f;
                const float G = (bal ? g[i] : 0.0f) + (a.renorm ? 0.0f : own);
                store_float(a.d_logits, row + e, a.logits_dtype, fmaf(p[i], G - pg, a.renorm ? own : 0.0f));
            }
        }
        if (a.d_rw) {
            __syncwarp();
            if (id >= 0)
                at[id] = 0.0f;
            __syncwarp();
        }
    }
}

template <int V>
cudaError_t forward(const RouterArgs &a, cudaStream_t s)
{
    const size_t bal_smem = ((size_t)a.E + 1 + (size_t)kRouterWarps * a.E) * 4;
    if (!a.counts) {
        // few rows: a warp each on as many SMs as there are
        const int warps = a.M >= a.num_sms * kRouterWarps ? kRouterWarps : a.M >= 4 * a.num_sms ? 4 : 1;
        const int need = (a.M + warps - 1) / warps, most = a.num_sms * (64 / kRouterWarps) * (kRouterWarps / warps);
        k_router_forward<V, false><<<need < most ? need : most, warps * 32, 0, s>>>(a);
        return cudaGetLastError();
    }
    const int n = router_balance_ctas(a.M);
    if (n > 0)
        k_router_forward<V, true><<<n, kRouterWarps * 32, bal_smem, s>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (n == 1 || e != cudaSuccess)
        return e;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = n > 0;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(kJoin);
    cfg.blockDim = dim3(kJoinThreads);
    cfg.stream = s;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_router_join, a, n);
}

template <int V>
cudaError_t backward(const RouterArgs &a, cudaStream_t s)
{
    const int need = (a.M + kBackWarps - 1) / kBackWarps, most = a.num_sms * 8;
    k_router_backward<V><<<need < most ? need : most, kBackWarps * 32, (size_t)kBackWarps * a.E * 4, s>>>(a);
    return cudaGetLastError();
}

// The smallest instantiation that holds E experts.
template <typename F>
cudaError_t by_width(int E, F f)
{
    const int v = (E + 31) / 32;
    if (v <= 1) return f(std::integral_constant<int, 1>());
    if (v <= 2) return f(std::integral_constant<int, 2>());
    if (v <= 4) return f(std::integral_constant<int, 4>());
    if (v <= 6) return f(std::integral_constant<int, 6>());
    if (v <= 8) return f(std::integral_constant<int, 8>());
    if (v <= 10) return f(std::integral_constant<int, 10>());
    if (v <= 12) return f(std::integral_constant<int, 12>());
    if (v <= 16) return f(std::integral_constant<int, 16>());
    return f(std::integral_constant<int, 32>());
}

}  // namespace

// The balance pass of more than 512 experts needs more than 48 KB of sums.
cudaError_t router_set_attributes()
{
    return cudaFuncSetAttribute(k_router_forward<32, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (EXL3_MAX_EXPERTS * (kRouterWarps + 1) + 1) * 4);
}

size_t router_workspace_bytes(int M, int E)
{
    const size_t n = router_balance_ctas(M);
    return (n * (2 * (size_t)E + 1) * 4 + 256) / 256 * 256;
}

cudaError_t launch_router_forward(const RouterArgs &a, cudaStream_t s)
{
    if (a.M == 0 && !a.counts)
        return cudaSuccess;
    return by_width(a.E, [&](auto v) { return forward<v.value>(a, s); });
}

cudaError_t launch_router_backward(const RouterArgs &a, cudaStream_t s)
{
    return by_width(a.E, [&](auto v) { return backward<v.value>(a, s); });
}

}  // namespace exl3
