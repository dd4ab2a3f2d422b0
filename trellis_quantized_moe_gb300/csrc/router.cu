// Router: softmax top-k with route weights, balance loss and per-expert
// counts, and the gradient of the logits (include/exl3.h, "router").
//
// A warp owns a row: lane l holds the logits of experts 2l, 2l + 1, 2l + 64, ...
// in registers (pairs: half the loads, stores and conversions), so the row is
// read once.  Forward: m = max l, s = sum exp(l - m),
// p_e = exp(l_e - m) / s (kept as the pair: m + log s in fp32 would lose s for
// large |m|); then topk rounds of a warp-wide maximum over order-preserving
// integer keys, ties to the lower expert (Chooser).  Backward, with G_e = dL/dp_e
// (balance term on valid rows, plus the route weights' gradient where they are
// plain probabilities):
//   dl_e = p_e (G_e - sum_j p_j G_j),
// and renormalised weights w, which depend on the chosen logits only, add
// w_i (d_i - sum_j w_j d_j) at the chosen experts.
//
// exp is expf and divisions are true ones: with 2^x of a rounded product and
// approximate reciprocals and logarithms fp32 results were up to twice as far from 64
// bits as the formula in fp32 (65536 x 192, forward and backward: 51 us so, 56 now).
//
// What bounds it: not HBM but the instructions per row, most of them the
// choice's.  Measured at 65536 x 192 bf16, top 8, graph replay: forward with the
// balance and its join 32 us (399 instructions a row, 74% of the issue slots, the
// ALU pipe 54% busy, DRAM 10%), backward 19 us (278 instructions a row).
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

// The expert of a lane's value i.
EXL3_DEV int expert_of(int i) { return 64 * (i / 2) + 2 * (threadIdx.x & 31) + (i & 1); }

// A row of logits as it lies in memory: V / 2 pairs a lane.
template <int DT, int V>
struct RawRow {
    using T = std::conditional_t<DT == EXL3_F32, float, uint16_t>;
    using Pair = std::conditional_t<DT == EXL3_F32, float2, uint32_t>;
    Pair v[V / 2];
    EXL3_DEV void load(const void *p, size_t row, int E)
    {
        const T *q = static_cast<const T *>(p) + row;
        if ((E & 1) == 0) {                        // every pair is aligned and whole
#pragma unroll
            for (int i = 0; i < V / 2; i++)
                v[i] = expert_of(2 * i) < E ? *reinterpret_cast<const Pair *>(q + expert_of(2 * i)) : Pair{};
        } else {
#pragma unroll
            for (int i = 0; i < V / 2; i++) {
                const int e = expert_of(2 * i);
                const T a = e < E ? q[e] : T(0), b = e + 1 < E ? q[e + 1] : T(0);
                if constexpr (DT == EXL3_F32)
                    v[i] = make_float2(a, b);
                else
                    v[i] = (uint32_t)a | (uint32_t)b << 16;
            }
        }
    }
    EXL3_DEV float get(int i) const
    {
        if constexpr (DT == EXL3_F32) {
            return i & 1 ? v[i / 2].y : v[i / 2].x;
        } else if constexpr (DT == EXL3_BF16) {
            return __uint_as_float(i & 1 ? v[i / 2] & 0xFFFF0000u : v[i / 2] << 16);
        } else {
            const __half2 h = *reinterpret_cast<const __half2 *>(&v[i / 2]);
            return i & 1 ? __high2float(h) : __low2float(h);
        }
    }
};

// The gradient of a row, rounded to the logits' type.
template <int DT, int V>
EXL3_DEV void store_row(void *p, size_t row, int E, const float (&d)[V])
{
    if ((E & 1) == 0) {
#pragma unroll
        for (int i = 0; i < V; i += 2)
            if (expert_of(i) < E) {
                if constexpr (DT == EXL3_F32) {
                    *reinterpret_cast<float2 *>(static_cast<float *>(p) + row + expert_of(i)) = make_float2(d[i], d[i + 1]);
                } else if constexpr (DT == EXL3_BF16) {
                    *reinterpret_cast<__nv_bfloat162 *>(static_cast<__nv_bfloat16 *>(p) + row + expert_of(i)) =
                        __floats2bfloat162_rn(d[i], d[i + 1]);
                } else {
                    *reinterpret_cast<__half2 *>(static_cast<__half *>(p) + row + expert_of(i)) =
                        __floats2half2_rn(d[i], d[i + 1]);
                }
            }
    } else {
#pragma unroll
        for (int i = 0; i < V; i++)
            if (expert_of(i) < E)
                store_float(p, row + expert_of(i), DT, d[i]);
    }
}

// Unsigned integers in the order of the logits, -0 as +0 and NaN as -inf.
// 16-bit logits (as fp32) order by their upper 19 bits: the lower 13 bits take
// the complement of the expert, so that one integer maximum also settles ties.
EXL3_DEV uint32_t order_key(float l)
{
    const uint32_t u = __float_as_uint(fmaxf(l, -INFINITY) + 0.0f);
    return u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
}
EXL3_DEV float key_logit(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k); }

constexpr uint32_t kExpertBits = 0x1FFF;           // 13 bits; 1024 experts need 10

// Batcher's merge exchange: sorts v[0..V) descending, with `swap` exchanging a
// pair that is out of order.
template <int V, typename Swap>
EXL3_DEV void sort_network(Swap swap)
{
    constexpr int kP2 = V <= 1 ? 1 : V <= 2 ? 2 : V <= 4 ? 4 : V <= 8 ? 8 : V <= 16 ? 16 : 32;
#pragma unroll
    for (int p = 1; p < kP2; p *= 2)
#pragma unroll
        for (int k = p; k >= 1; k /= 2)
#pragma unroll
            for (int j = k % p; j + k < kP2; j += 2 * k)
#pragma unroll
                for (int i = 0; i < k; i++)
                    if (i + j + k < V && (i + j) / (2 * p) == (i + j + k) / (2 * p))
                        swap(i + j, i + j + k);
}

// The row's experts in order of choice, one call per round: every lane keeps
// its own experts sorted (a network of V log^2 V exchanges without branches) and
// shows the first; the owner of the warp's best moves up.  The network lies in
// registers up to V = 12; at 16 and 32 (more than 384 experts) the compiler keeps
// its loops, and the keys are in local memory (64 to 624 bytes a thread, with
// what spills).
template <bool PACKED, int V>
struct Chooser;

template <int V>
struct Chooser<true, V> {                          // 16-bit logits: expert in the key
    uint32_t k[V];
    template <bool FULL>
    EXL3_DEV void init(const float (&l)[V], int E)
    {
#pragma unroll
        for (int i = 0; i < V; i++) {
            const int e = expert_of(i);
            k[i] = FULL || e < E ? (order_key(l[i]) & ~kExpertBits) | (kExpertBits - e) : 0u;
        }
    }
    EXL3_DEV void sort()
    {
        sort_network<V>([&](int a, int b) {
            const uint32_t hi = max(k[a], k[b]), lo = min(k[a], k[b]);
            k[a] = hi;
            k[b] = lo;
        });
    }
    // this round's choice: the owner leaves it in out[j]
    EXL3_DEV uint32_t next(int j, uint2 *out)
    {
        const uint32_t b = __reduce_max_sync(0xffffffffu, k[0]);
        const bool own = k[0] == b;
        if (own)
            out[j].x = b;
#pragma unroll
        for (int i = 0; i + 1 < V; i++)
            k[i] = own ? k[i + 1] : k[i];
        k[V - 1] = own ? 0u : k[V - 1];
        return b;
    }
    // a negative logit's key has ones where the fraction ends
    static EXL3_DEV uint32_t key(uint32_t b) { return b & 0x80000000u ? b & ~kExpertBits : b | kExpertBits; }
    // lane j < topk: round j's choice
    EXL3_DEV uint2 collect(int topk, const uint2 *out) const
    {
        __syncwarp();
        const int lane = threadIdx.x & 31;
        const uint32_t b = lane < topk ? out[lane].x : 0u;
        __syncwarp();                              // read before the next row's are written
        return make_uint2(b, kExpertBits - (b & kExpertBits));
    }
};

template <int V>
struct Chooser<false, V> {                         // fp32 logits: key and expert side by side
    uint32_t k[V], mine = 0;
    int e[V], id = 0;
    template <bool FULL>
    EXL3_DEV void init(const float (&l)[V], int E)
    {
#pragma unroll
        for (int i = 0; i < V; i++) {
            e[i] = expert_of(i);
            k[i] = FULL || e[i] < E ? order_key(l[i]) : 0u;   // every logit's key is above 0
        }
    }
    EXL3_DEV void sort()
    {
        sort_network<V>([&](int a, int b) {
            const bool x = k[a] < k[b] || (k[a] == k[b] && e[a] > e[b]);
            const uint32_t ka = k[a];
            const int ea = e[a];
            k[a] = x ? k[b] : ka;
            e[a] = x ? e[b] : ea;
            k[b] = x ? ka : k[b];
            e[b] = x ? ea : e[b];
        });
    }
    // this round's choice, kept by lane j (through shared memory, as above, the
    // longer rounds of this type were slower)
    EXL3_DEV uint32_t next(int j, uint2 *)
    {
        const uint32_t b = __reduce_max_sync(0xffffffffu, k[0]);
        const int x = __reduce_min_sync(0xffffffffu, k[0] == b ? e[0] : 0x7FFFFFFF);
        const bool own = e[0] == x && k[0] == b;
        mine = (threadIdx.x & 31) == j ? b : mine;
        id = (threadIdx.x & 31) == j ? x : id;
#pragma unroll
        for (int i = 0; i + 1 < V; i++) {
            k[i] = own ? k[i + 1] : k[i];
            e[i] = own ? e[i + 1] : e[i];
        }
        k[V - 1] = own ? 0u : k[V - 1];
        return b;
    }
    static EXL3_DEV uint32_t key(uint32_t b) { return b; }
    EXL3_DEV uint2 collect(int, const uint2 *) const { return make_uint2(mine, id); }
};

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
template <int DT, int V, bool BAL>
__global__ void __launch_bounds__(kRouterWarps * 32, V <= 12 ? 2 : 1) k_router_forward(RouterArgs a)
{
    extern __shared__ float sm[];                  // BAL: [E + 1] counts, then [warps][E] sums
    __shared__ float scratch[32];
    __shared__ uint2 chosen[kRouterWarps][EXL3_ROUTER_MAX_TOPK];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    const int E = a.E, k = a.topk;
    int32_t *cnt = reinterpret_cast<int32_t *>(sm);
    float psum[V];
    int nvalid = 0;
    grid_dep_wait();                               // logits may come from the kernel before
    grid_dep_launch();
    if (BAL) {
        for (int e = threadIdx.x; e <= E; e += blockDim.x)
            cnt[e] = 0;
#pragma unroll
        for (int i = 0; i < V; i++)
            psum[i] = 0.0f;
        __syncthreads();
    }
    const int step = gridDim.x * nw;
    RawRow<DT, V> raw;
    int t = blockIdx.x * nw + warp;
    if (t < a.M)
        raw.load(a.logits, (size_t)t * E, E);
    for (; t < a.M; t += step) {
        float l[V];
        using C = Chooser<DT != EXL3_F32, V>;
        C choose;
        if (E == 32 * V) {                         // no absent experts
#pragma unroll
            for (int i = 0; i < V; i++)
                l[i] = raw.get(i);
            choose.template init<true>(l, E);
        } else {
#pragma unroll
            for (int i = 0; i < V; i++)
                l[i] = expert_of(i) < E ? raw.get(i) : -INFINITY;
            choose.template init<false>(l, E);
        }
        choose.sort();
        const bool ok = BAL && (!a.valid || a.valid[t] != 0);
        if (t + step < a.M)                        // the next row, one round of work ahead
            raw.load(a.logits, (size_t)(t + step) * E, E);
        uint2 *out = chosen[warp];
        // the first choice has the largest logit
        const float m = key_logit(C::key(choose.next(0, out)));
        const float ref = m == -INFINITY ? 0.0f : m;
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < V; i++) {
            l[i] = expf(l[i] - ref);
            s += l[i];
        }
        s = warp_sum(s);
        const float inv = s == 0.0f ? 0.0f : 1.0f / s;
        if (a.stats && lane == 0)
            reinterpret_cast<float2 *>(a.stats)[t] = make_float2(ref, s);
        if (ok) {
            nvalid++;
#pragma unroll
            for (int i = 0; i < V; i++)
                psum[i] = fmaf(l[i], inv, psum[i]);
        }
#pragma unroll 4
        for (int j = 1; j < k; j++)
            choose.next(j, out);
        const uint2 mine = choose.collect(k, out);
        const int id = (int)mine.y;
        // (a division of its own: one rounding less than a product with inv)
        float w = lane < k && s != 0.0f ? expf(key_logit(C::key(mine.x)) - ref) / s : 0.0f;
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
        if (expert_of(i) < E)
            rows[warp * E + expert_of(i)] = psum[i];
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

EXL3_DEV void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
EXL3_DEV void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
EXL3_DEV void cluster_sync()
{
    cluster_arrive();
    cluster_wait();
}

__global__ void __cluster_dims__(kJoin, 1, 1) __launch_bounds__(kJoinThreads) k_router_join(RouterArgs a, int n)
{
    __shared__ float sp[kJoinThreads], scratch[32], parts[kJoin];
    __shared__ int sc[kJoinThreads];
    const int E = a.E, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    cluster_arrive();                              // CTA 0's shared memory may be written after the wait
    grid_dep_wait();
    // valid rows: a thread per CTA of the balance pass
    const int valid = threadIdx.x < n ? a.pcount[(size_t)threadIdx.x * (E + 1) + E] : 0;
    const int per = (E + kJoin - 1) / kJoin, e0 = blockIdx.x * per, e1 = min(E, e0 + per);
    float dot = 0.0f;
    for (int base = e0; base < e1; base += 32) {   // 32 experts at a time, 32 threads each
        const int e = base + lane;
        float p = 0.0f;
        int c = 0;
        // every load in flight at once: a loop with a remainder took 10 us here
        constexpr int kMost = (kRouterCtas + 31) / 32;
        float lp[kMost];
        int lc[kMost];
#pragma unroll
        for (int u = 0; u < kMost; u++) {
            const int g = warp + 32 * u;
            const bool in = e < e1 && g < n;
            lp[u] = in ? a.psum[(size_t)g * E + e] : 0.0f;
            lc[u] = in ? a.pcount[(size_t)g * (E + 1) + e] : 0;
        }
#pragma unroll
        for (int u = 0; u < kMost; u++) {
            p += lp[u];
            c += lc[u];
        }
        sp[threadIdx.x] = p;
        sc[threadIdx.x] = c;
        __syncthreads();
        if (warp == 0 && e < e1) {
#pragma unroll
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
    if (blockIdx.x == 0) {
        const int t = __reduce_add_sync(0xffffffffu, valid);
        if (lane == 0)
            sc[warp] = t;
        __syncthreads();
    }
    cluster_wait();
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
        int T = 0;
        for (int i = 0; i < 32; i++)
            T += sc[i];
        a.counts[E] = T;
        *a.loss = loss_of(a, v, T);
    }
}

constexpr int kBackWarps = 8;

template <int DT, int V>
__global__ void __launch_bounds__(kBackWarps * 32, V <= 6 ? 4 : 1) k_router_backward(RouterArgs a)
{
    extern __shared__ float sm[];                  // [warps][E, even]: the row's gradients at chosen experts
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int E = a.E, k = a.topk;
    const int pitch = (E + 1) / 2 * 2;             // read in pairs
    float *at = sm + warp * pitch;
    for (int e = lane; e < pitch; e += 32)
        at[e] = 0.0f;
    __syncwarp();
    grid_dep_wait();                               // the inputs may come from the kernel before
    grid_dep_launch();
    float g[V];                                    // balance gradient of p_e on valid rows
    {
        float cg = 0.0f;
        if (a.counts) {
            const float T = (float)a.counts[E];
            cg = T > 0.0f ? *a.d_loss * (float)E / ((float)k * T * T) : 0.0f;
        }
#pragma unroll
        for (int i = 0; i < V; i++)
            g[i] = a.counts && expert_of(i) < E ? cg * (float)a.counts[expert_of(i)] : 0.0f;
    }
    // one row's inputs, read a row ahead of their use
    struct Row {
        RawRow<DT, V> raw;
        float2 st;
        float d, chosen;
        int id;
        bool bal;
    } next;
    const int step = gridDim.x * kBackWarps;
    int t = blockIdx.x * kBackWarps + warp;
    size_t at_next = (size_t)t * E, choice = (size_t)t * k + lane;       // of the row fetched next
    const size_t row_step = (size_t)step * E, choice_step = (size_t)step * k;
    auto fetch = [&](int t, Row &r) {
        r.raw.load(a.logits, at_next, E);
        r.st = reinterpret_cast<const float2 *>(a.stats)[t];
        r.bal = a.counts && (!a.valid || a.valid[t] != 0);
        r.id = -1;
        r.d = r.chosen = 0.0f;
        if (a.d_rw && lane < k) {
            r.id = a.ids[choice];
            r.d = load_act(a.d_rw, choice, a.rw_dtype);
            if ((unsigned)r.id >= (unsigned)E)
                r.id = -1;
            else if (a.renorm)
                r.chosen = load_act(a.logits, at_next + r.id, DT);
        }
        at_next += row_step;
        choice += choice_step;
    };
    const bool full = E == 32 * V;                 // no absent experts
    size_t here = at_next;
    if (t < a.M)
        fetch(t, next);
    for (; t < a.M; t += step, here += row_step) {
        const Row r = next;
        if (t + step < a.M)
            fetch(t + step, next);
        const float inv = r.st.y == 0.0f ? 0.0f : 1.0f / r.st.y;       // 0: a row of -inf only, p = 0
        if (a.d_rw) {
            float add = r.d;
            if (a.renorm) {                        // w_j (d_j - sum w d), beside the softmax's own term
                const float pj = r.id >= 0 ? expf(r.chosen - r.st.x) * inv : 0.0f;
                const float total = warp_sum(pj);
                const float w = total == 0.0f ? 0.0f : pj / total;
                const float wd = warp_sum(r.id >= 0 ? w * r.d : 0.0f);
                add = w * (r.d - wd);
            }
            if (r.id >= 0)
                at[r.id] = add;
            __syncwarp();
        }
        float p[V], own[V];                        // absent experts: nothing stored, not in any sum
#pragma unroll
        for (int i = 0; i < V; i += 2) {
            const float2 at2 = a.d_rw && (full || expert_of(i) < E)
                                   ? *reinterpret_cast<const float2 *>(at + expert_of(i))
                                   : make_float2(0.0f, 0.0f);
            own[i] = at2.x;
            own[i + 1] = at2.y;
            p[i] = expf(r.raw.get(i) - r.st.x) * inv;
            p[i + 1] = expf(r.raw.get(i + 1) - r.st.x) * inv;
        }
        // sum of p_e x_e over the row's experts
        auto expectation = [&](const float (&x)[V]) {
            float v = 0.0f;
            if (full) {
#pragma unroll
                for (int i = 0; i < V; i++)
                    v = fmaf(p[i], x[i], v);
            } else {
#pragma unroll
                for (int i = 0; i < V; i++)
                    v = expert_of(i) < E ? fmaf(p[i], x[i], v) : v;
            }
            return warp_sum(v);
        };
        if (!a.renorm) {
            if (r.bal)
#pragma unroll
                for (int i = 0; i < V; i++)
                    own[i] += g[i];
            const float pg = expectation(own);
#pragma unroll
            for (int i = 0; i < V; i++)
                own[i] = p[i] * (own[i] - pg);
        } else if (r.bal) {
            const float pg = expectation(g);
#pragma unroll
            for (int i = 0; i < V; i++)
                own[i] = fmaf(p[i], g[i] - pg, own[i]);
        } else {                                   // a NaN row stays one
#pragma unroll
            for (int i = 0; i < V; i++)
                own[i] = fmaf(p[i], 0.0f, own[i]);
        }
        store_row<DT, V>(a.d_logits, here, E, own);
        if (a.d_rw) {
            __syncwarp();
            if (r.id >= 0)
                at[r.id] = 0.0f;
            __syncwarp();
        }
    }
}

// Launches that may start while the kernel before them in the stream still
// runs; each kernel waits for it before it reads anything.
template <typename... P, typename... A>
cudaError_t launch(void (*kernel)(P...), int grid, int threads, size_t smem, cudaStream_t s, const A &...args)
{
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <int DT, int V>
cudaError_t forward(const RouterArgs &a, cudaStream_t s)
{
    const size_t bal_smem = ((size_t)a.E + 1 + (size_t)kRouterWarps * a.E) * 4;
    if (!a.counts) {
        // four warps (192 experts, with 16 / 4 / 1: 100 rows 1.7 / 1.6 / 1.7 us,
        // 5000 rows 3.7 / 3.3 / 5.5, 20000 rows 8.8 / 8.4 / 10.3).  Registers let 8 to
        // 10 of the 16 CTAs run at a time, so that above some 6000 rows the grid's
        // last wave is partly empty.
        constexpr int kW = 4;
        const int need = (a.M + kW - 1) / kW, most = a.num_sms * (64 / kW);
        return launch(k_router_forward<DT, V, false>, need < most ? need : most, kW * 32, 0, s, a);
    }
    const int n = router_balance_ctas(a.M);
    const cudaError_t e =
        n > 0 ? launch(k_router_forward<DT, V, true>, n, kRouterWarps * 32, bal_smem, s, a) : cudaSuccess;
    return n == 1 || e != cudaSuccess ? e : launch(k_router_join, kJoin, kJoinThreads, 0, s, a, n);
}

// Four CTAs an SM run at a time up to 192 experts; wider rows take 84 registers
// and more, so that three and fewer do and a large batch ends in a part of a wave.
template <int DT, int V>
cudaError_t backward(const RouterArgs &a, cudaStream_t s)
{
    const int need = (a.M + kBackWarps - 1) / kBackWarps, most = a.num_sms * 4;     // one wave up to 192 experts
    return launch(k_router_backward<DT, V>, need < most ? need : most, kBackWarps * 32,
                  (size_t)kBackWarps * ((a.E + 1) / 2 * 2) * 4, s, a);
}

// f(dtype, experts per lane) for the smallest instantiation that holds E experts.
template <int DT, typename F>
cudaError_t by_width(int E, F f)
{
    constexpr std::integral_constant<int, DT> dt;
    const int v = (E + 63) / 64 * 2;
    if (v <= 2) return f(dt, std::integral_constant<int, 2>());
    if (v <= 4) return f(dt, std::integral_constant<int, 4>());
    if (v <= 6) return f(dt, std::integral_constant<int, 6>());
    if (v <= 8) return f(dt, std::integral_constant<int, 8>());
    if (v <= 10) return f(dt, std::integral_constant<int, 10>());
    if (v <= 12) return f(dt, std::integral_constant<int, 12>());
    if (v <= 16) return f(dt, std::integral_constant<int, 16>());
    return f(dt, std::integral_constant<int, 32>());
}

template <typename F>
cudaError_t by_row(int dtype, int E, F f)
{
    return dtype == EXL3_F32    ? by_width<EXL3_F32>(E, f)
           : dtype == EXL3_BF16 ? by_width<EXL3_BF16>(E, f)
                                : by_width<EXL3_F16>(E, f);
}

}  // namespace

// The balance pass of more than 512 experts needs more than 48 KB of sums.
cudaError_t router_set_attributes()
{
    const int most = (EXL3_MAX_EXPERTS * (kRouterWarps + 1) + 1) * 4;
    const auto attr = cudaFuncAttributeMaxDynamicSharedMemorySize;
    cudaError_t e = cudaFuncSetAttribute(k_router_forward<EXL3_F32, 32, true>, attr, most);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(k_router_forward<EXL3_BF16, 32, true>, attr, most);
    return e == cudaSuccess ? cudaFuncSetAttribute(k_router_forward<EXL3_F16, 32, true>, attr, most) : e;
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
    return by_row(a.logits_dtype, a.E, [&](auto dt, auto v) { return forward<dt.value, v.value>(a, s); });
}

cudaError_t launch_router_backward(const RouterArgs &a, cudaStream_t s)
{
    return by_row(a.logits_dtype, a.E, [&](auto dt, auto v) { return backward<dt.value, v.value>(a, s); });
}

}  // namespace exl3
