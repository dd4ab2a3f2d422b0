// Adapters for batches of few rows: both products in one launch.
//   h[s] = h_scale * W1 x[perm[s]],  y[perm[s]] = base[perm[s]] + y_scale * h[s] W2
// (W1, W2 = A, B forward; B, A backward).
//
// A decode batch reads each adapter once for a row or a few, so it is bound by
// latencies: two launches with partial sums through memory between them took
// 10 us of GPU time for one row.  Here a cluster of CTAs takes a tile of up to
// eight rows of one adapter.  Its warps share the contraction of the first
// product in 32-wide blocks; the partial h are added warp by warp in
// shared memory, then CTA by CTA over distributed shared memory (a fixed
// order) and split into two parts of the operand type, so every CTA has h and
// goes on with its own columns of the second product, whose weights and base
// rows are already on their way.
//
// Operands go from global memory to mma.sync fragments directly, 16 bytes a
// lane.  First product (M = ranks, N = rows): a lane's eight consecutive k
// feed two MMAs as (0,1 | 2,3) and (4,5 | 6,7); the order of a contraction is
// free as long as both operands use it.  Second product (M = columns): lane
// (g, t) loads rows j = 2t, 2t+1, 2t+8, 2t+9 of W2 at columns 8g .. 8g+7 and
// interleaves pairs; MMA i takes columns 8g+i and 8g+i+4 as its rows g and
// g+8, so that a lane ends up with eight consecutive columns of two rows of y.
//
// The second product takes h's two parts (its rounded value and the rest) as
// B operands beside the same weights: 0.5 us of the 64 rows below.  f16 sums the
// rests' products in accumulators of their own (split2): another 0.3 us.
//
// Measured (bf16, 5120 -> 1536): one row, rank 16: 4.7 us; 64 rows over 40
// adapters of ranks 8 to 64: 10.7 us for 20 MB (1.9 TB/s).  What it spends: 2 us
// on plan and tables, 4 on the first product's weights (three rounds of loads
// of what the registers hold), 1 each on the two reductions and the second
// product, the rest on start and end.  Sixteen-row tiles, three CTAs an SM and deeper or shallower rounds
// were no faster.
#include "lora_common.cuh"

namespace exl3 {
namespace lora {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kRows = kLoraSmallTile;
static_assert(kRows == 8, "a tile's rows are one MMA's N");

template <bool BF>
EXL3_DEV void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1)
{
    if constexpr (BF)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
            "{%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        mma_16816(d, a0, a1, a2, a3, b0, b1);
}

EXL3_DEV void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
EXL3_DEV void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
EXL3_DEV void cluster_sync()
{
    cluster_arrive();
    cluster_wait();
}

EXL3_DEV float4 ld_cluster(uint32_t addr, int rank)
{
    uint32_t remote;
    float4 v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(addr), "r"(rank));
    asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(remote)
                 : "memory");
    return v;
}

EXL3_DEV uint4 ld16_or_zero(const uint8_t *p, bool in)
{
    return in ? __ldg(reinterpret_cast<const uint4 *>(p)) : make_uint4(0, 0, 0, 0);
}

// MT: 16-rank blocks of the largest rank.  Dynamic shared memory: the warps'
// partial h [kWarps][16 MT][8], the CTA's [16 MT][8], and h's two parts [2][8][16 MT + 8].
template <int MT>
constexpr int rows_smem()
{
    return (kWarps + 1) * 16 * MT * kRows * 4 + 2 * kRows * (16 * MT + 8) * 2;
}

template <bool BF, int MT>
__global__ void __launch_bounds__(kThreads, 2) k_lora_rows(LoraRowsArgs a)
{
    extern __shared__ __align__(16) uint8_t smem[];
    constexpr int dtype = BF ? EXL3_BF16 : EXL3_F16;
    constexpr int kPitch = 16 * MT + 8;
    float *red = reinterpret_cast<float *>(smem);
    float *hpart = red + kWarps * 16 * MT * kRows;
    uint16_t *h16 = reinterpret_cast<uint16_t *>(hpart + 16 * MT * kRows);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, q = lane & 3;
    const int ctas = a.ctas, all_warps = ctas * kWarps;
    const int cta = blockIdx.x % ctas, own = blockIdx.x / ctas;
    grid_dep_wait();                // plan, tables and rows may come from the kernel before
    grid_dep_launch();              // only now: the kernels after read the plan before their own wait
    auto zero_fill = [&]() {
        const size_t all = a.y ? (size_t)a.M * a.out_width / 8 : 0;
        for (size_t i = (size_t)blockIdx.x * kThreads + tid; i < all; i += (size_t)gridDim.x * kThreads)
            static_cast<uint4 *>(a.y)[i] = make_uint4(0, 0, 0, 0);
    };
    const LoraPlanLayout L = lora_plan_layout(a.M, a.N);
    const int4 *tiles = reinterpret_cast<const int4 *>(a.plan + L.small / 4);
    const int32_t *perm = a.plan + L.perm / 4;
    // the tile is read along with the header that says whether it is one (the
    // host has checked the plan's size, the launch has no more clusters than
    // the list has room)
    int4 t = tiles[own];
    const bool plan_bad = !plan_ok(a.plan, a.M, a.N);
    const int ntiles = a.plan[kLpSmallTiles], active = a.plan[kLpSmallActive];
    if (plan_bad) {
        const bool made = a.plan[kLpMagic] == kLoraMagic && a.plan[kLpM] == a.M && a.plan[kLpN] == a.N;
        if (blockIdx.x == 0 && tid == 0)
            a.hdr[kHdrError] = made ? a.plan[kLpError] : EXL3_DERR_PLAN;
        zero_fill();
        return;
    }
    if (own >= ntiles)
        t = make_int4(-1, 0, 0, 0);
    auto entry_bad = [&](int e) {
        const int r = a.rank[e];
        bool bad = r < 0 || r > a.max_rank;
        if (r > 0) {
            bad |= !a.W1[e] || (a.W1[e] & 15) || !a.W2[e] || (a.W2[e] & 15);
            if (a.GA)
                bad |= !a.GA[e] || (a.GA[e] & 15) || !a.GB[e] || (a.GB[e] & 15);
        }
        return bad;
    };
    // every CTA checks every table entry in use: none has to wait for another
    bool bad = false;
    if (a.GA)
        for (int e = tid; e < a.N; e += kThreads)
            bad |= entry_bad(e);
    else
        for (int i = tid; i < active; i += kThreads)
            bad |= entry_bad(tiles[i].x);

    int rank = 0;
    const uint8_t *w1 = nullptr, *w2 = nullptr;
    if (t.x >= 0 && !entry_bad(t.x)) {
        rank = a.rank[t.x];
        w1 = reinterpret_cast<const uint8_t *>(a.W1[t.x]);
        w2 = reinterpret_cast<const uint8_t *>(a.W2[t.x]);
    }
    const int nmt = (rank + 15) / 16;
    const float alpha = rank > 0 ? a.scale[t.x] : 1.0f;
    const size_t in_pitch = (size_t)a.in_width * 2, out_pitch = (size_t)a.out_width * 2;

    if (nmt > 0) {
        float acc[MT][4];
#pragma unroll
        for (int m = 0; m < MT; m++)
#pragma unroll
            for (int i = 0; i < 4; i++)
                acc[m][i] = 0.0f;
        const bool in0 = g < t.z;
        const uint8_t *x = static_cast<const uint8_t *>(a.x) + (in0 ? perm[t.y + g] : 0) * in_pitch + q * 16;
        const uint8_t *w = w1 + g * in_pitch + q * 16;
        constexpr int kU = MT == 1 ? 6 : MT == 2 ? 4 : MT == 4 ? 2 : 1;     // blocks in flight
        const int blocks = a.in_width / 32;
        for (int b0 = cta * kWarps + warp; b0 < blocks; b0 += kU * all_warps) {
            uint4 fx[kU], fw0[kU][MT], fw1[kU][MT];
#pragma unroll
            for (int u = 0; u < kU; u++) {
                const size_t o = (size_t)(b0 + u * all_warps) * 64;
                const bool in = b0 + u * all_warps < blocks;
                fx[u] = ld16_or_zero(x + o, in && in0);
#pragma unroll
                for (int m = 0; m < MT; m++) {
                    fw0[u][m] = ld16_or_zero(w + o + m * 16 * in_pitch, in && 16 * m + g < rank);
                    fw1[u][m] = ld16_or_zero(w + o + (m * 16 + 8) * in_pitch, in && 16 * m + 8 + g < rank);
                }
            }
#pragma unroll
            for (int u = 0; u < kU; u++)
#pragma unroll
                for (int m = 0; m < MT; m++)
                    if (m < nmt) {
                        const uint4 p = fw0[u][m], r = fw1[u][m];
                        mma16816<BF>(acc[m], p.x, r.x, p.y, r.y, fx[u].x, fx[u].y);
                        mma16816<BF>(acc[m], p.z, r.z, p.w, r.w, fx[u].z, fx[u].w);
                    }
        }
        float *mine = red + warp * (16 * MT * kRows);
#pragma unroll
        for (int m = 0; m < MT; m++)
            if (m < nmt) {
                *reinterpret_cast<float2 *>(mine + (16 * m + g) * kRows + 2 * q) = make_float2(acc[m][0], acc[m][1]);
                *reinterpret_cast<float2 *>(mine + (16 * m + g + 8) * kRows + 2 * q) =
                    make_float2(acc[m][2], acc[m][3]);
            }
    }
    // the second product's first weights and base rows, on their way during the reduction
    constexpr int kPre = MT < 4 ? MT : 4;
    constexpr bool kAhead = MT <= 2;               // registers for two groups
    // (rows that only keep base need nothing when it is y already)
    const int groups = a.y && own < ntiles && (nmt > 0 || a.base != a.y) ? a.out_width / 64 : 0;
    const int first = warp * ctas + cta;
    // W2 rows of 16-rank step s at column group `grp`
    auto load_w2 = [&](int s, int grp, uint4 (&f)[4]) {
        const uint8_t *p = w2 + (size_t)grp * 128 + g * 16;
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const int j = 16 * s + 2 * q + (i & 1) + (i >> 1) * 8;
            f[i] = ld16_or_zero(p + j * out_pitch, j < rank);
        }
    };
    int yrow[2];                                   // rows 2q, 2q+1 of the tile
#pragma unroll
    for (int i = 0; i < 2; i++)
        yrow[i] = 2 * q + i < t.z ? perm[t.y + 2 * q + i] : -1;
    auto load_base = [&](int grp, uint4 (&f)[2]) {
#pragma unroll
        for (int i = 0; i < 2; i++)
            f[i] = ld16_or_zero(static_cast<const uint8_t *>(a.base) + (yrow[i] < 0 ? 0 : yrow[i]) * out_pitch +
                                    (size_t)grp * 128 + g * 16,
                                a.base != nullptr && yrow[i] >= 0);
    };
    uint4 pre[kPre][4], fb[2];
    if (first < groups) {
#pragma unroll
        for (int s = 0; s < kPre; s++)
            if (s < nmt)
                load_w2(s, first, pre[s]);
        load_base(first, fb);
    }
    if (__syncthreads_or(bad)) {                   // the same verdict in every CTA
        if (blockIdx.x == 0 && tid == 0)
            a.hdr[kHdrError] = EXL3_DERR_TABLE;
        zero_fill();
        return;
    }
    if (blockIdx.x == 0 && tid == 0)
        a.hdr[kHdrError] = 0;
    if (own >= ntiles)
        return;                                    // the whole cluster
    const int n4 = nmt * 16 * (kRows / 4);         // float4s of h, [rank][row]
    for (int i = tid; i < n4; i += kThreads) {
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarps; w++) {
            const float4 f = reinterpret_cast<const float4 *>(red + w * (16 * MT * kRows))[i];
            v.x += f.x; v.y += f.y; v.z += f.z; v.w += f.w;
        }
        reinterpret_cast<float4 *>(hpart)[i] = v;
    }
    cluster_sync();
    const float hs = a.scale_h ? alpha : 1.0f;
    for (int i = tid; i < n4; i += kThreads) {
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f), f[8];
#pragma unroll
        for (int r = 0; r < 8; r++)
            f[r] = ld_cluster(smem_addr(hpart) + i * 16, min(r, ctas - 1));
#pragma unroll
        for (int r = 0; r < 8; r++)
            if (r < ctas) {
                v.x += f[r].x; v.y += f[r].y; v.z += f[r].z; v.w += f[r].w;
            }
        const int j = i / (kRows / 4), r = i % (kRows / 4) * 4;
        const float z[4] = {v.x * hs, v.y * hs, v.z * hs, v.w * hs};
#pragma unroll
        for (int e = 0; e < 4; e++) {
            uint32_t hi, lo;
            split2(j < rank ? z[e] : 0.0f, 0.0f, dtype, hi, lo);
            h16[(r + e) * kPitch + j] = (uint16_t)hi;
            h16[(kRows + r + e) * kPitch + j] = (uint16_t)lo;
            if (a.h && cta == 0 && r + e < t.z) {
                uint16_t *h = static_cast<uint16_t *>(a.h) + (size_t)(t.y + r + e) * lora_h_pitch(a.h_cols) + j;
                h[0] = (uint16_t)hi;
                h[a.h_cols] = (uint16_t)lo;
            }
        }
    }
    // from here on the cluster's other CTAs may still be reading hpart
    cluster_arrive();
    __syncthreads();
    const float ys = a.scale_h ? 1.0f : alpha;
    for (int grp = first; grp < groups; grp += all_warps) {
        constexpr int kAcc = BF ? 4 : 8, kRest = kAcc - 4;     // f16: the rests' products from kRest on
        float acc[kAcc][4];
#pragma unroll
        for (int i = 0; i < kAcc; i++)
#pragma unroll
            for (int e = 0; e < 4; e++)
                acc[i][e] = 0.0f;
        if (grp != first && !kAhead)
            load_base(grp, fb);
        uint4 cur[kPre][4], cb[2] = {fb[0], fb[1]};
#pragma unroll
        for (int s = 0; s < kPre; s++)
#pragma unroll
            for (int i = 0; i < 4; i++)
                cur[s][i] = pre[s][i];
        if (kAhead && grp + all_warps < groups) {  // the next group's, while this one is worked on
#pragma unroll
            for (int s = 0; s < kPre; s++)
                if (s < nmt)
                    load_w2(s, grp + all_warps, pre[s]);
            load_base(grp + all_warps, fb);
        }
#pragma unroll
        for (int s = 0; s < MT; s++)
            if (s < nmt) {
                uint4 f[4];
                if (s < kPre && (kAhead || grp == first)) {
#pragma unroll
                    for (int i = 0; i < 4; i++)
                        f[i] = cur[s < kPre ? s : 0][i];
                } else {
                    load_w2(s, grp, f);
                }
                const uint32_t *hb = reinterpret_cast<const uint32_t *>(h16 + g * kPitch + 16 * s + 2 * q);
                const uint32_t b0 = hb[0], b1 = hb[4];
                const uint32_t l0 = hb[kRows * kPitch / 2], l1 = hb[kRows * kPitch / 2 + 4];
                const uint32_t *pa = reinterpret_cast<const uint32_t *>(&f[0]);
                const uint32_t *pb = reinterpret_cast<const uint32_t *>(&f[1]);
                const uint32_t *pc = reinterpret_cast<const uint32_t *>(&f[2]);
                const uint32_t *pd = reinterpret_cast<const uint32_t *>(&f[3]);
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const uint32_t sel = i & 1 ? 0x7632u : 0x5410u;
                    const uint32_t a0 = prmt(pa[i / 2], pb[i / 2], sel), a1 = prmt(pa[2 + i / 2], pb[2 + i / 2], sel);
                    const uint32_t a2 = prmt(pc[i / 2], pd[i / 2], sel), a3 = prmt(pc[2 + i / 2], pd[2 + i / 2], sel);
                    mma16816<BF>(acc[i], a0, a1, a2, a3, b0, b1);
                    mma16816<BF>(acc[kRest + i], a0, a1, a2, a3, l0, l1);
                }
            }
        if constexpr (!BF) {
#pragma unroll
            for (int i = 0; i < 4; i++)
#pragma unroll
                for (int e = 0; e < 4; e++)
                    acc[i][e] = fmaf(acc[kRest + i][e], 1.0f / (1 << kRestBits), acc[i][e]);
        }
        // lane: rows 2q, 2q+1 (accumulators 0, 1 of columns 0-3; 2, 3 of columns 4-7)
#pragma unroll
        for (int i = 0; i < 2; i++) {
            if (yrow[i] < 0)
                continue;
            uint4 u = cb[i];
            if (nmt > 0) {
                uint32_t *pu = reinterpret_cast<uint32_t *>(&u);
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    const float2 f = unpack2(pu[e], dtype);
                    const int lo = (2 * e) & 3, up = (e >= 2) * 2 + i;
                    pu[e] = pack2(fmaf(ys, acc[lo][up], f.x), fmaf(ys, acc[lo + 1][up], f.y), dtype);
                }
            }
            *reinterpret_cast<uint4 *>(static_cast<uint8_t *>(a.y) + yrow[i] * out_pitch + (size_t)grp * 128 + g * 16) = u;
        }
    }
    cluster_wait();                                // nobody reads this CTA's partials any more
}

template <bool BF, int MT>
cudaError_t launch(const LoraRowsArgs &a, int clusters, cudaStream_t s)
{
    cudaLaunchAttribute at[2] = {};
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = a.ctas;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(clusters * a.ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = rows_smem<MT>();
    cfg.stream = s;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, k_lora_rows<BF, MT>, a);
}

template <bool BF>
cudaError_t launch_ranks(const LoraRowsArgs &a, int clusters, cudaStream_t s)
{
    if (a.h_cols <= 16)
        return launch<BF, 1>(a, clusters, s);
    if (a.h_cols <= 32)
        return launch<BF, 2>(a, clusters, s);
    return a.h_cols <= 64 ? launch<BF, 4>(a, clusters, s) : launch<BF, 8>(a, clusters, s);
}

}  // namespace

}  // namespace lora

cudaError_t launch_lora_rows(LoraRowsArgs a, int sms, cudaStream_t s)
{
    // at most this many tiles: full ones, and one more per adapter in use and for rows without one
    const int clusters = a.M / kLoraSmallTile + (a.N < a.M ? a.N : a.M) + 1;
    // as many CTAs per tile as fit in one wave (two per SM), two at least: a
    // second wave starts with the whole chain of look-ups again (64 rows over 40
    // adapters: 10.3 us a call with four, 13.2 with eight in two waves)
    a.ctas = clusters * 8 <= 2 * sms ? 8 : clusters * 4 <= 2 * sms ? 4 : 2;
    return a.act_dtype == EXL3_BF16 ? lora::launch_ranks<true>(a, clusters, s)
                                    : lora::launch_ranks<false>(a, clusters, s);
}

}  // namespace exl3
