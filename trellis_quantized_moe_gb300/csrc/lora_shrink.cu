// Adapters, first product: h[s][j] = sum_i x[perm[s]][i] W_a[j][i] over the
// rows grouped by adapter (x A^T forward, dy B^T backward).
//
// 2 r products per element of x (r <= 128) against 2 bytes: the kernel is
// bound by reading x once, so what counts is bytes in flight on every SM.
// The tiles' contractions, laid end to end as 128-wide stages, are shared out
// evenly over one CTA per SM whatever the tile count (a batch of few rows is
// split over its width, one of many is not); a tile cut by the shares leaves
// one fp32 partial per CTA, which k_lora_join adds in CTA order.  A stage
// is 128 rows x 256 bytes of x and the adapter's rank x 256 bytes of W, copied
// by cp.async (gathered rows: sixteen lanes per 256 bytes of a row) into a ring
// by two groups of loader warps that take turns; one thread issues tcgen05.mma
// (M = 128 rows, N = rank rounded up to 16), four warps drain the accumulator,
// double-buffered in TMEM.
//
// Measured: 16384 rows x 5120 bf16, rank 16: 36 us for 168 MB (4.7 TB/s); the
// same gathered copies through a ring without MMAs take 28.8.  Once running it
// holds 5.9 TB/s; the rest is the start (plan, tile, rows, first bytes one
// after the other: 5 us) and CTAs that end up to 4 us apart.  8192 rows, rank
// 128: 26 us, W through L2 adding as many bytes per stage as x.
#include "lora_common.cuh"

namespace exl3 {
namespace lora {

namespace {

constexpr int kThreads = 480;       // 8 loader warps in two groups, 4 epilogue, MMA, fence, check warp
constexpr int kXBytes = 2 * 128 * 128;   // two 64-wide blocks
constexpr int kRingBytes = 208 * 1024;
constexpr int kMaxSlots = 6;
constexpr int kBufCols = 128;       // TMEM columns per accumulator

EXL3_HD inline int stage_bytes(int h_cols) { return kXBytes + h_cols * 256; }
EXL3_HD inline int ring_slots(int h_cols)
{
    const int n = kRingBytes / stage_bytes(h_cols);
    return n < kMaxSlots ? n : kMaxSlots;
}

struct Ctl {
    uint64_t full[kMaxSlots], ready[kMaxSlots], empty[kMaxSlots], tfull[2], tempty[2], drain;
    uint32_t tmem;
    int abort;
};

// The tables of every adapter in use, by one warp of CTA 0 (the others start
// on their rows meanwhile).
__device__ void check_tables(const LoraShrinkArgs &a)
{
    int err;
    if (a.plan[kLpMagic] != kLoraMagic || a.plan[kLpM] != a.M || a.plan[kLpN] != a.N) {
        err = EXL3_DERR_PLAN;
    } else {
        err = a.plan[kLpError];
        const int32_t *off = a.plan + lora_plan_layout(a.M, a.N).offsets / 4;
#pragma unroll 4
        for (int i = threadIdx.x & 31; i < a.N; i += 32) {
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
    const bool table = __any_sync(0xffffffffu, err & EXL3_DERR_TABLE);
    if ((threadIdx.x & 31) == 0)
        a.hdr[kHdrError] = err | (table ? EXL3_DERR_TABLE : 0);
}

__global__ void __launch_bounds__(kThreads, 1) k_lora_shrink(LoraShrinkArgs a)
{
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ Ctl c;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    grid_dep_wait();                // plan, tables and rows may come from the kernel before
    grid_dep_launch();              // only now: the kernels after read them before their own wait
    if (blockIdx.x == 0 && warp == 14)
        check_tables(a);
    if (!plan_ok(a.plan, a.M, a.N))
        return;
    const LoraPlanLayout L = lora_plan_layout(a.M, a.N);
    const int4 *tiles = reinterpret_cast<const int4 *>(a.plan + L.tiles / 4);
    const int32_t *perm = a.plan + L.perm / 4;
    const int ks = a.width / kShrinkK, total = a.plan[kLpActive] * ks;
    const int per = lora_share(total, gridDim.x, kShrinkMin);
    const int begin = blockIdx.x * per, end = min(total, begin + per);
    if (begin >= end)
        return;
    const int sbytes = stage_bytes(a.h_cols), nslots = ring_slots(a.h_cols);
    volatile int *abort = &c.abort;
    if (tid == 0) {
        for (int i = 0; i < nslots; i++) {
            mbar_init(&c.full[i], 128);
            mbar_init(&c.ready[i], 1);
            mbar_init(&c.empty[i], 1);
        }
        for (int i = 0; i < 2; i++) {
            mbar_init(&c.tfull[i], 1);
            mbar_init(&c.tempty[i], 128);
        }
        mbar_init(&c.drain, 1);
        c.abort = 0;
        fence_mbar_init();
    }
    if (warp == 12)
        tmem_alloc(&c.tmem, 2 * kBufCols);
    fence_before();
    __syncthreads();
    fence_after();

    // rank of a tile's adapter as every role sees it: 0 for a bad table entry
    auto tile_rank = [&](int e) {
        const int r = a.rank[e];
        const int64_t w = a.W[e];
        return r < 0 || r > a.max_rank || !w || (w & 15) ? 0 : r;
    };

    if (warp < 8) {
        // group 0 takes the even stages of the share, group 1 the odd ones
        const int group = warp >> 2, gt = tid & 127, ch = gt & 15, r0 = gt >> 4;
        const size_t wstep = (size_t)a.width * 16;             // 8 rows of W
        int row[16], next_row[16];                 // rows r0 + 8 i of this tile and the next; -1: none
        const uint8_t *w = nullptr;
        const size_t pitch = (size_t)a.width * 2;
        int rank = 0, rp = 16;
        Ring put;
        put.slot = group;
        int tile = (begin + group) / ks, k = (begin + group) % ks;
        // A tile's rows are looked up one tile ahead, its descriptor two: a
        // look-up in the open drains the ring for two memory latencies.
        const int last_tile = (end - 1) / ks;
        int4 next_t = tiles[min(tile, last_tile)], next2_t = tiles[min(tile + 1, last_tile)];
        auto look_up = [&]() {
#pragma unroll
            for (int i = 0; i < 16; i++)
                next_row[i] = r0 + 8 * i < next_t.z ? perm[next_t.y + r0 + 8 * i] : -1;
        };
        look_up();
        bool fresh = true;
        for (int s = begin + group; s < end; s += 2) {
            if (fresh) {
                rank = tile_rank(next_t.x);
                rp = max(16, (rank + 15) / 16 * 16);
                w = reinterpret_cast<const uint8_t *>(a.W[next_t.x]) + (size_t)r0 * pitch + ch * 16;
#pragma unroll
                for (int i = 0; i < 16; i++)
                    row[i] = next_row[i];
                next_t = next2_t;
                look_up();
                next2_t = tiles[min(tile + 2, last_tile)];
                fresh = false;
            }
            if (!wait_bar(&c.empty[put.slot], put.phase ^ 1, abort, a.hdr))
                break;
            const uint32_t dst = smem_addr(smem + (size_t)put.slot * sbytes);
            const uint8_t *x = static_cast<const uint8_t *>(a.x) + (size_t)k * 256 + ch * 16;
            // 64-wide block ch / 8, row r0 + 8 i, chunk ch % 8
            const uint32_t dx = dst + (ch >> 3) * (128 * 128) + swz(r0, ch & 7);
#pragma unroll
            for (int i = 0; i < 16; i++)
                cp_async16(dx + i * 1024, row[i] < 0 ? x : x + row[i] * pitch, row[i] >= 0);
            const uint8_t *wk = w + (size_t)k * 256;
            const uint32_t dw = dst + kXBytes + (ch >> 3) * (rp * 128) + swz(r0, ch & 7);
            for (int i = 0; i < rp / 8; i++, wk += wstep) {
                const bool v = r0 + 8 * i < rank;
                cp_async16(dw + i * 1024, v ? wk : static_cast<const uint8_t *>(a.x), v);
            }
            cp_async_arrive(&c.full[put.slot]);
            put.next2(nslots);
            k += 2;
            if (k >= ks) {
                fresh = true;
                tile++;
                k -= ks;
                if (k >= ks) {                     // ks = 1: this group skips a tile
                    tile++;
                    k -= ks;
                    next_t = next2_t;
                    look_up();
                    next2_t = tiles[min(tile + 1, last_tile)];
                }
            }
        }
        cp_async_wait_all();
    } else if (warp < 12) {
        const int q = warp & 3, row = 32 * q + lane;
        int tile = begin / ks;
        Ring t;
        for (int s = begin; s < end; tile++) {
            const int4 ti = tiles[tile];
            const int rp = max(16, (tile_rank(ti.x) + 15) / 16 * 16);
            if (!warp_wait_bar(&c.tfull[t.slot], t.phase, abort, a.hdr))
                break;
            fence_after();
            float *out = a.part + ((size_t)ti.y + 128 * (size_t)blockIdx.x + row) * a.h_cols;
            const uint32_t addr = c.tmem + ((uint32_t)(32 * q) << 16) + t.slot * kBufCols;
            for (int j = 0; j < rp; j += 16) {
                uint32_t v[16];
                tmem_ld16_issue(addr + j, v);
                tmem_ld16_wait(v);
                if (row < ti.z)
#pragma unroll
                    for (int i = 0; i < 16; i += 4)
                        *reinterpret_cast<uint4 *>(out + j + i) = make_uint4(v[i], v[i + 1], v[i + 2], v[i + 3]);
            }
            fence_before();
            mbar_arrive(&c.tempty[t.slot]);
            t.next(2);
            s = (tile + 1) * ks;
        }
    } else if (warp == 12 && lane == 0) {
        int tile = begin / ks, k = begin % ks;
        Ring get, t;
        uint32_t id = 0;
        int rp = 16;
        bool fresh = true, ok = true;
        for (int s = begin; s < end && ok; s++) {
            if (fresh) {
                rp = max(16, (tile_rank(tiles[tile].x) + 15) / 16 * 16);
                id = idesc(rp, a.act_dtype, 0, 0);
                if (!(ok = wait_bar(&c.tempty[t.slot], t.phase ^ 1, abort, a.hdr)))
                    break;
                fence_after();
            }
            if (!(ok = wait_bar(&c.ready[get.slot], get.phase, abort, a.hdr)))
                break;
            fence_after();
            const uint32_t xs = smem_addr(smem + (size_t)get.slot * sbytes);
#pragma unroll
            for (int i = 0; i < 8; i++)
                mma_f16(c.tmem + t.slot * kBufCols, desc_k_major(xs + (i >> 2) * (128 * 128) + 32 * (i & 3)),
                        desc_k_major(xs + kXBytes + (i >> 2) * (rp * 128) + 32 * (i & 3)), id, !(fresh && i == 0));
            mma_commit(&c.empty[get.slot]);
            get.next(nslots);
            fresh = false;
            if (++k == ks || s + 1 == end) {
                mma_commit(&c.tfull[t.slot]);
                t.next(2);
                k = 0;
                tile++;
                fresh = true;
            }
        }
        if (!ok)
            drain_mmas(&c.drain);
    } else if (warp == 13 && lane == 0) {
        // the proxy fence between the copies and the MMAs, off the MMA
        // thread's path (one thread, every stage in order: a thread that left
        // stages out could meet a barrier a whole phase early)
        Ring get;
        for (int s = begin; s < end; s++) {
            if (!wait_bar(&c.full[get.slot], get.phase, abort, a.hdr))
                break;
            fence_proxy();
            mbar_arrive(&c.ready[get.slot]);
            get.next(nslots);
        }
    }
    fence_before();
    __syncthreads();
    fence_after();
    __syncwarp();
    if (warp == 12)
        tmem_free(c.tmem, 2 * kBufCols);
}

// Adds a tile's partials and splits the sums into the second product's operands.
// A thread has four columns of one row and the partials of four CTAs in flight
// (they lie in L2); a block takes as many rows as its threads have at the
// largest rank.
constexpr int kJoinThreads = 256;

EXL3_HD inline int join_lanes(int rank_cols) { return rank_cols <= 16 ? 4 : rank_cols <= 32 ? 8 : rank_cols <= 64 ? 16 : 32; }
EXL3_HD inline int join_rows(int h_cols) { return kJoinThreads / join_lanes(h_cols); }

__global__ void __launch_bounds__(kJoinThreads) k_lora_join(LoraJoinArgs a)
{
    grid_dep_launch();
    // (a CTA that has nothing to do waits too: the kernel after this one takes
    // its end for the end of the kernels before)
    if (!plan_ok(a.plan, a.M, a.N)) {
        grid_dep_wait();
        return;
    }
    const LoraPlanLayout L = lora_plan_layout(a.M, a.N);
    const int rows = join_rows(a.h_cols), blocks = kLoraTile / rows;
    const int active = a.plan[kLpActive], tile = blockIdx.x / blocks;
    if (tile >= active) {
        grid_dep_wait();
        return;
    }
    const int4 t = reinterpret_cast<const int4 *>(a.plan + L.tiles / 4)[tile];
    const int rank = min(max(a.rank[t.x], 0), a.h_cols), rp = (rank + 15) / 16 * 16;
    const float alpha = a.scale_h ? a.scale[t.x] : 1.0f;
    const int ks = a.shrink_width / kShrinkK, per = lora_share(active * ks, a.shrink_ctas, kShrinkMin);
    const int c0 = tile * ks / per, c1 = ((tile + 1) * ks - 1) / per;
    const int lanes = join_lanes(a.h_cols), j = threadIdx.x % lanes * 4;
    const int r = blockIdx.x % blocks * rows + threadIdx.x / lanes;
    grid_dep_wait();
    const int err = a.hdr[kHdrError];              // looked at before the store only
    if (j < rp && r < t.z) {
        const size_t cta = 128 * (size_t)a.h_cols;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        const float *p = a.part + (size_t)(t.y + r) * a.h_cols + j + c0 * cta;
        constexpr int kC = 4;
        for (int c = c0; c <= c1; c += kC, p += kC * cta) {
            float4 f[kC];
#pragma unroll
            for (int d = 0; d < kC; d++)
                f[d] = *reinterpret_cast<const float4 *>(p + min(d, c1 - c) * cta);
#pragma unroll
            for (int d = 0; d < kC; d++)
                if (c + d <= c1) {
                    v.x += f[d].x; v.y += f[d].y; v.z += f[d].z; v.w += f[d].w;
                }
        }
        if (err == 0) {
            uint2 hi, lo;
            split2(j < rank ? v.x * alpha : 0.f, j + 1 < rank ? v.y * alpha : 0.f, a.act_dtype, hi.x, lo.x);
            split2(j + 2 < rank ? v.z * alpha : 0.f, j + 3 < rank ? v.w * alpha : 0.f, a.act_dtype, hi.y, lo.y);
            uint16_t *h = static_cast<uint16_t *>(a.h) + (size_t)(t.y + r) * lora_h_pitch(a.h_cols) + j;
            *reinterpret_cast<uint2 *>(h) = hi;
            *reinterpret_cast<uint2 *>(h + a.h_cols) = lo;
        }
    }
}

}  // namespace

}  // namespace lora

cudaError_t launch_lora_join(const LoraJoinArgs &a, cudaStream_t s)
{
    const int tiles = a.M / kLoraTile + (a.N < a.M ? a.N : a.M);       // of adapters, at most
    return lora::launch_dependent(lora::k_lora_join, tiles * (kLoraTile / lora::join_rows(a.h_cols)),
                                  lora::kJoinThreads, 0, s, a);
}

cudaError_t lora_shrink_set_attributes()
{
    return cudaFuncSetAttribute(lora::k_lora_shrink, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                lora::kRingBytes);
}

cudaError_t launch_lora_shrink(const LoraShrinkArgs &a, int ctas, cudaStream_t s)
{
    const int smem = lora::ring_slots(a.h_cols) * lora::stage_bytes(a.h_cols);
    return lora::launch_dependent(lora::k_lora_shrink, ctas, lora::kThreads, smem, s, a);
}

}  // namespace exl3
