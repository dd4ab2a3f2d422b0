// Adapters, second product: y[perm[s]][n] = base[perm[s]][n] + alpha * sum_j
// h[s][j] W_a[j][n] over the rows grouped by adapter (h B forward, dh A
// backward), with h = the sum of the shrink kernel's partials.
//
// Bound by reading base and writing y once (2 r products per 4 bytes).  An
// item is a tile of 128 rows x 128 outputs; a CTA takes a contiguous share of
// the items, so a tile's h is joined once per CTA and stays in shared memory
// for its output blocks.  Rows of base arrive, and rows of y leave, as 256-byte
// bulk copies (one per row: the rows are scattered) into slots of 272-byte
// rows, a pitch on which a thread per row has no bank conflicts: the epilogue
// thread that owns a row reads its accumulator from TMEM, adds it to the row
// in place and sends the row off itself, with no exchange between threads.
#include "lora_common.cuh"

namespace exl3 {
namespace lora {

namespace {

constexpr int kThreads = 448;       // 4 W loader, 4 epilogue, MMA, base and 4 join warps
constexpr int kPitch = 272;         // bytes of a row slot: 256 + 16
constexpr int kRowSlot = 128 * kPitch;
constexpr int kTBufs = 4;           // TMEM accumulators of 128 columns
constexpr int kMaxRing = 4;

// Shared memory by largest rank: two buffers of h, W blocks, row slots.
struct Geom {
    int h_bytes, w_bytes, nw, nrow, total;
};
EXL3_HD inline Geom geom(int h_cols)
{
    Geom g;
    g.h_bytes = (h_cols + 63) / 64 * 128 * 128;
    g.w_bytes = h_cols * 256;
    g.nw = h_cols > 64 ? 2 : 3;
    g.nrow = h_cols > 64 ? 2 : 4;
    g.total = 2 * g.h_bytes + g.nw * g.w_bytes + g.nrow * kRowSlot;
    return g;
}

struct Ctl {
    uint64_t hfull[2], hempty[2], wfull[kMaxRing], wempty[kMaxRing], bfull[kMaxRing], bempty[kMaxRing],
        tfull[kTBufs], tempty[kTBufs];
    uint32_t tmem;
    int abort;
};

// Joins h of one tile, thread jt of 128: the partials of CTAs c0..c1 in that
// order, scaled, zero from the rank on, rounded; into shared memory (hs) and,
// with keep, into a.h.  A thread has four columns of up to eight rows in
// flight: the partials lie in L2, and one load at a time took longer (r = 128:
// 40 us a tile) than everything else in the kernel.
EXL3_DEV void join_h(const LoraExpandArgs &a, const int4 &t, int rank, int c0, int c1, float alpha, uint8_t *hs,
                     bool keep, int jt)
{
    constexpr int kU = 8;
    const int rp = (rank + 15) / 16 * 16;
    const int lq = rp <= 16 ? 2 : rp <= 32 ? 3 : rp <= 64 ? 4 : 5;   // lanes per row: 2^lq
    const int j = (jt & ((1 << lq) - 1)) * 4, step = 128 >> lq;
    if (j >= rp)
        return;
    const size_t cta = 128 * (size_t)a.h_cols;
    for (int r0 = jt >> lq; r0 < t.z; r0 += kU * step) {
        float4 v[kU];
#pragma unroll
        for (int u = 0; u < kU; u++)
            v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
        const float *p = a.part + (size_t)(t.y + r0) * a.h_cols + j + c0 * cta;
        for (int c = c0; c <= c1; c++, p += cta) {
#pragma unroll
            for (int u = 0; u < kU; u++)
                if (r0 + u * step < t.z) {
                    const float4 f = *reinterpret_cast<const float4 *>(p + (size_t)u * step * a.h_cols);
                    v[u].x += f.x; v[u].y += f.y; v[u].z += f.z; v[u].w += f.w;
                }
        }
#pragma unroll
        for (int u = 0; u < kU; u++) {
            const int r = r0 + u * step;
            if (r >= t.z)
                break;
            const float4 f = v[u];
            const uint2 o = make_uint2(
                pack2(j < rank ? f.x * alpha : 0.f, j + 1 < rank ? f.y * alpha : 0.f, a.act_dtype),
                pack2(j + 2 < rank ? f.z * alpha : 0.f, j + 3 < rank ? f.w * alpha : 0.f, a.act_dtype));
            if (hs)
                *reinterpret_cast<uint2 *>(hs + (j >> 6) * (128 * 128) + swz(r, (j & 63) >> 3) + (j & 4) * 2) = o;
            if (keep)
                *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.h) + (size_t)(t.y + r) * a.h_cols + j) = o;
        }
    }
}

__global__ void __launch_bounds__(kThreads, 1) k_lora_expand(LoraExpandArgs a)
{
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ Ctl c;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    grid_dep_launch();
    // an error zero-fills y: 128 threads of every CTA, this one the i0-th
    auto zero_fill = [&](int i0) {
        const size_t all = a.y && i0 < 128 ? (size_t)a.M * a.width / 8 : 0;
        for (size_t i = (size_t)blockIdx.x * 128 + i0; i < all; i += (size_t)gridDim.x * 128)
            static_cast<uint4 *>(a.y)[i] = make_uint4(0, 0, 0, 0);
    };
    if (!plan_ok(a.plan, a.M, a.N)) {
        zero_fill(tid);
        return;
    }
    const LoraPlanLayout L = lora_plan_layout(a.M, a.N);
    const int4 *tiles = reinterpret_cast<const int4 *>(a.plan + L.tiles / 4);
    const int32_t *perm = a.plan + L.perm / 4;
    const int active = a.plan[kLpActive];
    const int sks = a.shrink_width / kLoraK;
    const int sper = lora_share(active * sks, a.shrink_ctas, kLoraMinStages);
    // rows without an adapter need nothing when y is base already
    const int ntiles = !a.y || a.base == a.y ? active : a.plan[kLpTiles];
    const int nb = a.y ? a.width / 128 : 1;
    const int total = ntiles * nb, per = lora_share(total, gridDim.x, 1);
    const int begin = blockIdx.x * per, end = min(total, begin + per);
    if (begin >= end) {
        grid_dep_wait();
        if (a.hdr[kHdrError])
            zero_fill(tid);
        return;
    }
    const Geom g = geom(a.h_cols);
    uint8_t *hbuf = smem, *wring = smem + 2 * g.h_bytes, *rows = wring + g.nw * g.w_bytes;
    volatile int *abort = &c.abort;
    if (tid == 0) {
        for (int i = 0; i < 2; i++) {
            mbar_init(&c.hfull[i], 128);
            mbar_init(&c.hempty[i], 1);
        }
        for (int i = 0; i < kMaxRing; i++) {
            mbar_init(&c.wfull[i], 128);
            mbar_init(&c.wempty[i], 1);
            mbar_init(&c.bfull[i], 1);
            mbar_init(&c.bempty[i], 128);
        }
        for (int i = 0; i < kTBufs; i++) {
            mbar_init(&c.tfull[i], 1);
            mbar_init(&c.tempty[i], 128);
        }
        c.abort = 0;
        fence_mbar_init();
    }
    if (warp == 8)
        tmem_alloc(&c.tmem, 128 * kTBufs);
    fence_before();
    __syncthreads();
    fence_after();

    // rank of a tile's adapter as every role sees it: 0 for a bad table entry
    // (the error word, which shrink writes, is not there yet)
    auto tile_rank = [&](const int4 &t) {
        if (t.x < 0)
            return 0;
        const int r = a.rank[t.x];
        const int64_t w = a.W[t.x];
        return r < 0 || r > a.h_cols || !w || (w & 15) ? 0 : r;
    };

    if (warp < 4 && a.y) {
        // W blocks: rp rows of 256 bytes as two halves of 128-byte rows;
        // sixteen lanes per row
        const int ch = tid & 15, j0 = tid >> 4;
        Ring w, done;
        bool ok = true;
        int pending = 0;                           // W blocks in flight
        auto finish = [&]() {                      // the oldest of them has landed
            fence_proxy();
            mbar_arrive(&c.wfull[done.slot]);
            done.next(g.nw);
            pending--;
        };
        for (int s = begin; s < end && ok;) {
            const int tile = s / nb, last = min(end, (tile + 1) * nb);
            const int4 t = tiles[tile];
            const int rank = tile_rank(t), rp = (rank + 15) / 16 * 16;
            if (rank == 0) {
                s = last;
                continue;
            }
            const uint8_t *W = reinterpret_cast<const uint8_t *>(a.W[t.x]);
            for (; s < last; s++) {
                if (!(ok = wait_bar(&c.wempty[w.slot], w.phase ^ 1, abort, a.hdr)))
                    break;
                const uint32_t dst = smem_addr(wring + w.slot * g.w_bytes) + (ch >> 3) * (rp * 128);
                const uint8_t *src = W + (size_t)(s % nb) * 256 + ch * 16;
                for (int j = j0; j < rp; j += 8)
                    cp_async16(dst + swz(j, ch & 7), j < rank ? src + (size_t)j * a.width * 2 : W, j < rank);
                cp_async_commit();
                w.next(g.nw);
                pending++;
                if (g.nw == 3 && pending > 2) {
                    cp_async_wait<2>();
                    finish();
                } else if (g.nw == 2 && pending > 1) {
                    cp_async_wait<1>();
                    finish();
                }
            }
        }
        cp_async_wait<0>();
        while (ok && pending)
            finish();
    } else if (warp >= 10) {
        grid_dep_wait();                           // the partials and the error word
        const bool bad = a.hdr[kHdrError] != 0;
        Ring hb;
        for (int s = begin; s < end;) {
            const int tile = s / nb, last = min(end, (tile + 1) * nb);
            const int4 t = tiles[tile];
            const int rank = tile_rank(t);
            if (rank > 0) {
                const float alpha = a.scale_h ? a.scale[t.x] : 1.0f;
                const int c0 = tile * sks / sper, c1 = ((tile + 1) * sks - 1) / sper;
                if (a.y && !wait_bar(&c.hempty[hb.slot], hb.phase ^ 1, abort, a.hdr))
                    break;
                if (!bad)
                    join_h(a, t, rank, c0, c1, alpha, a.y ? hbuf + hb.slot * g.h_bytes : nullptr,
                           a.h != nullptr && s % nb == 0, tid - 320);
                if (a.y) {
                    fence_proxy();
                    mbar_arrive(&c.hfull[hb.slot]);
                    hb.next(2);
                }
            }
            s = last;
        }
    } else if (warp >= 4 && warp < 8 && a.y) {
        const int q = warp & 3, row = 32 * q + lane;
        grid_dep_wait();                           // the error word
        const bool bad = a.hdr[kHdrError] != 0;
        Ring t4, b;
        int prev = -1;
        for (int s = begin; s < end;) {
            const int tile = s / nb, last = min(end, (tile + 1) * nb);
            const int4 t = tiles[tile];
            const bool live = row < t.z, mma = tile_rank(t) > 0;
            const float alpha = mma && !a.scale_h ? a.scale[t.x] : 1.0f;
            uint8_t *dst = static_cast<uint8_t *>(a.y) + (live ? (size_t)perm[t.y + row] * a.width * 2 : 0);
            bool ok = true;
            for (; s < last; s++) {
                ok = (!mma || wait_bar(&c.tfull[t4.slot], t4.phase, abort, a.hdr)) &&
                     (!a.base || wait_bar(&c.bfull[b.slot], b.phase, abort, a.hdr));
                if (!(ok = __all_sync(0xffffffffu, ok)))
                    break;
                fence_after();
                uint8_t *slot = rows + b.slot * kRowSlot + row * kPitch;
                const uint32_t acc = c.tmem + ((uint32_t)(32 * q) << 16) + t4.slot * 128;
#pragma unroll
                for (int n = 0; n < 128; n += 16) {
                    uint32_t v[16];
                    if (mma) {
                        tmem_ld16_issue(acc + n, v);
                        tmem_ld16_wait(v);
                    } else {
#pragma unroll
                        for (int i = 0; i < 16; i++)
                            v[i] = 0;
                    }
#pragma unroll
                    for (int i = 0; i < 16; i += 8) {
                        uint4 u = make_uint4(0, 0, 0, 0);
                        if (a.base)
                            u = *reinterpret_cast<const uint4 *>(slot + (n + i) * 2);
                        uint32_t *pu = reinterpret_cast<uint32_t *>(&u);
                        if (mma)
#pragma unroll
                            for (int e = 0; e < 4; e++) {
                                const float2 f = unpack2(pu[e], a.act_dtype);
                                pu[e] = pack2(fmaf(alpha, __uint_as_float(v[i + 2 * e]), f.x),
                                              fmaf(alpha, __uint_as_float(v[i + 2 * e + 1]), f.y), a.act_dtype);
                            }
                        *reinterpret_cast<uint4 *>(slot + (n + i) * 2) = u;
                    }
                }
                if (mma) {
                    fence_before();
                    mbar_arrive(&c.tempty[t4.slot]);
                    t4.next(kTBufs);
                }
                fence_proxy();
                if (live && !bad)
                    bulk_s2g(dst + (size_t)(s % nb) * 256, smem_addr(slot), 256);
                bulk_commit();
                bulk_wait_read<1>();               // the previous item's row has left its slot
                if (prev >= 0)
                    mbar_arrive(&c.bempty[prev]);
                prev = b.slot;
                b.next(g.nrow);
            }
            if (!ok)
                break;
        }
        bulk_wait_all();
        if (bad)
            zero_fill(tid - 128);
    } else if (warp == 8 && lane == 0 && a.y) {
        Ring hb, w, t4;
        bool ok = true;
        for (int s = begin; s < end && ok;) {
            const int tile = s / nb, last = min(end, (tile + 1) * nb);
            const int rank = tile_rank(tiles[tile]), rp = (rank + 15) / 16 * 16;
            if (rank == 0) {
                s = last;
                continue;
            }
            const uint32_t id = idesc(128, a.act_dtype, 0, 1);
            if (!(ok = wait_bar(&c.hfull[hb.slot], hb.phase, abort, a.hdr)))
                break;
            const uint32_t hs = smem_addr(hbuf + hb.slot * g.h_bytes);
            for (; s < last; s++) {
                if (!(ok = wait_bar(&c.wfull[w.slot], w.phase, abort, a.hdr) &&
                           wait_bar(&c.tempty[t4.slot], t4.phase ^ 1, abort, a.hdr)))
                    break;
                fence_after();
                const uint32_t ws = smem_addr(wring + w.slot * g.w_bytes);
                for (int k = 0; k < rp / 16; k++)
                    mma_f16(c.tmem + t4.slot * 128, desc_k_major(hs + (k >> 2) * (128 * 128) + (k & 3) * 32),
                            desc_mn_major(ws + k * 2048, rp * 128), id, k > 0);
                mma_commit(&c.wempty[w.slot]);
                mma_commit(&c.tfull[t4.slot]);
                w.next(g.nw);
                t4.next(kTBufs);
            }
            mma_commit(&c.hempty[hb.slot]);
            hb.next(2);
        }
    } else if (warp == 9 && a.y && a.base) {
        Ring b;
        bool ok = true;
        for (int s = begin; s < end && ok;) {
            const int tile = s / nb, last = min(end, (tile + 1) * nb);
            const int4 t = tiles[tile];
            const uint8_t *src[4];
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const int r = lane + 32 * i;
                src[i] = r < t.z ? static_cast<const uint8_t *>(a.base) + (size_t)perm[t.y + r] * a.width * 2 : nullptr;
            }
            for (; s < last; s++) {
                if (!(ok = warp_wait_bar(&c.bempty[b.slot], b.phase ^ 1, abort, a.hdr)))
                    break;
                if (lane == 0)
                    mbar_arrive_expect_tx(&c.bfull[b.slot], t.z * 256);
                __syncwarp();
                uint8_t *slot = rows + b.slot * kRowSlot;
#pragma unroll
                for (int i = 0; i < 4; i++)
                    if (src[i])
                        bulk_g2s(slot + (lane + 32 * i) * kPitch, src[i] + (size_t)(s % nb) * 256, 256,
                                 &c.bfull[b.slot]);
                b.next(g.nrow);
            }
        }
        // after a timeout elsewhere: copies in flight land before the CTA exits
        if (!ok || *abort)
            for (int i = 0; i < g.nrow; i++)
                mbar_wait(&c.bfull[i], (b.slot > (uint32_t)i ? b.phase : b.phase ^ 1));
    }
    fence_before();
    __syncthreads();
    fence_after();
    __syncwarp();
    if (warp == 8)
        tmem_free(c.tmem, 128 * kTBufs);
}

}  // namespace

}  // namespace lora

cudaError_t lora_expand_set_attributes()
{
    const int a = lora::geom(16).total, b = lora::geom(64).total, d = lora::geom(128).total;
    return cudaFuncSetAttribute(lora::k_lora_expand, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                a > b ? (a > d ? a : d) : (b > d ? b : d));
}

cudaError_t launch_lora_expand(const LoraExpandArgs &a, int ctas, cudaStream_t s)
{
    return lora::launch_dependent(lora::k_lora_expand, ctas, lora::kThreads, lora::geom(a.h_cols).total, s, a);
}

}  // namespace exl3
