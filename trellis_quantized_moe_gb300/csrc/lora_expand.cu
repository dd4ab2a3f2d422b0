// Adapters, second product: y[perm[s]][n] = base[perm[s]][n] + alpha * sum_j
// h[s][j] W_a[j][n] over the rows grouped by adapter (h B forward, dh A
// backward), with h in two parts as k_lora_join leaves it.
//
// Bound by reading base and writing y once (2 r products per 4 bytes).  An
// item is a tile of 128 rows x 128 outputs; a CTA takes a contiguous share of
// the items, so a tile's h is fetched once per CTA and stays on chip for its
// output blocks: in TMEM, as the MMA's A, h's two parts one after the other
// along the contraction (both against the same W block).  From shared memory
// that doubled contraction took 53 us instead of 35 in the largest case below
// and left the ring room for items of 64 outputs only: its rows pass through
// shared memory four times, W's two, and A would be read anew for every item.
// Two groups of loader warps take turns on the items and copy base rows
// (gathered) and the W block by cp.async; an epilogue thread owns a row, adds
// its accumulator (TMEM) to the row in place, and the warp then writes its 32
// rows out, 128 contiguous bytes at a time.  Row slots have 16 bytes of
// padding: a thread per row has no bank conflicts.  (One bulk copy per 256-byte
// row, in and out, took 38 cycles a copy: 5 us an item.)
//
// Measured: 16384 rows, 1536 outputs, rank 16: 19.5 us for 100 MB read and
// written (5.1 TB/s; 15.4 us at the copy rate, most of the rest before the
// first item ends); 8192 rows, 5120 outputs, ranks 64 and 128: 35 us after the
// kernel before for 168 MB.  Four epilogue warps instead of eight took 1.9 us
// an item instead of 1; a third accumulator, which fits beside h of ranks up
// to 64, saves 0.6 us a launch (4096 rows).
#include "lora_common.cuh"

namespace exl3 {
namespace lora {

namespace {

constexpr int kThreads = 672;       // 8 loader, 8 epilogue warps, MMA warp, 4 warps for h
constexpr int kMmaWarp = 16, kHWarp = 17, kHThreads = 128;
constexpr int kMaxRing = 4;
constexpr int kItemN = 128;             // outputs of an item
constexpr int kTmemCols = 512;
constexpr int kMaxTBufs = 3;

// TMEM: 3 or 2 accumulators, then two buffers of h (two parts, two values a column).
EXL3_HD inline int h_tcols(int h_cols) { return h_cols <= 64 ? 64 : 128; }
EXL3_HD inline int tbufs(int h_cols) { return h_cols <= 64 ? 3 : 2; }

// Shared memory by largest rank: slots of 128 padded rows and a W block.
struct Geom {
    int pitch, row_bytes, slot_bytes, nslots, total;
};
EXL3_HD inline Geom geom(int h_cols)
{
    Geom g{};
    g.pitch = kItemN * 2 + 16;
    g.row_bytes = 128 * g.pitch;                       // a multiple of 1024
    g.slot_bytes = g.row_bytes + h_cols * kItemN * 2;
    const int n = 220 * 1024 / g.slot_bytes;
    g.nslots = n < kMaxRing ? n : kMaxRing;
    g.total = g.nslots * g.slot_bytes;
    return g;
}

struct Ctl {
    uint64_t hfull[2], hempty[2], full[kMaxRing], empty[kMaxRing], tfull[kMaxTBufs], tempty[kMaxTBufs],
        drain;
    uint32_t tmem;
    int abort;
};

__global__ void __launch_bounds__(kThreads, 1) k_lora_expand(LoraExpandArgs a)
{
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ Ctl c;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    grid_dep_launch();
    // an error zero-fills y: 128 threads of every CTA, this one the i0-th
    auto zero_fill = [&](int i0) {
        const size_t all = i0 < 128 ? (size_t)a.M * a.width / 8 : 0;
        for (size_t i = (size_t)blockIdx.x * 128 + i0; i < all; i += (size_t)gridDim.x * 128)
            static_cast<uint4 *>(a.y)[i] = make_uint4(0, 0, 0, 0);
    };
    if (!plan_ok(a.plan, a.M, a.N)) {
        grid_dep_wait();            // (waited for by the kernels after)
        zero_fill(tid);
        return;
    }
    const LoraPlanLayout L = lora_plan_layout(a.M, a.N);
    const int4 *tiles = reinterpret_cast<const int4 *>(a.plan + L.tiles / 4);
    const int32_t *perm = a.plan + L.perm / 4;
    const int active = a.plan[kLpActive];
    // rows without an adapter need nothing when y is base already
    const int ntiles = a.base == a.y ? active : a.plan[kLpTiles];
    const int nb = a.width / kItemN;
    const int total = ntiles * nb, per = lora_share(total, gridDim.x, 1);
    const int begin = blockIdx.x * per, end = min(total, begin + per);
    if (begin >= end) {
        grid_dep_wait();
        if (a.hdr[kHdrError])
            zero_fill(tid);
        return;
    }
    const Geom g = geom(a.h_cols);
    uint8_t *ring = smem;
    volatile int *abort = &c.abort;
    if (tid == 0) {
        for (int i = 0; i < 2; i++) {
            mbar_init(&c.hfull[i], kHThreads);
            mbar_init(&c.hempty[i], 1);
        }
        for (int i = 0; i < kMaxRing; i++) {
            mbar_init(&c.full[i], 128);
            mbar_init(&c.empty[i], 257);             // the epilogue's threads and the MMA thread
        }
        for (int i = 0; i < tbufs(a.h_cols); i++) {
            mbar_init(&c.tfull[i], 1);
            mbar_init(&c.tempty[i], 256);
        }
        mbar_init(&c.drain, 1);
        c.abort = 0;
        fence_mbar_init();
    }
    if (warp == kMmaWarp)
        tmem_alloc(&c.tmem, kTmemCols);
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

    if (warp < 8) {
        // group 0 takes the even items of the share, group 1 the odd ones
        constexpr int kLanes = kItemN / 8, kStep = 128 / kLanes, kN = 128 / kStep;   // lanes per row, rows a pass
        const int group = warp >> 2, gt = tid & 127, ch = gt % kLanes, r0 = gt / kLanes;
        Ring put;
        put.slot = group;
        int rank = 0, rp = 0;
        int row[kN], next_row[kN];                 // rows r0 + i kStep of this tile and the next; -1: none
        const size_t pitch = (size_t)a.width * 2;
        const uint8_t *W = nullptr;
        // a tile's rows are looked up one tile ahead, its descriptor two
        int tile = -1, known = (begin + group) / nb;           // known: the tile next_t describes
        const int last_tile = (end - 1) / nb;
        int4 next_t = tiles[min(known, last_tile)], next2_t = tiles[min(known + 1, last_tile)];
        auto look_up = [&]() {
#pragma unroll
            for (int i = 0; i < kN; i++)
                next_row[i] = a.base && r0 + i * kStep < next_t.z ? perm[next_t.y + r0 + i * kStep] : -1;
        };
        look_up();
        for (int s = begin + group; s < end; s += 2) {
            if (s / nb != tile) {
                tile = s / nb;
                if (tile != known) {                           // nb = 1: a tile was the other group's
                    next_t = next2_t;
                    look_up();
                    next2_t = tiles[min(tile + 1, last_tile)];
                }
                rank = tile_rank(next_t);
                rp = (rank + 15) / 16 * 16;
                W = rank ? reinterpret_cast<const uint8_t *>(a.W[next_t.x]) + r0 * pitch + ch * 16 : nullptr;
#pragma unroll
                for (int i = 0; i < kN; i++)
                    row[i] = next_row[i];
                next_t = next2_t;
                look_up();
                known = tile + 1;
                next2_t = tiles[min(tile + 2, last_tile)];
            }
            if (!wait_bar(&c.empty[put.slot], put.phase ^ 1, abort, a.hdr))
                break;
            const size_t col = (size_t)(s - tile * nb) * (kItemN * 2);
            const uint32_t dst = smem_addr(ring + put.slot * g.slot_bytes), db = dst + r0 * g.pitch + ch * 16;
            const uint8_t *base = static_cast<const uint8_t *>(a.base) + col + ch * 16;
#pragma unroll
            for (int i = 0; i < kN; i++)
                if (row[i] >= 0)
                    cp_async16(db + i * kStep * g.pitch, base + row[i] * pitch, true);
            const uint32_t dw = dst + g.row_bytes + (ch >> 3) * (rp * 128);
            const uint8_t *w = W + col;
            for (int j = r0; j < rp; j += kStep, w += kStep * pitch)
                cp_async16(dw + swz(j, ch & 7), j < rank ? w : W, j < rank);
            cp_async_arrive(&c.full[put.slot]);
            put.next2(g.nslots);
        }
        cp_async_wait_all();
    } else if (warp >= kHWarp) {
        // h of each tile into TMEM, a row a lane: rp / 8 chunks of 16 bytes, and
        // as many of the rests
        const int q = warp & 3, row = 32 * q + lane;
        Ring hb;
        grid_dep_wait();                           // h comes from the kernels before
        for (int s = begin; s < end;) {
            const int tile = s / nb;
            const int4 t = tiles[tile];
            const int rank = tile_rank(t), hc = (rank + 15) / 16 * 2;
            if (rank > 0) {
                if (!warp_wait_bar(&c.hempty[hb.slot], hb.phase ^ 1, abort, a.hdr))
                    break;
                fence_after();
                const uint32_t dst = c.tmem + ((uint32_t)(32 * q) << 16) + tbufs(a.h_cols) * kItemN + hb.slot * h_tcols(a.h_cols);
                const uint8_t *h = static_cast<const uint8_t *>(a.h) +
                                   (size_t)(t.y + min(row, t.z - 1)) * lora_h_pitch(a.h_cols) * 2;
                for (int i = 0; i < 2 * hc; i += 8) {          // 2 hc is a multiple of 4
                    uint4 v[2][4];
#pragma unroll
                    for (int e = 0; e < 8; e++) {
                        const int k = min(i + e, 2 * hc - 1);
                        v[e >> 2][e & 3] = *reinterpret_cast<const uint4 *>(
                            h + (k < hc ? k * 16 : a.h_cols * 2 + (k - hc) * 16));
                    }
                    tmem_st16(dst + i * 4, v[0]);
                    if (i + 4 < 2 * hc)
                        tmem_st16(dst + i * 4 + 16, v[1]);
                }
                tmem_st_wait();
                fence_before();
                mbar_arrive(&c.hfull[hb.slot]);
                hb.next(2);
            }
            s = (tile + 1) * nb;
        }
    } else if (warp >= 8 && warp < kMmaWarp) {
        // warps 8 + q and 12 + q: rows 32 q .. 32 q + 31, half the columns each
        constexpr int kCols = kItemN / 2, kLanes = kCols / 8, kRows = 32 / kLanes;   // rows of one warp-wide store
        const int q = warp & 3, c0 = (warp - 8) / 4 * kCols, row = 32 * q + lane;
        grid_dep_wait();                           // the error word
        const bool bad = a.hdr[kHdrError] != 0;
        Ring t4, in;
        for (int s = begin; s < end;) {
            const int tile = s / nb, last = min(end, (tile + 1) * nb);
            const int4 t = tiles[tile];
            const bool mma = tile_rank(t) > 0;
            const float alpha = mma && !a.scale_h ? a.scale[t.x] : 1.0f;
            const size_t off = row < t.z ? (size_t)perm[t.y + row] * a.width * 2 : 0;
            const int rows = bad ? 0 : min(32, t.z - 32 * q);      // of this warp, to be written
            bool ok = true;
            for (; s < last; s++) {
                ok = wait_bar(&c.full[in.slot], in.phase, abort, a.hdr) &&
                     (!mma || wait_bar(&c.tfull[t4.slot], t4.phase, abort, a.hdr));
                if (!(ok = __all_sync(0xffffffffu, ok)))
                    break;
                fence_after();
                uint8_t *warp_rows = ring + in.slot * g.slot_bytes + 32 * q * g.pitch + c0 * 2;
                uint8_t *mine = warp_rows + lane * g.pitch;
                const uint32_t acc = c.tmem + ((uint32_t)(32 * q) << 16) + t4.slot * kItemN + c0;
                if ((mma || !a.base) && rows > 0) {            // warps past the tile's rows only keep step
#pragma unroll
                    for (int n = 0; n < kCols; n += 32) {
                        uint32_t v[32] = {};
                        if (mma)
                            tmem_ld32(acc + n, v);
#pragma unroll
                        for (int i = 0; i < 32; i += 8) {
                            uint4 u = make_uint4(0, 0, 0, 0);
                            if (a.base)
                                u = *reinterpret_cast<const uint4 *>(mine + (n + i) * 2);
                            uint32_t *pu = reinterpret_cast<uint32_t *>(&u);
#pragma unroll
                            for (int e = 0; e < 4; e++) {
                                const float2 f = unpack2(pu[e], a.act_dtype);
                                pu[e] = pack2(fmaf(alpha, __uint_as_float(v[i + 2 * e]), f.x),
                                              fmaf(alpha, __uint_as_float(v[i + 2 * e + 1]), f.y), a.act_dtype);
                            }
                            *reinterpret_cast<uint4 *>(mine + (n + i) * 2) = u;
                        }
                    }
                }
                if (mma) {
                    fence_before();
                    mbar_arrive(&c.tempty[t4.slot]);
                    t4.next(tbufs(a.h_cols));
                }
                __syncwarp();
                uint8_t *out = static_cast<uint8_t *>(a.y) + (size_t)(s - tile * nb) * (kItemN * 2) + c0 * 2 +
                               lane % kLanes * 16;
#pragma unroll
                for (int r0 = 0; r0 < 32; r0 += kRows) {
                    if (r0 >= rows)
                        break;
                    const int r = r0 + lane / kLanes;
                    const size_t o = __shfl_sync(0xffffffffu, off, r);
                    const uint4 u = *reinterpret_cast<const uint4 *>(warp_rows + r * g.pitch + lane % kLanes * 16);
                    if (r < rows)
                        *reinterpret_cast<uint4 *>(out + o) = u;
                }
                mbar_arrive(&c.empty[in.slot]);
                in.next(g.nslots);
            }
            if (!ok)
                break;
        }
        if (bad)
            zero_fill(tid - 256);
    } else if (warp == kMmaWarp && lane == 0) {
        Ring hb, in, t4;
        bool ok = true;
        for (int s = begin; s < end && ok;) {
            const int tile = s / nb, last = min(end, (tile + 1) * nb);
            const int rank = tile_rank(tiles[tile]), rp = (rank + 15) / 16 * 16;
            // Items without an MMA (no adapter, or one of rank 0) are waited for
            // and handed back all the same: a thread that left them out could be
            // a whole turn of the ring ahead of the loaders, or behind them, and
            // the phase's parity would not tell.
            if (rank == 0) {
                for (; s < last; s++) {
                    if (!(ok = wait_bar(&c.full[in.slot], in.phase, abort, a.hdr)))
                        break;
                    mbar_arrive(&c.empty[in.slot]);
                    in.next(g.nslots);
                }
                continue;
            }
            const uint32_t id = idesc(kItemN, a.act_dtype, 0, 1);
            if (!(ok = wait_bar(&c.hfull[hb.slot], hb.phase, abort, a.hdr)))
                break;
            const uint32_t hs = c.tmem + tbufs(a.h_cols) * kItemN + hb.slot * h_tcols(a.h_cols);
            fence_after();
            for (; s < last; s++) {
                if (!(ok = wait_bar(&c.full[in.slot], in.phase, abort, a.hdr) &&
                           wait_bar(&c.tempty[t4.slot], t4.phase ^ 1, abort, a.hdr)))
                    break;
                fence_proxy();
                fence_after();
                const uint32_t ws = smem_addr(ring + in.slot * g.slot_bytes + g.row_bytes);
                const int steps = rp / 16;
                // h's two parts against the same W: the rests first, whose sum
                // the first MMA of the values then divides
                const uint32_t acc = c.tmem + t4.slot * kItemN, rests = hs + 8 * steps;
                for (int k = 0; k < steps; k++)
                    mma_f16_a_tmem(acc, rests + 8 * k, desc_mn_major(ws + k * 2048, rp * 128), id, k > 0);
                if (a.act_dtype == EXL3_F16)
                    mma_f16_a_tmem_unscale(acc, hs, desc_mn_major(ws, rp * 128), id);
                else
                    mma_f16_a_tmem(acc, hs, desc_mn_major(ws, rp * 128), id, true);
                for (int k = 1; k < steps; k++)
                    mma_f16_a_tmem(acc, hs + 8 * k, desc_mn_major(ws + k * 2048, rp * 128), id, true);
                mma_commit(&c.tfull[t4.slot]);
                mbar_arrive(&c.empty[in.slot]);        // (the epilogue's wait for the MMAs' end)
                in.next(g.nslots);
                t4.next(tbufs(a.h_cols));
            }
            mma_commit(&c.hempty[hb.slot]);
            hb.next(2);
        }
        if (!ok)
            drain_mmas(&c.drain);
    }
    fence_before();
    __syncthreads();
    fence_after();
    __syncwarp();
    if (warp == kMmaWarp)
        tmem_free(c.tmem, kTmemCols);
}

}  // namespace

}  // namespace lora

cudaError_t lora_expand_set_attributes()
{
    return cudaFuncSetAttribute(lora::k_lora_expand, cudaFuncAttributeMaxDynamicSharedMemorySize, 220 * 1024);
}

cudaError_t launch_lora_expand(const LoraExpandArgs &a, int ctas, cudaStream_t s)
{
    return lora::launch_dependent(lora::k_lora_expand, ctas, lora::kThreads, lora::geom(a.h_cols).total, s, a);
}

}  // namespace exl3
