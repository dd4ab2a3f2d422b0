// Adapters, gradients of the weights: G_a[j][n] = scale * sum_s h[s][j]
// x[perm[s]][n] over each adapter's rows, for dA (dh, x) and dB (h, dy) in one
// launch.
//
// 2 r products per element of x or dy against 2 bytes: bound by reading both
// once.  An item is an adapter's 256 columns (two accumulators of 128 lanes,
// so that h is fetched half as often); its contraction runs over the
// rows in 64-row stages.  All stages of both products, laid end to end, are
// shared out evenly over one CTA per SM; an item inside one share is written
// out at once, one cut by the shares leaves at most two fp32 partials per CTA
// for the join kernel, which adds them in CTA order (no atomics: the same bits
// every time).  The rows come in as they lie in memory: both MMA operands are
// MN-major (x^T gives the 128 accumulator lanes, h the columns), so nothing is
// transposed.
//
// h comes in two parts (its rounded value and the rest), each a B operand of
// its own beside the same x: an MMA costs more when its x changes, so the two
// follow each other (alternating between the halves of x instead: 81 us for 77,
// 4096-row training of rank 32; one MMA of both parts' columns is no faster).
//
// Measured: 8192 rows, 5120 and 1536 columns, ranks 64 and 128: 31 us after the
// kernel before for 109 MB, then 9 us to join 40 MB of partials.  300 rows, 4096
// and 1408 columns, rank 8: 6 and 2 us.
#include "lora_common.cuh"

namespace exl3 {
namespace lora {

namespace {

constexpr int kThreads = 448;       // 8 loader warps in two groups, 4 epilogue, MMA, fence warp
constexpr int kBlock = 64 * 128;                 // 64 rows of 64 columns
constexpr int kXBytes = kOuterN / 64 * kBlock;
constexpr int kHalfCols = 128;                   // TMEM columns of one 128-column half
constexpr int kRingBytes = 208 * 1024;
constexpr int kMaxSlots = 6;
constexpr int kJoinThreads = 256;
constexpr int kJoinParts = 4;       // blocks per boundary that cuts an item
constexpr int kZeroBlocks = 64;     // join kernel: blocks that zero unused adapters' gradients

// a stage: 64 rows of x, of h and of h's remainders
EXL3_HD inline int part_bytes(int h_cols) { return (h_cols + 63) / 64 * kBlock; }
EXL3_HD inline int stage_bytes(int h_cols) { return kXBytes + 2 * part_bytes(h_cols); }
EXL3_HD inline int ring_slots(int h_cols)
{
    const int n = kRingBytes / stage_bytes(h_cols);
    return n < kMaxSlots ? n : kMaxSlots;
}

// TMEM: two accumulators of two halves, one filled while the other is drained.
// f16 sums the rests of h apart (split2), in the columns that ranks up to 64
// leave free; above, in the other accumulator's, so that there is only one (f16,
// 8192 rows, training, against bf16 or the rests in the same columns: ranks 64 and
// 128, 141 us and 140; 40 adapters of rank 100, whose items have four stages, 172
// and 153).
EXL3_HD inline int tbufs(int h_cols, int dtype) { return dtype == EXL3_F16 && h_cols > 64 ? 1 : 2; }
EXL3_HD inline int rest_cols(int h_cols, int dtype) { return dtype != EXL3_F16 ? 0 : h_cols <= 64 ? 64 : 2 * kHalfCols; }

struct Ctl {
    uint64_t full[kMaxSlots], ready[kMaxSlots], empty[kMaxSlots], tfull[2], tempty[2], drain;
    uint32_t tmem;
    int abort;
};

// Items of one adapter: 256 columns, the last one 128 where the width is an
// odd multiple of 128.
EXL3_HD inline int blocks(int width) { return (width + kOuterN - 1) / kOuterN; }

// Where a stage index lies: product p, adapter e, column block n, and the
// item's stages [first, first + len).
struct Item {
    int p, e, n, first, len;
};

// The adapter whose steps hold step q: the last e with steps[e] <= q.  One
// warp: 32 probes 32 apart, then 32 in a row (N <= 1024).
EXL3_DEV int find_adapter(const int32_t *steps, int N, int q)
{
    const int lane = threadIdx.x & 31;
    const int far = lane * 32;
    const unsigned m = __ballot_sync(0xffffffffu, far < N && steps[far] <= q);
    const int base = (31 - __clz(m)) * 32, near = base + lane;
    const unsigned k = __ballot_sync(0xffffffffu, near < N && steps[near] <= q);
    return base + 31 - __clz(k);
}

EXL3_DEV Item locate(const LoraOuterArgs &a, const int32_t *steps, int s)
{
    Item it;
    const int all = steps[a.N], n0 = blocks(a.p[0].width);
    it.p = s >= n0 * all;
    const int base = it.p ? n0 * all : 0, nb = blocks(a.p[it.p].width);
    it.e = find_adapter(steps, a.N, (s - base) / nb);
    it.len = steps[it.e + 1] - steps[it.e];
    const int in = s - base - steps[it.e] * nb;
    it.n = in / it.len;
    it.first = s - in % it.len;
    return it;
}

// The item after it.
EXL3_DEV void next_item(const LoraOuterArgs &a, const int32_t *steps, Item &it)
{
    it.first += it.len;
    if (++it.n < blocks(a.p[it.p].width))
        return;
    it.n = 0;
    do {
        if (++it.e == a.N) {
            it.e = 0;
            it.p++;
        }
        it.len = steps[it.e + 1] - steps[it.e];
    } while (it.len == 0 && it.p < 2);
}

EXL3_DEV int total_stages(const LoraOuterArgs &a, const int32_t *steps)
{
    return steps[a.N] * (blocks(a.p[0].width) + blocks(a.p[1].width));
}

// Zero gradients for the adapters without rows, dealt to `of` CTAs of the join.
EXL3_DEV void zero_unused(const LoraOuterArgs &a, const int32_t *steps, int worker, int of)
{
    for (int e = worker; e < a.N; e += of) {
        if (steps[e] != steps[e + 1] || a.rank[e] == 0)
            continue;
        for (int p = 0; p < 2; p++) {
            uint4 *out = reinterpret_cast<uint4 *>(a.p[p].G[e]);
            for (size_t i = threadIdx.x; i < (size_t)a.rank[e] * a.p[p].width / 8; i += kJoinThreads)
                out[i] = make_uint4(0, 0, 0, 0);
        }
    }
}

__global__ void __launch_bounds__(kThreads, 1) k_lora_outer(LoraOuterArgs a)
{
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ Ctl c;
    __shared__ Item start;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    grid_dep_launch();
    // (a CTA that has nothing to do waits too: the join takes this kernel's end
    // for the end of the kernels before)
    if (!plan_ok(a.plan, a.M, a.N)) {
        grid_dep_wait();
        return;
    }
    const LoraPlanLayout L = lora_plan_layout(a.M, a.N);
    const int32_t *perm = a.plan + L.perm / 4, *steps = a.plan + L.steps / 4, *offs = a.plan + L.offsets / 4;
    const int least = lora_outer_min(steps[a.N], a.plan[kLpUsed]);
    const int total = total_stages(a, steps), per = lora_share(total, gridDim.x, least);
    const int begin = min(total, (int)blockIdx.x * per), end = min(total, begin + per);
    if (begin >= end) {
        grid_dep_wait();
        return;
    }
    const int sbytes = stage_bytes(a.h_cols), nslots = ring_slots(a.h_cols);
    volatile int *abort = &c.abort;
    if (warp == 0) {
        const Item it = locate(a, steps, begin);
        if (lane == 0)
            start = it;
    }
    if (tid == 32) {
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
        tmem_alloc(&c.tmem, 4 * kHalfCols);
    fence_before();
    __syncthreads();
    fence_after();

    Item it = start;
    // (a bad table entry is in the error word, which only the epilogue reads)
    auto padded_rank = [&](int e) { return min(a.h_cols, max(16, (a.rank[e] + 15) / 16 * 16)); };
    if (warp < 8) {
        // group 0 takes the even stages of the share, group 1 the odd ones
        const int group = warp >> 2, gt = tid & 127;
        const int ch = gt & 31, r0 = gt >> 5;       // a warp per 512-byte row of x
        Ring put;
        put.slot = group;
        int row[16], slot0 = 0, rows = 0;            // rows of the current stage (-1: past the end)
        int hq = 0, hr = 0, hrows = 64, hn = 1;     // h: this thread's chunk, row, row step, passes
        bool hin = true, xin = true;                 // xin: this thread's chunk is in the item
        const uint8_t *x = nullptr, *h = nullptr;
        size_t pitch = 0;
        auto load_rows = [&](int k) {
#pragma unroll
            for (int i = 0; i < 16; i++) {
                const int r = k * kOuterK + r0 + 4 * i;
                row[i] = r < rows && xin ? perm[slot0 + r] : -1;
            }
        };
        int e_known = -1;
        auto enter = [&](int k) {
            if (it.e != e_known) {
                e_known = it.e;
                slot0 = offs[it.e];
                rows = offs[it.e + 1] - slot0;
            }
            x = static_cast<const uint8_t *>(a.p[it.p].x) + (size_t)it.n * (2 * kOuterN) + ch * 16;
            xin = it.n * kOuterN + ch * 8 < a.p[it.p].width;
            h = static_cast<const uint8_t *>(a.p[it.p].h);
            pitch = (size_t)a.p[it.p].width * 2;
            // a row of h is rp / 8 chunks, dealt to a power of two of lanes
            const int hc = padded_rank(it.e) / 8, lanes = hc <= 2 ? 2 : hc <= 4 ? 4 : hc <= 8 ? 8 : 16;
            hq = gt & (lanes - 1);
            hin = hq < hc;
            hrows = 128 / lanes;
            hr = gt / lanes;
            hn = lanes / 2;
            h += ((size_t)(slot0 + hr) * lora_h_pitch(a.h_cols) + hq * 8) * 2;
            load_rows(k);
        };
        int k = begin - it.first + group;
        auto settle = [&]() {                       // k past the item's end: into the next ones
            bool moved = false;
            while (k >= it.len) {
                k -= it.len;
                next_item(a, steps, it);
                moved = true;
            }
            return moved;
        };
        if (begin + group < end) {
            settle();
            enter(k);
        }
        grid_dep_wait();            // h (dh) comes from the kernels before
        for (int s = begin + group; s < end; s += 2) {
            if (!wait_bar(&c.empty[put.slot], put.phase ^ 1, abort, a.hdr))
                break;
            const uint32_t dst = smem_addr(smem + (size_t)put.slot * sbytes);
#pragma unroll
            for (int i = 0; i < 16; i++)
                cp_async16(dst + (ch >> 3) * kBlock + swz(r0 + 4 * i, ch & 7),
                           row[i] < 0 ? static_cast<const uint8_t *>(a.p[0].x) : x + (size_t)row[i] * pitch, row[i] >= 0);
            const size_t h_pitch = (size_t)lora_h_pitch(a.h_cols) * 2;
            const uint8_t *hk = h + k * kOuterK * h_pitch;
            if (hin)
                for (int i = 0; i < hn; i++) {
                    const int r = hr + i * hrows;
                    const bool v = k * kOuterK + r < rows;
                    const uint32_t to = dst + kXBytes + (hq >> 3) * kBlock + swz(r, hq & 7);
                    const uint8_t *from = v ? hk + i * hrows * h_pitch : static_cast<const uint8_t *>(a.p[0].x);
                    cp_async16(to, from, v);
                    cp_async16(to + part_bytes(a.h_cols), from + (v ? a.h_cols * 2 : 0), v);
                }
            cp_async_arrive(&c.full[put.slot]);
            put.next2(nslots);
            if (s + 2 < end) {
                k += 2;
                if (settle())
                    enter(k);
                else
                    load_rows(k);
            }
        }
        cp_async_wait_all();
    } else if (warp < 12) {
        const int q = warp & 3, col = 32 * q + lane;
        Ring t;
        grid_dep_wait();            // and so does the error word
        const bool bad = a.hdr[kHdrError] != 0;
        const int nbufs = tbufs(a.h_cols, a.act_dtype), rests = rest_cols(a.h_cols, a.act_dtype);
        for (int s = begin; s < end;) {
            const int stop = min(end, it.first + it.len);
            const bool whole = it.first >= begin && it.first + it.len <= end;
            const int rank = bad ? 0 : a.rank[it.e], width = a.p[it.p].width;
            const float alpha = a.p[it.p].scaled ? a.scale[it.e] : 1.0f;
            uint16_t *out = rank > 0 ? reinterpret_cast<uint16_t *>(a.p[it.p].G[it.e]) + it.n * kOuterN + col : nullptr;
            float *part = a.part + (2 * (size_t)blockIdx.x + (s > begin)) * kOuterN * a.h_cols + col;
            if (!warp_wait_bar(&c.tfull[t.slot], t.phase, abort, a.hdr))
                break;
            fence_after();
            const int halves = min(2, (width - it.n * kOuterN) / 128);
            for (int half = 0; half < halves; half++) {
                const uint32_t addr = c.tmem + ((uint32_t)(32 * q) << 16) + (2 * t.slot + half) * kHalfCols;
                for (int j = 0; j < rank; j += 16) {
                    uint32_t v[16];
                    tmem_ld16_issue(addr + j, v);
                    tmem_ld16_wait(v);
                    if (rests) {
                        uint32_t w[16];
                        tmem_ld16_issue(addr + rests + j, w);
                        tmem_ld16_wait(w);
#pragma unroll
                        for (int i = 0; i < 16; i++)
                            v[i] = __float_as_uint(fmaf(__uint_as_float(w[i]), 1.0f / (1 << kRestBits), __uint_as_float(v[i])));
                    }
                    if (whole) {
                        uint16_t *o = out + (size_t)j * width + half * 128;
#pragma unroll
                        for (int i = 0; i < 16; i += 2, o += 2 * width) {
                            const uint32_t u = pack2(alpha * __uint_as_float(v[i]), alpha * __uint_as_float(v[i + 1]),
                                                     a.act_dtype);
                            if (j + i < rank)
                                o[0] = (uint16_t)u;
                            if (j + i + 1 < rank)
                                o[width] = (uint16_t)(u >> 16);
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 16; i++)
                            part[(j + i) * kOuterN + half * 128] = __uint_as_float(v[i]);
                    }
                }
            }
            fence_before();
            mbar_arrive(&c.tempty[t.slot]);
            t.next(nbufs);
            s = stop;
            if (s < end)
                next_item(a, steps, it);
        }
    } else if (warp == 12 && lane == 0) {
        Ring get, t;
        bool ok = true;
        const int nbufs = tbufs(a.h_cols, a.act_dtype), rests = rest_cols(a.h_cols, a.act_dtype);
        for (int s = begin; s < end && ok;) {
            const int stop = min(end, it.first + it.len);
            const uint32_t id = idesc(padded_rank(it.e), a.act_dtype, 1, 1);
            if (!(ok = wait_bar(&c.tempty[t.slot], t.phase ^ 1, abort, a.hdr)))
                break;
            fence_after();
            const int halves = min(2, (a.p[it.p].width - it.n * kOuterN) / 128);
            bool first = true;
            for (; s < stop; s++) {
                if (!(ok = wait_bar(&c.ready[get.slot], get.phase, abort, a.hdr)))
                    break;
                fence_after();
                const uint32_t xs = smem_addr(smem + (size_t)get.slot * sbytes);
                for (int half = 0; half < halves; half++)
#pragma unroll
                    for (int i = 0; i < 4; i++)
#pragma unroll
                        for (int part = 0; part < 2; part++)
                            mma_f16(c.tmem + (2 * t.slot + half) * kHalfCols + part * rests,
                                    desc_mn_major(xs + half * 2 * kBlock + 2048 * i, kBlock),
                                    desc_mn_major(xs + kXBytes + part * part_bytes(a.h_cols) + 2048 * i, kBlock), id,
                                    !(first && i == 0 && (part == 0 || rests)));
                first = false;
                mma_commit(&c.empty[get.slot]);
                get.next(nslots);
            }
            mma_commit(&c.tfull[t.slot]);
            t.next(nbufs);
            if (s < end)
                next_item(a, steps, it);
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
        tmem_free(c.tmem, 4 * kHalfCols);
}

// Blocks 4c .. 4c + 3, c < ctas, work on the item that the boundary between
// shares c and c + 1 cuts, if it cuts one: an item has four blocks for each
// boundary in it, so that one with many partials is spread out too (7518 rows
// of one adapter of rank 68, 17 partials an item: 10 us; with eight blocks an
// item, whatever its partials, 15).  The other blocks zero the gradients of
// adapters without rows.
__global__ void __launch_bounds__(kJoinThreads) k_lora_outer_join(LoraOuterArgs a)
{
    grid_dep_launch();
    // (a CTA that has nothing to do waits too: the kernel after this one takes
    // its end for the end of the kernels before)
    if (!plan_ok(a.plan, a.M, a.N)) {
        grid_dep_wait();
        return;
    }
    const LoraPlanLayout L = lora_plan_layout(a.M, a.N);
    const int32_t *steps = a.plan + L.steps / 4;
    const int share = blockIdx.x / kJoinParts;
    if (share >= a.ctas) {
        grid_dep_wait();
        if (a.hdr[kHdrError])
            return;
        zero_unused(a, steps, blockIdx.x - a.ctas * kJoinParts, kZeroBlocks);
        return;
    }
    const int least = lora_outer_min(steps[a.N], a.plan[kLpUsed]);
    const int total = total_stages(a, steps), per = lora_share(total, a.ctas, least);
    const int cut = (share + 1) * per;
    if (cut >= total) {
        grid_dep_wait();
        return;
    }
    const Item it = locate(a, steps, cut);
    const int c0 = it.first / per, c1 = (it.first + it.len - 1) / per;
    if (it.first == cut) {
        grid_dep_wait();
        return;
    }
    const int rank = a.rank[it.e], width = a.p[it.p].width;
    const float alpha = a.p[it.p].scaled ? a.scale[it.e] : 1.0f;
    const size_t slot = kOuterN * (size_t)a.h_cols;
    const int quads = min(kOuterN, width - it.n * kOuterN) / 4;    // 64 or 32 a row
    grid_dep_wait();
    if (a.hdr[kHdrError])
        return;
    uint8_t *out = reinterpret_cast<uint8_t *>(a.p[it.p].G[it.e]);
    // four columns a thread
    constexpr int kU = 4, kC = 2;                  // kU * kC loads in flight
    const int step = (c1 - c0) * kJoinParts * kJoinThreads;
    for (int i0 = (blockIdx.x - c0 * kJoinParts) * kJoinThreads + threadIdx.x; i0 < rank * quads; i0 += kU * step) {
        float4 v[kU] = {};
        for (int c = c0; c <= c1; c += kC) {
            float4 f[kC][kU];
#pragma unroll
            for (int d = 0; d < kC; d++) {
                const float *p = a.part + (2 * (size_t)(c + d) + (max(it.first, (c + d) * per) > (c + d) * per)) * slot;
#pragma unroll
                for (int u = 0; u < kU; u++) {
                    const int i = i0 + u * step;
                    f[d][u] = c + d <= c1 && i < rank * quads
                                  ? *reinterpret_cast<const float4 *>(p + i / quads * kOuterN + i % quads * 4)
                                  : make_float4(0.f, 0.f, 0.f, 0.f);
                }
            }
#pragma unroll
            for (int d = 0; d < kC; d++)
#pragma unroll
                for (int u = 0; u < kU; u++) {
                    v[u].x += f[d][u].x; v[u].y += f[d][u].y; v[u].z += f[d][u].z; v[u].w += f[d][u].w;
                }
        }
#pragma unroll
        for (int u = 0; u < kU; u++) {
            const int i = i0 + u * step;
            if (i < rank * quads)
                *reinterpret_cast<uint2 *>(out + ((size_t)(i / quads) * width + it.n * kOuterN + i % quads * 4) * 2) =
                    make_uint2(pack2(alpha * v[u].x, alpha * v[u].y, a.act_dtype),
                               pack2(alpha * v[u].z, alpha * v[u].w, a.act_dtype));
        }
    }
}

}  // namespace

}  // namespace lora

cudaError_t lora_outer_set_attributes()
{
    return cudaFuncSetAttribute(lora::k_lora_outer, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                lora::kRingBytes);
}

cudaError_t launch_lora_outer(const LoraOuterArgs &a, cudaStream_t s)
{
    if (a.M > 0) {
        const cudaError_t e =
            launch_dependent(lora::k_lora_outer, a.ctas, lora::kThreads,
                             lora::ring_slots(a.h_cols) * lora::stage_bytes(a.h_cols), s, a);
        if (e != cudaSuccess)
            return e;
    }
    return launch_dependent(lora::k_lora_outer_join, a.ctas * lora::kJoinParts + lora::kZeroBlocks,
                            lora::kJoinThreads, 0, s, a);
}

cudaError_t lora_set_attributes()
{
    cudaError_t e = lora_plan_set_attributes();
    if (e == cudaSuccess)
        e = lora_shrink_set_attributes();
    if (e == cudaSuccess)
        e = lora_expand_set_attributes();
    return e == cudaSuccess ? lora_outer_set_attributes() : e;
}

}  // namespace exl3
