// Groups a batch's rows by adapter, in row order inside each group (a stable
// counting sort), and cuts the groups into tiles (include/exl3.h, "adapters").
//
// One CTA.  Each warp owns a contiguous chunk of rows: a histogram per warp,
// an exclusive scan of the group sizes and, inside a group, of the warps'
// counts, then every warp writes its chunk's rows at its own cursors.  Equal
// ids inside a 32-row step are ranked by __match_any_sync.  Once per batch,
// not per projection, so its latency is shared by every adapted projection.
//
// Bound by latencies: each warp reads its ids twice, one 32-row step after the
// other.  Graph replay, int32 ids, one adapter / 40 / 1024: 1 row 10 / 11 / 12 us, 64
// rows 11 / 15 / 13, 1000 rows 11 / 17 / 19, 16384 rows 19 / 41 / 55, 65536 rows 48 /
// 118 / 159.
#include "common.cuh"
#include "lora.h"

namespace exl3 {

namespace {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / 32;

// Exclusive block scan of one value per thread; `total` gets the block sum.
EXL3_DEV int scan_exclusive(int v, int *sums, int *total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, d);
        x += lane >= d ? y : 0;
    }
    if (lane == 31)
        sums[warp] = x;
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll 8
    for (int w = 0; w < kWarps; w++) {
        before += w < warp ? sums[w] : 0;
        all += sums[w];
    }
    __syncthreads();
    *total = all;
    return before + x - v;
}

// Writes one group's tiles of `size` rows, one per lane.
EXL3_DEV void write_tiles(int4 *tiles, int first, int adapter, int start, int rows, int size)
{
    const int n = (rows + size - 1) / size;
    for (int i = threadIdx.x & 31; i < n; i += 32)
        tiles[first + i] = make_int4(adapter, start + i * size, min(size, rows - i * size), 0);
}

template <typename IdT>
__global__ void __launch_bounds__(kThreads) k_lora_plan(LoraPlanArgs a)
{
    extern __shared__ int hist[];                  // [kWarps][N + 1]
    __shared__ int sums[kWarps], bad_s;
    const int N = a.N, G = N + 1, M = a.M;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const LoraPlanLayout L = lora_plan_layout(M, N);
    uint8_t *base = reinterpret_cast<uint8_t *>(a.plan);
    int32_t *offsets = reinterpret_cast<int32_t *>(base + L.offsets);
    int32_t *perm = reinterpret_cast<int32_t *>(base + L.perm);
    int4 *tiles = reinterpret_cast<int4 *>(base + L.tiles);
    int4 *small = reinterpret_cast<int4 *>(base + L.small);
    const IdT *ids = static_cast<const IdT *>(a.ids);

    for (int i = tid; i < kWarps * G; i += kThreads)
        hist[i] = 0;
    if (tid == 0)
        bad_s = 0;
    __syncthreads();

    const int steps = (M + kThreads - 1) / kThreads;      // 32-row steps per warp
    const int r0 = warp * steps * 32;
    int *mine = hist + warp * G;
    auto group = [&](int r) {
        const long long id = static_cast<long long>(ids[r]);
        if (id < -1 || id >= N)
            bad_s = 1;
        return id < 0 || id >= N ? N : (int)id;
    };
    for (int i = 0; i < steps; i++) {
        const int r = r0 + i * 32 + lane;
        const int g = r < M ? group(r) : -1;
        const unsigned same = __match_any_sync(0xffffffffu, g);
        if (g >= 0 && lane == __ffs(same) - 1)
            mine[g] += __popc(same);
        __syncwarp();
    }
    __syncthreads();

    // group g = tid: its size; the warps' counts become offsets inside it
    int rows = 0;
    if (tid < N)
#pragma unroll 8
        for (int w = 0; w < kWarps; w++) {
            const int c = hist[w * G + tid];
            hist[w * G + tid] = rows;
            rows += c;
        }
    int total, ntiles, nsmall;
    const int start = scan_exclusive(rows, sums, &total);
    const int t0 = scan_exclusive((rows + kLoraTile - 1) / kLoraTile, sums, &ntiles);
    const int s0 = scan_exclusive((rows + kLoraSmallTile - 1) / kLoraSmallTile, sums, &nsmall);
    int nsteps;
    const int k0 = scan_exclusive((rows + kOuterK - 1) / kOuterK, sums, &nsteps);
    int32_t *step_off = reinterpret_cast<int32_t *>(base + L.steps);
    if (tid < N)
        step_off[tid] = k0;
    if (tid == 0)
        step_off[N] = nsteps;
    if (tid < N) {
        offsets[tid] = start;
        for (int w = 0; w < kWarps; w++)
            hist[w * G + tid] += start;
    }
    if (tid == 0) {                                 // rows without an adapter come last
        int c = total;
        for (int w = 0; w < kWarps; w++) {
            const int n = hist[w * G + N];
            hist[w * G + N] = c;
            c += n;
        }
        offsets[N] = total;
        offsets[N + 1] = M;
    }
    const int used = __syncthreads_count(tid < N && rows > 0);
    for (int i = 0; i < steps; i++) {
        const int r = r0 + i * 32 + lane;
        const int g = r < M ? group(r) : -1;
        const unsigned same = __match_any_sync(0xffffffffu, g);
        const int cur = g >= 0 ? mine[g] : 0;
        __syncwarp();
        if (g >= 0) {
            perm[cur + __popc(same & ((1u << lane) - 1))] = r;
            if (lane == __ffs(same) - 1)
                mine[g] = cur + __popc(same);
        }
        __syncwarp();
    }
    // tiles: warp w writes the groups of its 32 threads one after the other
    for (int i = 0; i < 32; i++) {
        const int g = warp * 32 + i;
        const int n = __shfl_sync(0xffffffffu, rows, i), st = __shfl_sync(0xffffffffu, start, i);
        const int tt = __shfl_sync(0xffffffffu, t0, i), ss = __shfl_sync(0xffffffffu, s0, i);
        if (g < N && n > 0) {
            write_tiles(tiles, tt, g, st, n, kLoraTile);
            write_tiles(small, ss, g, st, n, kLoraSmallTile);
        }
    }
    const int idle = M - total;
    if (warp == 0) {
        write_tiles(tiles, ntiles, -1, total, idle, kLoraTile);
        write_tiles(small, nsmall, -1, total, idle, kLoraSmallTile);
    }
    if (tid == 0) {
        a.plan[kLpError] = bad_s ? EXL3_DERR_ROUTE_ID : 0;
        a.plan[kLpMagic] = kLoraMagic;
        a.plan[kLpM] = M;
        a.plan[kLpN] = N;
        a.plan[kLpActive] = ntiles;
        a.plan[kLpUsed] = used;
        a.plan[kLpSmallActive] = nsmall;
        a.plan[kLpTiles] = ntiles + (idle + kLoraTile - 1) / kLoraTile;
        a.plan[kLpSmallTiles] = nsmall + (idle + kLoraSmallTile - 1) / kLoraSmallTile;
    }
}

constexpr int kMaxSmem = kWarps * (EXL3_MAX_ADAPTERS + 1) * 4;

}  // namespace

cudaError_t lora_plan_set_attributes()
{
    cudaError_t e = cudaFuncSetAttribute(k_lora_plan<int32_t>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         kMaxSmem);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(k_lora_plan<int64_t>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
    return e;
}

cudaError_t launch_lora_plan(const LoraPlanArgs &a, int ids_dtype, cudaStream_t s)
{
    const size_t smem = (size_t)kWarps * (a.N + 1) * 4;
    if (ids_dtype == EXL3_I64)
        k_lora_plan<int64_t><<<1, kThreads, smem, s>>>(a);
    else
        k_lora_plan<int32_t><<<1, kThreads, smem, s>>>(a);
    return cudaGetLastError();
}

}  // namespace exl3
