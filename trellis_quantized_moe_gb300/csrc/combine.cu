// Rows of tokens to expert order and back (include/exl3.h, "dispatch and
// combine"):
//   k_dispatch          xp[slot(t, j)] = x[t]
//   k_combine           out[t] = base[t] + sum_j rw[t, j] y[slot(t, j)]
//   k_combine_backward  dy[slot(t, j)] = rw[t, j] d_out[t], d_rw[t, j] = <d_out[t], y[slot(t, j)]>
// All go through the batch in token order: a token's row is read or written once
// and the rows in expert order, each a contiguous piece of memory, once.  Bound by
// HBM.  Grids are as large as the work, not persistent: new CTAs' loads and old
// ones' stores then mix in longer runs (16384 x 8 rows of 5120 bf16, dispatch: 231
// -> 221 us).
#include "dispatch.h"
#include "rows.cuh"

namespace exl3 {

namespace {

// With 64 / 128 / 256 threads 8192 x 8 rows of 5120 bf16 combine in 128 / 128 / 137 us;
// of other widths, 105M elements in expert order (up to 16384 tokens): 264 wide 20 / 21 / 27, 1032
// wide 48 / 48 / 50, 1536 wide 40 / 42 / 44, 4096 wide 40 / 40 / 43 us, dispatch 640
// wide 35 / 31 / 31.  Rows below 1024 elements leave threads idle (128 wide: 2 TB/s).
constexpr int kThreads = 128;
// Rows of a token in flight (the same, 2 / 3 / 4 / 5 / 8: 146 / 143 / 128 / 136 / 139 us; one
// token 2.6 / 2.4 / 2.1 / 2.2 / 2.0; 2 / 4 / 8 of 1536 wide rows 49 / 42 / 45 us, of 4096
// 46 / 40 / 42).
constexpr int kBatch = 4;
constexpr int kRouteWarps = 4;          // routes of a backward CTA
// Pieces of a route's two rows in flight, for each lane (the backward of the same,
// 1 / 2 / 4 / 5: 228 / 209 / 208 / 208 us; one token 5.7 / 4.4 / 4.3 / 3.5; 2 / 4 / 5 /
// 8 of other widths as above: 640 wide 79 / 74 / 79 / 111, 1536 wide 74 / 73 / 75 / 83,
// 4096 wide 72 / 69 / 70 / 69 us).
constexpr int kAhead = 5;

// Slot of a route, -1 where it has none (or the table says what no plan says).
EXL3_DEV int slot_of(const RowsArgs &a, int f)
{
    const int s = a.slots[f];
    return s >= 0 && s < a.M * a.topk ? s : -1;
}

// A CTA takes kThreads pieces of one token.
struct Unit {
    int t, p;
    EXL3_DEV explicit Unit(int pieces)
    {
        const int cuts = (pieces + kThreads - 1) / kThreads;
        t = blockIdx.x / cuts;
        p = (blockIdx.x - t * cuts) * kThreads + threadIdx.x;
    }
};

__global__ void __launch_bounds__(kThreads) k_dispatch(RowsArgs a, int pieces)
{
    grid_dep_wait();
    grid_dep_launch();
    const Unit u(pieces);
    if (u.p >= pieces)
        return;
    const uint4 v = static_cast<const uint4 *>(a.x)[(size_t)u.t * pieces + u.p];
    for (int j = 0; j < a.topk; j++) {
        const int s = slot_of(a, u.t * a.topk + j);
        if (s >= 0)
            static_cast<uint4 *>(a.rows)[(size_t)s * pieces + u.p] = v;
    }
}

template <int DT>
__global__ void __launch_bounds__(kThreads) k_combine(RowsArgs a, int pieces)
{
    constexpr int N = kPiece<DT>;
    grid_dep_wait();
    grid_dep_launch();
    const Unit u(pieces);
    if (u.p >= pieces)
        return;
    const uint4 *y = static_cast<const uint4 *>(a.y) + u.p;
    float acc[N] = {};
    uint4 first = make_uint4(0, 0, 0, 0);
    if (a.x)
        first = static_cast<const uint4 *>(a.x)[(size_t)u.t * pieces + u.p];
    for (int j = 0; j < a.topk; j += kBatch) {
        int s[kBatch];
        float w[kBatch];
        uint4 v[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; i++) {
            const int f = u.t * a.topk + j + i;
            s[i] = j + i < a.topk ? slot_of(a, f) : -1;
            w[i] = a.rw && j + i < a.topk ? load_act(a.rw, f, a.rw_dtype) : 1.0f;
        }
#pragma unroll
        for (int i = 0; i < kBatch; i++)
            if (s[i] >= 0)
                v[i] = y[(size_t)s[i] * pieces];
        if (j == 0)
            unpack<DT>(first, acc);
#pragma unroll
        for (int i = 0; i < kBatch; i++)
            if (s[i] >= 0) {
                float x[N];
                unpack<DT>(v[i], x);
#pragma unroll
                for (int n = 0; n < N; n++)
                    acc[n] = fmaf(w[i], x[n], acc[n]);
            }
    }
    static_cast<uint4 *>(a.out)[(size_t)u.t * pieces + u.p] = pack<DT>(acc);
}

// A warp takes a route; the lanes' sums of d_rw join in a fixed tree.
template <int DT>
__global__ void __launch_bounds__(kRouteWarps * 32) k_combine_backward(RowsArgs a, int pieces)
{
    constexpr int N = kPiece<DT>;
    grid_dep_wait();
    grid_dep_launch();
    const int lane = threadIdx.x & 31, f = blockIdx.x * kRouteWarps + (threadIdx.x >> 5);
    if (f >= a.M * a.topk)
        return;
    const int s = slot_of(a, f);
    float dot = 0.0f;
    if (s >= 0) {
        const float w = a.rows ? load_act(a.rw, f, a.rw_dtype) : 0.0f;
        const uint4 *d = static_cast<const uint4 *>(a.x) + (size_t)(f / a.topk) * pieces;
        const uint4 *y = a.out ? static_cast<const uint4 *>(a.y) + (size_t)s * pieces : nullptr;
        uint4 *dy = a.rows ? static_cast<uint4 *>(a.rows) + (size_t)s * pieces : nullptr;
        for (int p0 = lane; p0 < pieces; p0 += 32 * kAhead) {
            uint4 dr[kAhead], yr[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; i++) {
                const int p = p0 + i * 32;
                if (p < pieces) {
                    dr[i] = d[p];
                    if (y)
                        yr[i] = y[p];
                }
            }
#pragma unroll
            for (int i = 0; i < kAhead; i++) {
                const int p = p0 + i * 32;
                if (p >= pieces)
                    break;
                float g[N], v[N];
                unpack<DT>(dr[i], g);
                if (y) {
                    unpack<DT>(yr[i], v);
#pragma unroll
                    for (int n = 0; n < N; n++)
                        dot = fmaf(g[n], v[n], dot);
                }
                if (dy) {
#pragma unroll
                    for (int n = 0; n < N; n++)
                        g[n] *= w;
                    dy[p] = pack<DT>(g);
                }
            }
        }
#pragma unroll
        for (int m = 16; m > 0; m >>= 1)
            dot += __shfl_xor_sync(0xffffffffu, dot, m);
    }
    if (a.out && lane == 0)
        store_float(a.out, f, a.rw_dtype, dot);
}

int pieces_of(const RowsArgs &a) { return a.width / (a.dtype == EXL3_F32 ? 4 : 8); }

// M * width < 2^38 keeps the grid below 2^31.
int units_of(const RowsArgs &a)
{
    return a.M * ((pieces_of(a) + kThreads - 1) / kThreads);
}

}  // namespace

cudaError_t launch_dispatch(const RowsArgs &a, cudaStream_t s)
{
    return launch_dependent(k_dispatch, units_of(a), kThreads, 0, s, a, pieces_of(a));
}

cudaError_t launch_combine(const RowsArgs &a, cudaStream_t s)
{
    const auto kernel = a.dtype == EXL3_F32    ? k_combine<EXL3_F32>
                        : a.dtype == EXL3_BF16 ? k_combine<EXL3_BF16>
                                               : k_combine<EXL3_F16>;
    return launch_dependent(kernel, units_of(a), kThreads, 0, s, a, pieces_of(a));
}

cudaError_t launch_combine_backward(const RowsArgs &a, cudaStream_t s)
{
    const auto kernel = a.dtype == EXL3_F32    ? k_combine_backward<EXL3_F32>
                        : a.dtype == EXL3_BF16 ? k_combine_backward<EXL3_BF16>
                                               : k_combine_backward<EXL3_F16>;
    return launch_dependent(kernel, (a.M * a.topk + kRouteWarps - 1) / kRouteWarps, kRouteWarps * 32, 0, s, a,
                            pieces_of(a));
}

}  // namespace exl3
