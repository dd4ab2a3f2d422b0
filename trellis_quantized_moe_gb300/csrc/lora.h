// Adapter plan, workspace layout, kernel arguments and launchers (internal).
#pragma once
#include <cuda_runtime_api.h>
#include <stdint.h>

#include "../../include/exl3.h"
#include "plan.h"

namespace exl3 {

constexpr int kLoraMagic = 0x4c6f5241;
constexpr int kLoraTile = 128;      // rows of a prompt tile
constexpr int kLoraSmallTile = 16;  // rows of a decode tile

enum LoraPlanWord {
    kLpError = 0,      // sticky device error word
    kLpMagic = 1,
    kLpM = 2,
    kLpN = 3,
    kLpTiles = 4,      // prompt tiles (adapter tiles first, idle rows' tiles last)
    kLpSmallTiles = 5,
    kLpActive = 6,     // prompt tiles of adapters
    kLpSmallActive = 7,
    kLpWords = 64
};

// Rows grouped by adapter: slot s holds row perm[s]; adapter a's slots are
// offsets[a] .. offsets[a+1], those without an adapter offsets[N] .. M.  A
// tile is (adapter or -1, first slot, rows, 0).
struct LoraPlanLayout {
    size_t offsets, perm, tiles, small, total;
};

EXL3_HD inline LoraPlanLayout lora_plan_layout(int M, int N)
{
    LoraPlanLayout L{};
    size_t o = kLpWords * 4;
    L.offsets = o; o = align_up(o + (size_t)(N + 2) * 4, 256);
    L.perm = o;    o = align_up(o + (size_t)M * 4, 256);
    L.tiles = o;   o = align_up(o + ((size_t)M / kLoraTile + N + 1) * 16, 256);
    L.small = o;   o = align_up(o + ((size_t)M / kLoraSmallTile + N + 1) * 16, 256);
    L.total = o;
    return L;
}

EXL3_HD inline int lora_h_cols(int max_rank) { return (max_rank + 15) / 16 * 16; }

struct LoraWsLayout {
    size_t hdr, h, total;
};

EXL3_HD inline LoraWsLayout lora_ws_layout(int M, int N, int in_f, int out_f, int max_rank)
{
    (void)N; (void)in_f; (void)out_f;
    LoraWsLayout L{};
    size_t o = 0;
    L.hdr = o; o = align_up(o + kHdrWords * 4, 256);
    L.h = o;   o = align_up(o + (size_t)M * lora_h_cols(max_rank) * 2, 256);
    L.total = o;
    return L;
}

struct LoraPlanArgs {
    const void *ids;
    int M, N;
    int32_t *plan;
};

// One of the three products, over the rows in plan order:
//   shrink h[s][j] = alpha_a * sum_i x[perm[s]][i] W_a[j][i]
//   expand y[perm[s]][n] = base[perm[s]][n] + alpha_a * sum_j h[s][j] W_a[j][n]
//   outer  G_a[j][n] = alpha_a * sum_s h[s][j] x[perm[s]][n]
// alpha_a is the adapter's scale where `scaled`, else 1.
struct LoraArgs {
    const int32_t *plan;
    int M, N, act_dtype, max_rank, h_cols, width, scaled, num_sms;
    const int64_t *W;
    const int32_t *rank;
    const float *scale;
    const int64_t *G;
    const void *x;
    void *h;
    const void *base;
    void *y;
    int32_t *hdr;
};

// Table entries of the adapters that have rows (all: of every adapter, and
// the gradient tables): the call's error word into hdr.
struct LoraCheckArgs {
    const int32_t *plan;
    int M, N, max_rank;
    const int64_t *A, *B, *GA, *GB;
    const int32_t *rank;
    int32_t *hdr;
};

cudaError_t lora_set_attributes();
cudaError_t launch_lora_plan(const LoraPlanArgs &a, int ids_dtype, cudaStream_t s);
cudaError_t launch_lora_check(const LoraCheckArgs &a, cudaStream_t s);
cudaError_t launch_lora_shrink(const LoraArgs &a, cudaStream_t s);
cudaError_t launch_lora_expand(const LoraArgs &a, cudaStream_t s);
cudaError_t launch_lora_outer(const LoraArgs &a, cudaStream_t s);

}  // namespace exl3
