// Adapter plan, workspace layout, kernel arguments and launchers (internal).
#pragma once
#include <cuda_runtime_api.h>
#include <stdint.h>

#include "../../include/exl3.h"
#include "plan.h"

namespace exl3 {

constexpr int kLoraMagic = 0x4c6f5241;
constexpr int kLoraTile = 128;      // rows of a prompt tile
constexpr int kLoraSmallTile = 8;   // rows of a decode tile

enum LoraPlanWord {
    kLpError = 0,      // sticky device error word
    kLpMagic = 1,
    kLpM = 2,
    kLpN = 3,
    kLpTiles = 4,      // prompt tiles (adapter tiles first, idle rows' tiles last)
    kLpSmallTiles = 5,
    kLpActive = 6,     // prompt tiles of adapters
    kLpSmallActive = 7,
    kLpUsed = 8,       // adapters that have rows
    kLpWords = 64
};

// Rows grouped by adapter: slot s holds row perm[s]; adapter a's slots are
// offsets[a] .. offsets[a+1], those without an adapter offsets[N] .. M.  A
// tile is (adapter or -1, first slot, rows, 0).  steps[a]: 64-row steps of the
// adapters before a (the outer product's contraction).
struct LoraPlanLayout {
    size_t offsets, perm, tiles, small, steps, total;
};

EXL3_HD inline LoraPlanLayout lora_plan_layout(int M, int N)
{
    LoraPlanLayout L{};
    size_t o = kLpWords * 4;
    L.offsets = o; o = align_up(o + (size_t)(N + 2) * 4, 256);
    L.perm = o;    o = align_up(o + (size_t)M * 4, 256);
    L.tiles = o;   o = align_up(o + ((size_t)M / kLoraTile + N + 1) * 16, 256);
    L.small = o;   o = align_up(o + ((size_t)M / kLoraSmallTile + N + 1) * 16, 256);
    L.steps = o;   o = align_up(o + (size_t)(N + 1) * 4, 256);
    L.total = o;
    return L;
}

// h and dh are operands of the products that follow, and those take 16-bit
// types.  One rounding there would be as large as the result's own (a gradient
// that one row determines had twice the error it needs), so a row keeps h in
// two parts, round(h) and the rounded rest (split2 in lora_common.cuh), and a
// product takes both: 2 lora_h_cols values a row, the rests from lora_h_cols on.
EXL3_HD inline int lora_h_cols(int max_rank) { return (max_rank + 15) / 16 * 16; }
EXL3_HD inline int lora_h_pitch(int h_cols) { return 2 * h_cols; }

// The products share their work out evenly over at most this many CTAs (one
// per SM); a workspace is sized for it whatever the device.
constexpr int kLoraCtas = 152;
constexpr int kShrinkK = 128;        // inputs of one shrink stage
constexpr int kOuterK = 64;          // rows of one outer stage
constexpr int kOuterN = 256;         // columns of one outer item
// Stages below which a CTA is not worth its share.  With 2 / 4 / 8: shrink,
// 1100-row forward 17.1 / 16.5 / 17.7 us, 4096-row training 75.9 / 74.9 / 76.1.
// An outer share is no shorter than a mean item (its stages: steps of the
// adapters that have rows) up to kOuterMin, so that short items are spread out
// and few are cut.  Training with least shares of 1 / 2 / 4 stages: 8 rows, rank
// 8, 13.3 / 14.2 / 16.6 us; 300 rows of four adapters of rank 16, 22.2 / 18.3 /
// 19.9; 256 rows of one of rank 128, 45.7 / 43.5 / 36.0.
constexpr int kShrinkMin = 4;
constexpr int kOuterMin = 4;
EXL3_HD inline int lora_outer_min(int steps, int used)
{
    const int mean = steps / (used > 1 ? used : 1);
    return mean < 1 ? 1 : mean < kOuterMin ? mean : kOuterMin;
}

// `total` units in contiguous shares: CTA c takes [c*per, (c+1)*per).
EXL3_HD inline int lora_share(int total, int ctas, int least)
{
    const int per = (total + ctas - 1) / ctas;
    return per > least ? per : least;
}

// Workspace: error word, dh, and fp32 partial sums.  A shrink tile t cut by
// the shares holds one partial [rows][h_cols] per CTA c that has a part of it,
// at row (first slot of t) + 128 c: parts of one tile are 128 rows apart, and
// a later tile never has a lower c, so none overlap.  The outer product keeps
// at most two partials [h_cols][kOuterN] per CTA (its first and its last item).
struct LoraWsLayout {
    size_t hdr, h, part, total;
};

EXL3_HD inline LoraWsLayout lora_ws_layout(int M, int N, int in_f, int out_f, int max_rank)
{
    (void)N; (void)in_f; (void)out_f;
    LoraWsLayout L{};
    const size_t hc = lora_h_cols(max_rank), shrink = (size_t)M + 128 * (size_t)kLoraCtas;
    const size_t outer = 2 * kOuterN * (size_t)kLoraCtas;
    size_t o = 0;
    L.hdr = o;  o = align_up(o + kHdrWords * 4, 256);
    L.h = o;    o = align_up(o + (size_t)M * lora_h_pitch((int)hc) * 2, 256);
    L.part = o; o = align_up(o + (shrink > outer ? shrink : outer) * hc * 4, 256);
    L.total = o;
    return L;
}

struct LoraPlanArgs {
    const void *ids;
    int M, N;
    int32_t *plan;
};

// shrink: partial sums over the width of h[s][j] = sum_i x[perm[s]][i] W_a[j][i].
// Its first CTA also checks the tables (those of adapters that have rows; with
// gradient tables, of every adapter) and writes the call's error word.
struct LoraShrinkArgs {
    const int32_t *plan;
    int M, N, act_dtype, max_rank, h_cols, width;
    const void *x;
    const int64_t *W;
    const int32_t *rank;
    float *part;
    const int64_t *A, *B, *GA, *GB;
    int32_t *hdr;
};

// join: h[s][j] = h_scale * (sum of shrink's partials) in two parts of the activation
// type, zero from the adapter's rank up to the next multiple of 16; h_scale:
// the adapter's scale where `scale_h`, else 1.
struct LoraJoinArgs {
    const int32_t *plan;
    int M, N, act_dtype, h_cols, scale_h;
    const float *part;
    int shrink_width, shrink_ctas;  // the shares that cut shrink's tiles
    const int32_t *rank;
    const float *scale;
    void *h;
    const int32_t *hdr;
};

// expand: y[perm[s]][n] = base[perm[s]][n] + y_scale * sum_j h[s][j] W_a[j][n];
// y_scale: 1 where `scale_h`, else the adapter's scale.
struct LoraExpandArgs {
    const int32_t *plan;
    int M, N, act_dtype, h_cols, width, scale_h;
    const void *h;
    const int64_t *W;
    const int32_t *rank;
    const float *scale;
    const void *base;
    void *y;
    int32_t *hdr;
};

// rows: both products of a batch of few rows (and the table check) in one
// launch: h = h_scale * W1 x, y = base + y_scale * h W2.
struct LoraRowsArgs {
    const int32_t *plan;
    int M, N, act_dtype, max_rank, h_cols, in_width, out_width, scale_h;
    int ctas;                       // of one cluster (set by the launcher)
    const void *x;
    const int64_t *W1, *W2, *GA, *GB;
    const int32_t *rank;
    const float *scale;
    const void *base;
    void *y, *h;
    int32_t *hdr;
};

// outer: G_a[j][n] = g_scale * sum_s h[s][j] x[perm[s]][n], two such products
// (dA and dB) in one launch; g_scale: the adapter's scale where `scaled`.
struct LoraOuterArgs {
    const int32_t *plan;
    int M, N, act_dtype, h_cols, ctas;
    const int32_t *rank;
    const float *scale;
    struct Product {
        const void *x, *h;
        const int64_t *G;
        int width, scaled;
    } p[2];
    float *part;
    int32_t *hdr;
};

cudaError_t lora_set_attributes();
cudaError_t launch_lora_plan(const LoraPlanArgs &a, int ids_dtype, cudaStream_t s);
cudaError_t launch_lora_shrink(const LoraShrinkArgs &a, int ctas, cudaStream_t s);
cudaError_t launch_lora_join(const LoraJoinArgs &a, cudaStream_t s);
cudaError_t launch_lora_expand(const LoraExpandArgs &a, int ctas, cudaStream_t s);
cudaError_t launch_lora_rows(LoraRowsArgs a, int sms, cudaStream_t s);
cudaError_t launch_lora_outer(const LoraOuterArgs &a, cudaStream_t s);
cudaError_t lora_plan_set_attributes();
cudaError_t lora_shrink_set_attributes();
cudaError_t lora_expand_set_attributes();
cudaError_t lora_outer_set_attributes();

}  // namespace exl3
