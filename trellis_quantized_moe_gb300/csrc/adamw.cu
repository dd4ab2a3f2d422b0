// AdamW over many tensors (include/exl3.h, "optimiser").
//
// k_adamw_begin checks the tables, counts the step and turns the step's scalars
// into a few floats in the workspace.  k_adamw makes the step: a warp takes a block
// of 256 elements at a time, eight a lane, so that with 8-bit states the warp holds
// what shares a scale: the largest value is one warp reduction, and everything is
// read and written once.
//
// Bound by HBM where there are masters or 32-bit states (245M elements, 8-bit states
// and masters: 611 us, 6.4 TB/s; 9.5M with 32-bit states: 44.9 us, 5.9 TB/s), by
// instructions and latency with 8-bit states alone (20M elements: 41.9 us, 4.9 TB/s;
// 42 instructions an element, two cycles of three issue).  Warps take few blocks and
// there are as many CTAs as that needs: the loads of new CTAs then meet the stores
// of old ones in long runs (245M elements of a 16-byte pattern without arithmetic:
// 7.0 TB/s so, 6.0 to 6.7 with persistent CTAs whatever their copies).  Rounding at
// random is bound by instructions: 245M elements 1.13, 20M elements 1.44 times as long
// as to the nearest.  Of all kinds three spill, one or two registers: f32 parameters
// with 32-bit states, and 16-bit ones with f32 gradients, masters and codes rounded to
// the nearest (245M elements: 710 us, 6.2 TB/s).
#include <cuda_fp8.h>
#include <type_traits>

#include "adamw.h"
#include "rows.cuh"

namespace exl3 {

namespace {

constexpr int kBeginThreads = 512;
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr float kTop = 448.0f;          // largest e4m3 value
constexpr float kTopInv = 1.0f / 448.0f;
constexpr float kLeast = 0.001953125f;  // smallest above zero, 2^-9

// Random bits that depend on the step and on an element's place in its tensor
// alone, so that they are the same in every grouping, replay and grid: the high half
// of a product with an odd constant folded into the low one, a few times over.  The
// constants are the first 32 bits of the fractions of the golden ratio and of the
// roots of 2, 3, 11 and 17 (odd ones).  Words of 512 elements over 8192 steps and of
// 65536 over 64: mean, chi-square of 1024 bins, counts of rare values, correlations
// between steps, between elements and across both as of independent ones.
constexpr uint32_t kGolden = 0x9e3779b9u, kRoot2 = 0x6a09e667u, kRoot3 = 0xbb67ae85u, kRoot11 = 0x510e527fu,
                   kRoot17 = 0x1f83d9abu;

EXL3_DEV uint32_t fold(uint32_t x, uint32_t odd)
{
    const uint64_t p = (uint64_t)x * odd;
    return (uint32_t)(p >> 32) ^ (uint32_t)p;
}

EXL3_DEV bool bad_pointer(const int64_t *table, int i, int align)
{
    const int64_t p = table ? table[i] : align;
    return p == 0 || (p & (align - 1)) != 0;
}

// One CTA: with 1 / 1152 / 3000 / 10000 tensors of a block each a step takes 3.6 / 5.9 /
// 9.6 / 21 us.
__global__ void __launch_bounds__(kBeginThreads) k_adamw_begin(AdamwArgs a)
{
    grid_dep_wait();
    grid_dep_launch();
    const exl3_adamw_tensors &t = a.t;
    bool bad = false;
    AdamwScalars s{};
    int32_t now = 0;
    if (threadIdx.x == 0) {                         // while the others check the tables
        const float gs = a.grad_scale ? *a.grad_scale : 1.0f;
        const double lr = a.lr_scale ? a.lr * (double)*a.lr_scale : a.lr;
        const int32_t made = *a.step;
        bad = t.first[0] != 0 || t.first[t.N] != t.blocks || made < 0 || made == INT32_MAX;
        now = bad ? 1 : made + 1;
        // 1 - beta^t: expm1 keeps its digits where beta^t is near one
        const float first = -expm1f((float)(now * a.log_beta1)), second = -expm1f((float)(now * a.log_beta2));
        s.decay = (float)(1.0 - lr * a.weight_decay);
        s.rate = (float)-lr / first;
        s.run = isfinite(gs) && isfinite(s.decay) && isfinite(s.rate);
        s.root = 1.0f / sqrtf(second);
        s.grad = gs;
        s.second = gs * sqrtf(a.c2);
        s.seed = fold(fold((uint32_t)now ^ kGolden, kRoot2), kRoot3);
    }
    for (int i = (int)threadIdx.x - 32; i < t.N; i += kBeginThreads - 32) {
        if (i < 0)                                  // the first warp
            break;
        const int64_t n = t.numel[i], b = t.first[i], e = t.first[i + 1];
        bad |= n < 0 || b < 0 || e - b != n / kAdamwBlock + (n % kAdamwBlock != 0);
        // no short circuits: all loads of the round at once
        const bool p = bad_pointer(t.param, i, 16) | bad_pointer(t.grad, i, 16) | bad_pointer(t.m, i, 16) |
                       bad_pointer(t.v, i, 16) | bad_pointer(t.master, i, 16) | bad_pointer(t.m_scale, i, 4) |
                       bad_pointer(t.v_scale, i, 4);
        bad |= n > 0 && p;
    }
    bad = __syncthreads_or(bad);
    if (threadIdx.x == 0) {
        if (bad) {
            s.error = EXL3_DERR_TABLE;
            s.run = 0;
        }
        *a.out = s;
        if (s.run)
            *a.step = now;
    }
}

// Square root and reciprocal within 1 ulp.  A subnormal v counts (eps may be far
// smaller than its root; 1% of 245M elements' time); the denominator is at least
// eps, a normal number.
EXL3_DEV float root_of(float v)
{
    float r;
    asm("sqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
EXL3_DEV float reciprocal(float v)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// ---------------------------------------------------------------- eight elements of a lane
template <int DT>
struct Raw {
    static constexpr int kWords = DT == EXL3_F32 ? 8 : DT == EXL3_E4M3 ? 2 : 4;
    static constexpr int kBytes = kWords / 2;           // of an element
    uint32_t w[kWords];

    EXL3_DEV void load(const void *p)
    {
        if constexpr (kWords == 2) {
            const uint2 u = *static_cast<const uint2 *>(p);
            w[0] = u.x;
            w[1] = u.y;
        } else {
#pragma unroll
            for (int k = 0; k < kWords / 4; k++) {
                const uint4 u = static_cast<const uint4 *>(p)[k];
                w[4 * k] = u.x;
                w[4 * k + 1] = u.y;
                w[4 * k + 2] = u.z;
                w[4 * k + 3] = u.w;
            }
        }
    }
    // FULL: all eight, else n (0..8)
    template <bool FULL>
    EXL3_DEV void store(void *p, int n) const
    {
        if constexpr (FULL && kWords == 2) {
            *static_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
        } else if constexpr (FULL) {
#pragma unroll
            for (int k = 0; k < kWords / 4; k++)
                static_cast<uint4 *>(p)[k] = make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
        } else {
#pragma unroll
            for (int k = 0; k < 8; k++)
                if (k < n) {
                    if constexpr (kBytes == 4)
                        static_cast<uint32_t *>(p)[k] = w[k];
                    else if constexpr (kBytes == 2)
                        static_cast<uint16_t *>(p)[k] = (uint16_t)(w[k / 2] >> (k % 2 * 16));
                    else
                        static_cast<uint8_t *>(p)[k] = (uint8_t)(w[k / 4] >> (k % 4 * 8));
                }
        }
    }
    EXL3_DEV void get(float (&v)[8]) const
    {
        if constexpr (DT == EXL3_F32) {
#pragma unroll
            for (int k = 0; k < 8; k++)
                v[k] = __uint_as_float(w[k]);
        } else if constexpr (DT == EXL3_E4M3) {
#pragma unroll
            for (int k = 0; k < 4; k++) {
                const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[k / 2] >> (k % 2 * 16)), __NV_E4M3);
                const float2 f = __half22float2(__half2(h));
                v[2 * k] = f.x;
                v[2 * k + 1] = f.y;
            }
        } else {
            unpack<DT>(make_uint4(w[0], w[1], w[2], w[3]), v);
        }
    }
    EXL3_DEV void set(const float (&v)[8])
    {
        if constexpr (DT == EXL3_F32) {
#pragma unroll
            for (int k = 0; k < 8; k++)
                w[k] = __float_as_uint(v[k]);
        } else if constexpr (DT == EXL3_E4M3) {
#pragma unroll
            for (int k = 0; k < 2; k++) {
                const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * k], v[4 * k + 1]), __NV_SATFINITE, __NV_E4M3);
                const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * k + 2], v[4 * k + 3]), __NV_SATFINITE, __NV_E4M3);
                w[k] = lo | hi << 16;
            }
        } else {
            const uint4 u = pack<DT>(v);
            w[0] = u.x;
            w[1] = u.y;
            w[2] = u.z;
            w[3] = u.w;
        }
    }
};

// The e4m3 value next to y at or below |y|, or the one above it with the
// probability that keeps the mean: 20 random bits added below the last one that is
// kept.  Below 2^-6 codes are a fixed 2^-9 apart, which adding 2^-6 makes the
// floats' own spacing.  (beta2 = 0.9999 moves a root by some 2^-11 of a code's width a
// step, of which 20 bits keep 2^-9.)  A NaN stays one.
EXL3_DEV float rounded_at_random(float y, uint32_t bits20)
{
    const float a = fabsf(y), up = a < 0.015625f ? 0.015625f : 0.0f;
    const float low = __uint_as_float((__float_as_uint(a + up) + bits20) & 0xfff00000u) - up;
    return a < 512.0f ? copysignf(low, y) : y;
}

// The largest |value| of the warp's 256, NaNs left out: bit patterns of floats above zero order as integers.
EXL3_DEV float block_top(const float (&v)[8])
{
    float top = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; k++)
        top = fmaxf(top, fabsf(v[k]));
    return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));
}

// A tensor's arrays from one of its blocks on.
struct Arrays {
    char *param, *grad, *m, *v, *master;
    float *m_scale, *v_scale;
};

// The last tensor that begins at block b or before, by a warp: 32 places at a time.
EXL3_DEV int tensor_of(const int64_t *first, int N, int64_t b, int lane)
{
    int lo = 0;
    for (int n = N; n > 1;) {
        const int step = (n + 31) / 32, at = lane * step;
        const unsigned before = __ballot_sync(0xffffffffu, at < n && first[lo + at] <= b);
        const int c = (__popc(before) - 1) * step;
        lo += c;
        n = min(step, n - c);
    }
    return lo;
}

// WHOLE: all 16 bytes, else the first `bytes` and zeros.
template <bool WHOLE>
EXL3_DEV void copy_async16(uint32_t dst, const void *src, int bytes)
{
    if constexpr (WHOLE)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
    else
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
EXL3_DEV void copy_async4(uint32_t dst, const void *src)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

// All but the newest n groups of the thread's copies (a constant after unrolling).
EXL3_DEV void wait_copies(int n)
{
    switch (n) {
    case 0: asm volatile("cp.async.wait_group 0;" ::: "memory"); break;
    case 1: asm volatile("cp.async.wait_group 1;" ::: "memory"); break;
    default: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
    }
}

// What a warp does: its blocks' arrays go to shared memory of its own, so that
// loads in flight cost no registers and a block's end needs no branches in them.
template <int PT, int GT, bool CODES, bool MASTER, bool RANDOM>
struct Warp {
    using Grad = Raw<GT>;
    using Weight = Raw<MASTER ? EXL3_F32 : PT>;
    using State = Raw<CODES ? EXL3_E4M3 : EXL3_F32>;
    static constexpr int kWeight = kAdamwBlock * Grad::kBytes, kM = kWeight + kAdamwBlock * Weight::kBytes;
    static constexpr int kV = kM + kAdamwBlock * State::kBytes, kScales = kV + kAdamwBlock * State::kBytes;
    static constexpr int kStage = kScales + (CODES ? 16 : 0);
    // Blocks of a warp, all on their way at once.  8-bit states: 20M elements with 2 /
    // 3 / 4 take 42.8 / 41.7 / 41.4 us, 245M with masters 621 / 603 / 626 (before roots
    // of subnormal v, 611 with them; 725 with five CTAs an SM, whose registers spill);
    // 32-bit states: 9.5M elements with 1 / 2 / 4 took 47.8 / 49.1 / 51.2 us.
    static constexpr int kPer = CODES ? 3 : 1;
    static constexpr int kSmem = kWarps * kPer * kStage;

    // The bytes of a block's array, 16 a lane and step; rem: its elements, behind which comes zero.
    template <int BYTES, bool FULL>
    EXL3_DEV static void fetch_array(uint32_t dst, const char *src, int rem, int lane)
    {
        constexpr int kPieces = kAdamwBlock * BYTES / 16;
#pragma unroll
        for (int q = 0; q < kPieces; q += 32) {
            const int at = (q + lane) * 16;
            if (kPieces >= 32 || lane < kPieces) {
                const int n = FULL ? 16 : min(16, max(0, rem * BYTES - at));
                copy_async16<FULL>(dst + at, FULL || n > 0 ? src + at : src, n);
            }
        }
    }
    // Block j of the arrays.
    template <bool FULL>
    EXL3_DEV static void fetch(uint32_t dst, const Arrays &t, int j, int rem, int lane)
    {
        const int at = j * kAdamwBlock;
        fetch_array<Grad::kBytes, FULL>(dst, t.grad + at * Grad::kBytes, rem, lane);
        fetch_array<Weight::kBytes, FULL>(dst + kWeight, (MASTER ? t.master : t.param) + at * Weight::kBytes, rem, lane);
        if constexpr (CODES) {                          // half a warp each
            const int piece = lane % 16 * 16;
            const int n = FULL ? 16 : min(16, max(0, rem - piece));
            const char *src = (lane < 16 ? t.m : t.v) + at;
            copy_async16<FULL>(dst + (lane < 16 ? kM : kV) + piece, FULL || n > 0 ? src + piece : src, n);
            if (lane % 16 == 0)
                copy_async4(dst + kScales + lane / 4, (lane < 16 ? t.m_scale : t.v_scale) + j);
        } else {
            fetch_array<State::kBytes, FULL>(dst + kM, t.m + at * 4, rem, lane);
            fetch_array<State::kBytes, FULL>(dst + kV, t.v + at * 4, rem, lane);
        }
    }

    // One block.  m's recurrence is single rounded operations, no fused ones: a
    // value of m that is nearly the block's largest decides the next step's scale, and
    // so its 8-bit code is to depend on the inputs alone.  v: with the code d, its
    // scale r and x the gradient as it came, (x second)^2 + (d (r sqrt(beta2)))^2; in
    // 32 bits beta2 itself, an error of which would be 1 / (1 - beta2) times as
    // large in a v of many steps.
    template <bool FULL>
    EXL3_DEV static void step(const AdamwArgs &a, const char *stage, const Arrays &t, int64_t block, int j, int rem,
                              int lane)
    {
        const int n = FULL ? 8 : min(8, max(0, rem - lane * 8));
        const int at = j * kAdamwBlock + lane * 8;
        Grad g;
        Weight p;
        State m, v;
        g.load(stage + lane * 8 * Grad::kBytes);
        p.load(stage + kWeight + lane * 8 * Weight::kBytes);
        m.load(stage + kM + lane * 8 * State::kBytes);
        v.load(stage + kV + lane * 8 * State::kBytes);
        float ms = 1.0f, vs = 1.0f;
        if constexpr (CODES) {
            ms = *reinterpret_cast<const float *>(stage + kScales);
            vs = *reinterpret_cast<const float *>(stage + kScales + 4);
        }
        const float decay = a.out->decay, rate = a.out->rate, root_scale = a.out->root, scale = a.out->grad,
                    second = a.out->second;
        vs *= a.root_b2;
        float gf[8], pf[8], mf[8], vf[8];
        g.get(gf);
        p.get(pf);
        m.get(mf);
        v.get(vf);
#pragma unroll
        for (int k = 0; k < 8; k++) {
            const float h = gf[k] * second;
            if constexpr (CODES)
                mf[k] = __fmul_rn(mf[k], ms);
            mf[k] = __fadd_rn(__fmul_rn(mf[k], a.b1), __fmul_rn(__fmul_rn(gf[k], scale), a.c1));
            if constexpr (CODES) {
                const float r = vf[k] * vs;
                vf[k] = fmaf(h, h, r * r);
            } else {
                vf[k] = fmaf(h, h, vf[k] * a.b2);
            }
            const float root = root_of(vf[k]);
            pf[k] = fmaf(mf[k] * rate, reciprocal(fmaf(root, root_scale, a.eps)), pf[k] * decay);
            if constexpr (CODES)
                vf[k] = root;
        }
        p.set(pf);
        p.template store<FULL>((MASTER ? t.master : t.param) + at * Weight::kBytes, n);
        if constexpr (MASTER) {
            Raw<PT> low;
            low.set(pf);
            low.template store<FULL>(t.param + at * low.kBytes, n);
        }
        if constexpr (CODES) {
            // one reciprocal for both scales: half the lanes each
            const float mt = block_top(mf), vt = block_top(vf);
            const float mine = lane < 16 ? mt : vt;
            // nothing at all, or nothing above 2^-117, is zero; an infinity makes the block NaN
            const bool some = mine > 6.0e-36f;
            const float inv = some ? __fmul_rn(__frcp_rn(mine), kTop) : 0.0f;
            const float mi = __shfl_sync(0xffffffffu, inv, 0), vi = __shfl_sync(0xffffffffu, inv, 31);
            bool above = vi > 0.0f;                         // as nearly always; a NaN is not
#pragma unroll
            for (int k = 0; k < 8; k++) {
                above = above && vf[k] > 0.0f;
                mf[k] = __fmul_rn(mf[k], mi);
            }
            if (above) {
#pragma unroll
                for (int k = 0; k < 8; k++)
                    vf[k] = fmaxf(vf[k] * vi, kLeast);
            } else {
#pragma unroll
                for (int k = 0; k < 8; k++) {
                    const float y = vf[k] * vi;
                    vf[k] = y > 0.0f ? fmaxf(y, kLeast) : y;
                }
            }
            if constexpr (RANDOM) {
                const int64_t b = block + j;
                uint32_t s = fold(a.out->seed ^ (uint32_t)b, kRoot2) + (uint32_t)(b >> 32) + lane * kGolden;
                s = fold(s, kRoot3);
#pragma unroll
                for (int k = 0; k < 8; k++) {
                    // 20 bits each, eight of them the high ones of the first, the low ones of the second
                    const uint32_t w = fold(fold(s + k * kGolden, kRoot11) ^ s, kRoot17);
                    mf[k] = rounded_at_random(mf[k], w & 0xfffffu);
                    vf[k] = rounded_at_random(vf[k], w >> 12);
                }
            }
            if (lane % 16 == 0)
                (lane == 0 ? t.m_scale : t.v_scale)[j] = some ? mine * kTopInv : 0.0f;
        }
        m.set(mf);
        m.template store<FULL>(t.m + at * State::kBytes, n);
        v.set(vf);
        v.template store<FULL>(t.v + at * State::kBytes, n);
    }
};

template <int PT, int GT, bool CODES, bool MASTER, bool RANDOM>
__global__ void __launch_bounds__(kThreads, 4) k_adamw(AdamwArgs a)
{
    using W = Warp<PT, GT, CODES, MASTER, RANDOM>;
    extern __shared__ __align__(16) char stages[];
    grid_dep_wait();
    grid_dep_launch();
    const exl3_adamw_tensors &t = a.t;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t b = ((int64_t)blockIdx.x * kWarps + warp) * W::kPer;
    if (!a.out->run || b >= t.blocks)
        return;
    const int64_t stop = min(b + W::kPer, t.blocks);
    char *mine = stages + warp * W::kPer * W::kStage;
    for (int i = tensor_of(t.first, t.N, b, lane); b < stop; i++) {
        const int64_t block = b - t.first[i], at = block * kAdamwBlock;
        const int run = (int)(min(stop, t.first[i + 1]) - b);       // 0: an empty tensor
        const int left = (int)min((int64_t)W::kPer * kAdamwBlock, t.numel[i] - at);
        const auto array = [i, at](const int64_t *table, int bytes) { return reinterpret_cast<char *>(table[i]) + at * bytes; };
        const auto scales = [i, block](const int64_t *table) { return reinterpret_cast<float *>(table[i]) + block; };
        const Arrays x{array(t.param, Raw<PT>::kBytes), array(t.grad, Raw<GT>::kBytes), array(t.m, W::State::kBytes),
                       array(t.v, W::State::kBytes), MASTER ? array(t.master, 4) : nullptr,
                       CODES ? scales(t.m_scale) : nullptr, CODES ? scales(t.v_scale) : nullptr};
        if (left == W::kPer * kAdamwBlock && run == W::kPer) {
#pragma unroll
            for (int j = 0; j < W::kPer; j++) {
                W::template fetch<true>(smem_addr(mine) + j * W::kStage, x, j, kAdamwBlock, lane);
                asm volatile("cp.async.commit_group;" ::: "memory");
            }
#pragma unroll
            for (int j = 0; j < W::kPer; j++) {
                wait_copies(W::kPer - 1 - j);
                __syncwarp();
                W::template step<true>(a, mine + j * W::kStage, x, block, j, kAdamwBlock, lane);
            }
        } else {                                    // a tensor's end
#pragma unroll 1
            for (int j = 0; j < run; j++)
                W::template fetch<false>(smem_addr(mine) + j * W::kStage, x, j, left - j * kAdamwBlock, lane);
            asm volatile("cp.async.commit_group;" ::: "memory");
            wait_copies(0);
            __syncwarp();
#pragma unroll 1
            for (int j = 0; j < run; j++) {
                const int rem = left - j * kAdamwBlock;
                if (rem >= kAdamwBlock)
                    W::template step<true>(a, mine + j * W::kStage, x, block, j, rem, lane);
                else
                    W::template step<false>(a, mine + j * W::kStage, x, block, j, rem, lane);
            }
        }
        __syncwarp();
        b += run;
    }
}

// f(parameter type, gradient type, 8-bit states, masters, random rounding) as constants
template <typename F>
cudaError_t by_kind(const exl3_adamw_tensors &t, F f)
{
    const auto rest = [&](auto p, auto g) {
        constexpr std::true_type yes;
        constexpr std::false_type no;
        const auto state = [&](auto master) {
            switch (t.state_dtype) {
            case EXL3_E4M3:
                return f(p, g, yes, master, no);
            case EXL3_E4M3_RANDOM:
                return f(p, g, yes, master, yes);
            default:
                return f(p, g, no, master, no);
            }
        };
        if constexpr (decltype(p)::value != EXL3_F32)
            if (t.master)
                return state(yes);
        return state(no);
    };
    constexpr std::integral_constant<int, EXL3_F16> f16;
    constexpr std::integral_constant<int, EXL3_BF16> bf16;
    constexpr std::integral_constant<int, EXL3_F32> f32;
    const bool wide = t.grad_dtype == EXL3_F32;
    switch (t.param_dtype) {
    case EXL3_F32:
        return rest(f32, f32);
    case EXL3_BF16:
        return wide ? rest(bf16, f32) : rest(bf16, bf16);
    default:
        return wide ? rest(f16, f32) : rest(f16, f16);
    }
}

}  // namespace

cudaError_t adamw_set_attributes()
{
    exl3_adamw_tensors t{};
    const int64_t some = 0;
    for (int param = EXL3_F16; param <= EXL3_F32; param++)
        for (int kind = 0; kind < 12; kind++) {
            t.param_dtype = param;
            t.grad_dtype = kind & 1 ? EXL3_F32 : param;
            t.master = kind & 2 ? &some : nullptr;
            t.state_dtype = kind < 4 ? EXL3_F32 : kind < 8 ? EXL3_E4M3 : EXL3_E4M3_RANDOM;
            const cudaError_t e = by_kind(t, [](auto p, auto g, auto codes, auto master, auto random) {
                return cudaFuncSetAttribute(k_adamw<p.value, g.value, codes.value, master.value, random.value>,
                                            cudaFuncAttributeMaxDynamicSharedMemorySize,
                                            Warp<p.value, g.value, codes.value, master.value, random.value>::kSmem);
            });
            if (e != cudaSuccess)
                return e;
        }
    return cudaSuccess;
}

cudaError_t launch_adamw(const AdamwArgs &a, cudaStream_t s)
{
    const cudaError_t e = launch_dependent(k_adamw_begin, 1, kBeginThreads, 0, s, a);
    if (e != cudaSuccess || a.t.blocks == 0)
        return e;
    return by_kind(a.t, [&](auto p, auto g, auto codes, auto master, auto random) {
        using W = Warp<p.value, g.value, codes.value, master.value, random.value>;
        constexpr int kBlocks = kWarps * W::kPer;
        return launch_dependent(k_adamw<p.value, g.value, codes.value, master.value, random.value>,
                                (int)((a.t.blocks + kBlocks - 1) / kBlocks), kThreads, W::kSmem, s, a);
    });
}

}  // namespace exl3
