// What the adapters' tensor-core kernels share: descriptors, copies, the even
// split of a launch's work and the swizzled shared-memory layout.
//
// Operand layouts (16-bit elements, 128-byte rows in groups of 8, the 16-byte
// chunk c of row r stored at chunk c ^ (r % 8), tiles aligned to 1024 bytes):
//   K-major:  rows are M or N indices, a row holds 64 contraction steps;
//   MN-major: rows are contraction steps, a row holds 64 M or N indices; the
//             next 64 of them start `lbo` bytes on, the next 8 steps 1024.
#pragma once
#include "common.cuh"
#include "expert_tc.cuh"
#include "lora.h"

namespace exl3 {
namespace lora {

using tc::fence_after;
using tc::fence_before;
using tc::mbar_arrive;
using tc::mma_commit;
using tc::mma_f16;
using tc::tmem_ld16_issue;
using tc::tmem_ld16_wait;
using tc::wait_bar;
using tc::warp_wait_bar;

constexpr int kRestBits = 11;       // f16: the rests of h and dh are kept times 2^11 (split2)

EXL3_DEV void cp_async16(uint32_t dst, const void *src, bool valid)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0)
                 : "memory");
}
EXL3_DEV void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }
// Arrives on `bar` when the thread's copies so far have landed.  The reader
// then runs the proxy fence: one in the copying threads waits for every copy
// they have in flight (16384-row shrink: 40 us with it there, whatever the ring).
EXL3_DEV void cp_async_arrive(uint64_t *bar)
{
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
}
EXL3_DEV void fence_proxy() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

EXL3_DEV uint32_t swz(int row, int chunk) { return (uint32_t)(row * 128 + ((chunk ^ (row & 7)) << 4)); }

EXL3_DEV uint64_t desc_k_major(uint32_t addr) { return tc::smem_desc_swz(addr, 1024, 128); }
EXL3_DEV uint64_t desc_mn_major(uint32_t addr, uint32_t lbo)
{
    uint64_t d = (uint64_t)((addr >> 4) & 0x3FFF);
    d |= (uint64_t)((lbo >> 4) & 0x3FFF) << 16;
    d |= (uint64_t)(1024 >> 4) << 32;
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)2 << 61;
    return d;
}

// f32 accumulate, 16-bit A and B, M = 128, N = n; ta / tb: that operand is MN-major
EXL3_DEV uint32_t idesc(int n, int act_dtype, int ta, int tb)
{
    const uint32_t f = act_dtype == EXL3_BF16 ? 1u : 0u;
    return (1u << 4) | (f << 7) | (f << 10) | ((uint32_t)ta << 15) | ((uint32_t)tb << 16) |
           ((uint32_t)(n >> 3) << 17) | (8u << 24);
}

// 32 accumulator columns of the warp's lane quarter.
EXL3_DEV void tmem_ld32(uint32_t taddr, uint32_t (&v)[32])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
          "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]),
          "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]),
          "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
        : "r"(taddr));
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
                   "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]),
                   "+r"(v[15]), "+r"(v[16]), "+r"(v[17]), "+r"(v[18]), "+r"(v[19]), "+r"(v[20]), "+r"(v[21]),
                   "+r"(v[22]), "+r"(v[23]), "+r"(v[24]), "+r"(v[25]), "+r"(v[26]), "+r"(v[27]), "+r"(v[28]),
                   "+r"(v[29]), "+r"(v[30]), "+r"(v[31])::"memory");
}

// 16 columns of the warp's lane quarter, to be followed by tmem_st_wait.
EXL3_DEV void tmem_st16(uint32_t taddr, const uint4 (&v)[4])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
                     taddr),
                 "r"(v[0].x), "r"(v[0].y), "r"(v[0].z), "r"(v[0].w), "r"(v[1].x), "r"(v[1].y), "r"(v[1].z),
                 "r"(v[1].w), "r"(v[2].x), "r"(v[2].y), "r"(v[2].z), "r"(v[2].w), "r"(v[3].x), "r"(v[3].y),
                 "r"(v[3].z), "r"(v[3].w)
                 : "memory");
}
EXL3_DEV void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// MMA whose A is in TMEM: lane = row, two consecutive k a column, 8 columns for its 16 k.
EXL3_DEV void mma_f16_a_tmem(uint32_t d, uint32_t a, uint64_t b, uint32_t id, bool accumulate)
{
    asm volatile("{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
                 " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
                 "r"(a), "l"(b), "r"(id), "r"((uint32_t)accumulate)
                 : "memory");
}
// The same with D = A B + D / 2^kRestBits.
EXL3_DEV void mma_f16_a_tmem_unscale(uint32_t d, uint32_t a, uint64_t b, uint32_t id)
{
    asm volatile("{\n .reg .pred p;\n setp.ne.u32 p, 1, 0;\n"
                 " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p, %4;\n}\n" ::"r"(d),
                 "r"(a), "l"(b), "r"(id), "n"(kRestBits)
                 : "memory");
}

EXL3_DEV void tmem_alloc(uint32_t *dst, uint32_t cols)
{
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(dst)),
                 "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
EXL3_DEV void tmem_free(uint32_t addr, uint32_t cols)
{
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols) : "memory");
}

// Two values rounded to the activation type, lo in the low half.
EXL3_DEV uint32_t pack2(float lo, float hi, int dtype)
{
    if (dtype == EXL3_BF16) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&v);
    }
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}
EXL3_DEV float2 unpack2(uint32_t u, int dtype)
{
    if (dtype == EXL3_BF16)
        return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&u));
    return __half22float2(*reinterpret_cast<const __half2 *>(&u));
}

// Two values as two parts each of the 16-bit type: hi = round(v), lo =
// round(rest_scale (v - hi)).  bf16 (rest_scale 1): 16 bits of v together.  f16:
// the rest is kept 2^11 times as large (at most 32768 beside the largest hi), and
// what reads it sums its products apart and divides once: 22 bits of v down to
// 2^-14, below it an absolute error of 2^-36 (unscaled it was 2^-25, 0.2 to 5%
// of gradients whose dh lay between 6e-6 and 3e-7).  Where hi overflows it
// stands alone, so that a product gives the infinity and not inf - inf.
EXL3_DEV float rest_scale(int dtype) { return dtype == EXL3_F16 ? (float)(1 << kRestBits) : 1.0f; }
EXL3_DEV void split2(float x, float y, int dtype, uint32_t &hi, uint32_t &lo)
{
    hi = pack2(x, y, dtype);
    const float2 f = unpack2(hi, dtype);
    const float s = rest_scale(dtype);
    lo = pack2(fabsf(f.x) < INFINITY ? s * (x - f.x) : 0.0f, fabsf(f.y) < INFINITY ? s * (y - f.y) : 0.0f, dtype);
}

EXL3_DEV bool plan_ok(const int32_t *plan, int M, int N)
{
    return plan[kLpMagic] == kLoraMagic && plan[kLpM] == M && plan[kLpN] == N && plan[kLpError] == 0;
}

// After a wait ran out: the MMAs issued so far end (waited for with a limit)
// before their TMEM is freed.
EXL3_DEV void drain_mmas(uint64_t *bar)
{
    mma_commit(bar);
    mbar_wait(bar, 0);
}

// Launch that may start while the kernel before it in the stream still runs;
// the kernel itself waits (grid_dep_wait) before it touches that one's results.
template <typename Args>
cudaError_t launch_dependent(void (*kernel)(Args), int grid, int threads, size_t smem, cudaStream_t s, const Args &a)
{
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

// Ring position over n slots.
struct Ring {
    uint32_t slot = 0, phase = 0;
    EXL3_DEV void next(uint32_t n)
    {
        if (++slot == n) {
            slot = 0;
            phase ^= 1;
        }
    }
    // two at a time (n >= 2), for loader groups that take turns
    EXL3_DEV void next2(uint32_t n)
    {
        slot += 2;
        if (slot >= n) {
            slot -= n;
            phase ^= 1;
        }
    }
};

}  // namespace lora
}  // namespace exl3
