// tcgen05.cuh -- inline PTX of the 5th-generation tensor cores and tensor
// memory, shared by the GEMM and the attention kernel.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include "common.cuh"

namespace q4 {

// Host: cuTensorMapEncodeTiled of the driver, or null (api.cu).
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

__device__ __forceinline__ void tmem_alloc(uint32_t *dst_smem, uint32_t ncols)
{
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(dst_smem)),
                 "r"(ncols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void tmem_dealloc(uint32_t taddr, uint32_t ncols)
{
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols)
                 : "memory");
}

// Shared-memory matrix descriptor, 128-byte swizzle (tcgen05 descriptor
// format, version 1).  K-major (a row's k contiguous): 8-row groups 1024
// bytes apart, the leading offset unused.  MN-major (a k's rows contiguous):
// 8-k groups 1024 bytes apart, runs of 64 rows `lead` bytes apart.
__device__ __forceinline__ uint64_t sw128_desc(uint32_t saddr, uint32_t lead = 16u)
{
    uint64_t d = 0;
    d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
    d |= static_cast<uint64_t>(lead >> 4) << 16;   // leading byte offset
    d |= static_cast<uint64_t>(1024u >> 4) << 32;  // stride byte offset: next 8-row (8-k) group
    d |= static_cast<uint64_t>(1) << 46;           // descriptor version
    d |= static_cast<uint64_t>(2) << 61;           // 128-byte swizzle
    return d;
}

// Instruction descriptor, kind::f16: f32 accumulate, A/B bf16 (ab = 1) or
// f16 (ab = 0), both K-major, M = 128, N = n (a multiple of 16, 16..256).
// With IDESC_B_MN added, B is MN-major.
constexpr uint32_t IDESC_B_MN = 1u << 16;
__host__ __device__ constexpr uint32_t idesc_f16(uint32_t ab, uint32_t n)
{
    return (1u << 4) | (ab << 7) | (ab << 10) | ((n >> 3) << 17) | ((128u >> 4) << 24);
}

// Products of a 128-row tile in groups of MMAs under one election, called by a
// whole warp (one lane, always the same, issues), with a commit behind them.
// d (tensor memory) = a * b^T over K = 16 * N of 64-element chunks 16 KB
// apart, K-major in shared memory (descriptors of their first bytes).
template <int N>
__device__ __forceinline__ void mma_rows_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint64_t *bar)
{
    static_assert(N == 4 || N == 8, "64 or 128 wide");
    const uint32_t al = static_cast<uint32_t>(a), ah = static_cast<uint32_t>(a >> 32);
    const uint32_t bl = static_cast<uint32_t>(b), bh = static_cast<uint32_t>(b >> 32);
    if constexpr (N == 8)
        asm volatile(
        "{\n\t.reg .pred e, p, t;\n\t.reg .b32 x;\n\t.reg .b64 a, b;\n\t"
        "elect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 p, %6, 0;\n\tsetp.eq.b32 t, %6, %6;\n\t"
        "add.u32 x, %1, 0;\n\tmov.b64 a, {x, %3};\n\tadd.u32 x, %2, 0;\n\tmov.b64 b, {x, %4};\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %5, p;\n\t"
        "add.u32 x, %1, 2;\n\tmov.b64 a, {x, %3};\n\tadd.u32 x, %2, 2;\n\tmov.b64 b, {x, %4};\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %5, t;\n\t"
        "add.u32 x, %1, 4;\n\tmov.b64 a, {x, %3};\n\tadd.u32 x, %2, 4;\n\tmov.b64 b, {x, %4};\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %5, t;\n\t"
        "add.u32 x, %1, 6;\n\tmov.b64 a, {x, %3};\n\tadd.u32 x, %2, 6;\n\tmov.b64 b, {x, %4};\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %5, t;\n\t"
        "add.u32 x, %1, 1024;\n\tmov.b64 a, {x, %3};\n\tadd.u32 x, %2, 1024;\n\tmov.b64 b, {x, %4};\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %5, t;\n\t"
        "add.u32 x, %1, 1026;\n\tmov.b64 a, {x, %3};\n\tadd.u32 x, %2, 1026;\n\tmov.b64 b, {x, %4};\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %5, t;\n\t"
        "add.u32 x, %1, 1028;\n\tmov.b64 a, {x, %3};\n\tadd.u32 x, %2, 1028;\n\tmov.b64 b, {x, %4};\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %5, t;\n\t"
        "add.u32 x, %1, 1030;\n\tmov.b64 a, {x, %3};\n\tadd.u32 x, %2, 1030;\n\tmov.b64 b, {x, %4};\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %5, t;\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%7];\n\t}" ::"r"(d),
            "r"(al), "r"(bl), "r"(ah), "r"(bh), "r"(idesc), "r"(0u), "r"(smem_u32(bar))
            : "memory");
    else
        asm volatile(
        "{\n\t.reg .pred e, p, t;\n\t.reg .b32 x;\n\t.reg .b64 a, b;\n\t"
        "elect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 p, %6, 0;\n\tsetp.eq.b32 t, %6, %6;\n\t"
        "add.u32 x, %1, 0;\n\tmov.b64 a, {x, %3};\n\tadd.u32 x, %2, 0;\n\tmov.b64 b, {x, %4};\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %5, p;\n\t"
        "add.u32 x, %1, 2;\n\tmov.b64 a, {x, %3};\n\tadd.u32 x, %2, 2;\n\tmov.b64 b, {x, %4};\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %5, t;\n\t"
        "add.u32 x, %1, 4;\n\tmov.b64 a, {x, %3};\n\tadd.u32 x, %2, 4;\n\tmov.b64 b, {x, %4};\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %5, t;\n\t"
        "add.u32 x, %1, 6;\n\tmov.b64 a, {x, %3};\n\tadd.u32 x, %2, 6;\n\tmov.b64 b, {x, %4};\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %5, t;\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%7];\n\t}" ::"r"(d),
            "r"(al), "r"(bl), "r"(ah), "r"(bh), "r"(idesc), "r"(0u), "r"(smem_u32(bar))
            : "memory");
}
// d += a * b over K = 128 (d = when !acc): a in tensor memory, b MN-major in
// shared memory, 128 bytes a row.
__device__ __forceinline__ void mma_rows_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool acc)
{
    const uint32_t bl = static_cast<uint32_t>(b), bh = static_cast<uint32_t>(b >> 32);
    asm volatile(
        "{\n\t.reg .pred e, p, t;\n\t.reg .b32 x;\n\t.reg .b64 a, b;\n\t"
        "elect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 p, %6, 0;\n\tsetp.eq.b32 t, %6, %6;\n\t"
        "add.u32 x, %2, 0;\n\tmov.b64 b, {x, %4};\n\tadd.u32 x, %1, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], b, %5, p;\n\t"
        "add.u32 x, %2, 128;\n\tmov.b64 b, {x, %4};\n\tadd.u32 x, %1, 8;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], b, %5, t;\n\t"
        "add.u32 x, %2, 256;\n\tmov.b64 b, {x, %4};\n\tadd.u32 x, %1, 16;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], b, %5, t;\n\t"
        "add.u32 x, %2, 384;\n\tmov.b64 b, {x, %4};\n\tadd.u32 x, %1, 24;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], b, %5, t;\n\t"
        "add.u32 x, %2, 512;\n\tmov.b64 b, {x, %4};\n\tadd.u32 x, %1, 32;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], b, %5, t;\n\t"
        "add.u32 x, %2, 640;\n\tmov.b64 b, {x, %4};\n\tadd.u32 x, %1, 40;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], b, %5, t;\n\t"
        "add.u32 x, %2, 768;\n\tmov.b64 b, {x, %4};\n\tadd.u32 x, %1, 48;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], b, %5, t;\n\t"
        "add.u32 x, %2, 896;\n\tmov.b64 b, {x, %4};\n\tadd.u32 x, %1, 56;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], b, %5, t;\n\t"
        "}" ::"r"(d),
        "r"(a), "r"(bl), "r"(0u), "r"(bh), "r"(idesc), "r"(static_cast<uint32_t>(acc))
        : "memory");
}

__device__ __forceinline__ void mma_commit_elected(uint64_t *bar)
{
    asm volatile(
        "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar))
        : "memory");
}

__device__ __forceinline__ void mma_commit(uint64_t *bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                     smem_u32(bar))
                 : "memory");
}

#define Q4_R8(a, o) "r"(a[o + 0]), "r"(a[o + 1]), "r"(a[o + 2]), "r"(a[o + 3]), "r"(a[o + 4]), \
    "r"(a[o + 5]), "r"(a[o + 6]), "r"(a[o + 7])
#define Q4_W8(a, o) "=r"(a[o + 0]), "=r"(a[o + 1]), "=r"(a[o + 2]), "=r"(a[o + 3]), \
    "=r"(a[o + 4]), "=r"(a[o + 5]), "=r"(a[o + 6]), "=r"(a[o + 7])

// 32 consecutive 32-bit columns of this warp's 32 lanes <- v (thread i: lane i).
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&v)[32])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
        "%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
        Q4_R8(v, 0), Q4_R8(v, 8), Q4_R8(v, 16), Q4_R8(v, 24)
        : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&v)[16])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
        "%14,%15,%16};" ::"r"(taddr),
        Q4_R8(v, 0), Q4_R8(v, 8)
        : "memory");
}

__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// v <- consecutive columns of this warp's lanes; complete at tmem_wait_ld.
__device__ __forceinline__ void tmem_ld16x(uint32_t taddr, uint32_t (&v)[16])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
        "%15}, [%16];"
        : Q4_W8(v, 0), Q4_W8(v, 8)
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_ld32x(uint32_t taddr, uint32_t (&v)[32])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
        "%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : Q4_W8(v, 0), Q4_W8(v, 8), Q4_W8(v, 16), Q4_W8(v, 24)
        : "r"(taddr)
        : "memory");
}
// Waits for this warp's tensor-memory loads; tied to the registers they fill,
// so that no use of v can be moved before it.
#define Q4_RW8(a, o) "+r"(a[o + 0]), "+r"(a[o + 1]), "+r"(a[o + 2]), "+r"(a[o + 3]), \
    "+r"(a[o + 4]), "+r"(a[o + 5]), "+r"(a[o + 6]), "+r"(a[o + 7])
__device__ __forceinline__ void tmem_wait_ld_of(uint32_t (&v)[16])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;" : Q4_RW8(v, 0), Q4_RW8(v, 8) : : "memory");
}
__device__ __forceinline__ void tmem_wait_ld_of(uint32_t (&v)[32])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : Q4_RW8(v, 0), Q4_RW8(v, 8), Q4_RW8(v, 16), Q4_RW8(v, 24)
                 :
                 : "memory");
}
#undef Q4_RW8
#undef Q4_R8
#undef Q4_W8

// C consecutive 32-bit columns (C = 16 or 32) of this warp's lanes.
template <int C>
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&v)[C])
{
    if constexpr (C == 16)
        tmem_ld16x(taddr, v);
    else
        tmem_ld32x(taddr, v);
}

}  // namespace q4
