// zccl_tcgen05.cuh -- PTX wrappers for the fifth-generation tensor cores:
// tensor-memory allocation and loads, the e4m3 matrix instruction with its
// descriptors, and two-dimensional TMA loads.
#pragma once

#include <cstdint>
#include <cuda.h>

#include "zccl_common.cuh"

namespace zccl {

// Tensor memory: `columns` (a power of two, 32..512) for the whole CTA, by one
// warp; the address is written to shared memory.
__device__ __forceinline__ void tmem_alloc(uint32_t* dst, uint32_t columns)
{
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(dst)), "r"(columns)
                 : "memory");
}
__device__ __forceinline__ void tmem_release_permit()
{
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t columns)
{
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(columns) : "memory");
}

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// A K-major operand tile in shared memory, rows of 128 bytes, 128-byte
// swizzle: start address, 1024 bytes between groups of 8 rows.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr)
{
    return (uint64_t)((addr & 0x3FFFFu) >> 4) | (1ull << 16) | ((uint64_t)(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}

// Instruction descriptor: fp32 accumulator, e4m3 operands, both K-major.
__host__ __device__ constexpr uint32_t instr_desc(uint32_t m, uint32_t n) { return (1u << 4) | ((n >> 3) << 17) | ((m >> 4) << 24); }

// d = a b over a block of 128 values of the reduction axis (four instructions of
// 32, 32 bytes apart in the swizzled rows), then arrivals on two barriers when
// they are done.  A whole warp calls it, so that its operands stay in uniform registers;
// one elected lane issues.
__device__ __forceinline__ void mma_block_e4m3(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint64_t* bar0,
                                               uint64_t* bar1)
{
    asm volatile(
        "{\n .reg .pred one, add, set;\n .reg .b64 a1, b1, a2, b2, a3, b3;\n"
        " elect.sync _|one, 0xFFFFFFFF;\n setp.eq.u32 add, 0, 0;\n setp.ne.u32 set, 0, 0;\n"
        " add.u64 a1, %1, 2;\n add.u64 b1, %2, 2;\n add.u64 a2, %1, 4;\n add.u64 b2, %2, 4;\n"
        " add.u64 a3, %1, 6;\n add.u64 b3, %2, 6;\n"
        " @one tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, set;\n"
        " @one tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a1, b1, %3, add;\n"
        " @one tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a2, b2, %3, add;\n"
        " @one tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a3, b3, %3, add;\n"
        " @one tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%4];\n"
        " @one tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%5];\n}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(smem_addr(bar0)), "r"(smem_addr(bar1))
        : "memory");
}

// Arrives on `bar` when the matrix instructions this thread issued so far are done.
__device__ __forceinline__ void mma_commit(uint64_t* bar)
{
    asm volatile(
        "{\n .reg .pred one;\n elect.sync _|one, 0xFFFFFFFF;\n"
        " @one tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}" ::"r"(smem_addr(bar))
        : "memory");
}

// 32 columns of the warp's 32 lanes of tensor memory: lane l, column i in r[i].
__device__ __forceinline__ void tmem_load32(uint32_t addr, uint32_t (&r)[32])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
          "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]),
          "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]),
          "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr));
}

// Waits for this thread's tensor-memory loads.  The registers pass through, so
// that no use of them can move above the wait.
__device__ __forceinline__ void tmem_wait32(uint32_t (&r)[32])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                 "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]),
                 "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]),
                 "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
                 :
                 : "memory");
}

// Two fp32 values in an instruction, each rounded on its own.  At half the rate
// of the single ones they do no more in a second, but they leave every other
// issue slot to the warps that keep the tensor cores fed.
__device__ __forceinline__ void fma2(float& c0, float& c1, float a0, float a1, float b0, float b1)
{
    asm("{\n .reg .b64 a, b, c;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n mov.b64 c, {%0, %1};\n"
        " fma.rn.f32x2 c, a, b, c;\n mov.b64 {%0, %1}, c;\n}"
        : "+f"(c0), "+f"(c1)
        : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}
__device__ __forceinline__ float2 mul2(float a0, float a1, float b)
{
    float2 d;
    asm("{\n .reg .b64 a, b, c;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %4};\n mul.rn.f32x2 c, a, b;\n mov.b64 {%0, %1}, c;\n}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a0), "f"(a1), "f"(b));
    return d;
}

// A box of a two-dimensional tensor map to shared memory, completing on `bar`.
__device__ __forceinline__ void tma_load_2d(void* dst, const CUtensorMap* map, int32_t x, int32_t y, uint64_t* bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(
            smem_addr(dst)),
        "l"(map), "r"(smem_addr(bar)), "r"(x), "r"(y)
        : "memory");
}

// A box of shared memory to a two-dimensional tensor map (bulk-group completion).
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, const void* src, int32_t x, int32_t y)
{
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(map),
                 "r"(smem_addr(src)), "r"(x), "r"(y)
                 : "memory");
}

template <int kRegs>
__device__ __forceinline__ void regs_fewer() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs)); }
template <int kRegs>
__device__ __forceinline__ void regs_more() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs)); }

}  // namespace zccl
