/*
 * dma.h -- direct-to-LDS copies (buffer loads whose destination is LDS) and
 * the waits for them.  Internal, device code.
 */
#ifndef GEMM355_DMA_H
#define GEMM355_DMA_H

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <utility>

namespace g355 {

namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));

/* Buffer loads whose offset is past num_records return zero (and write zero
 * to LDS for the direct-to-LDS form): rows beyond M or N and K-chunks beyond
 * K are read through offset kOOB. */
constexpr uint32_t kNumRecords = 0x7FFFFF00u;
constexpr uint32_t kOOB = 0x80000000u;

/* The four dwords of a raw buffer resource: 48-bit base, stride 0,
 * num_records, and the gfx9-family word 3 (32-bit data format). */
__device__ __forceinline__ i32x4 rsrc_words(const void *base)
{
    const uint64_t a = (uint64_t)(uintptr_t)base;
    return i32x4{__builtin_amdgcn_readfirstlane((int)(uint32_t)a),
                 __builtin_amdgcn_readfirstlane((int)(uint32_t)(a >> 32) & 0xFFFF),
                 (int)kNumRecords, 0x00020000};
}

/* Compile-time unrolling: f(integral_constant<int, t>) for t = 0 .. N-1. */
template <int... T, class F>
__device__ __forceinline__ void unroll_seq(std::integer_sequence<int, T...>, F &&f)
{
    (f(std::integral_constant<int, T>{}), ...);
}
template <int N, class F>
__device__ __forceinline__ void unroll(F &&f)
{
    unroll_seq(std::make_integer_sequence<int, N>{}, static_cast<F &&>(f));
}

/* 32-bit LDS address of a __shared__ object. */
__device__ __forceinline__ uint32_t lds_addr(const uint8_t *p)
{
    return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) uint8_t *)p;
}

/* One direct-to-LDS copy: each lane fetches 16 bytes at voffset from the
 * buffer and the wavefront writes them to LDS at lds_base + OFF .. + 1023
 * (lane l at + 16 l).  Issued as inline assembly so that the compiler neither
 * waits for it before unrelated LDS reads nor counts it (completion is
 * awaited explicitly), and so that the LDS address is formed in M0 right at
 * the load from one base register and an immediate. */
template <int OFF>
__device__ __forceinline__ void dma16(const i32x4 &rsrc, uint32_t lds_base, uint32_t voffset)
{
    /* s_add writes SCC: declared clobbered, or the compiler could keep a
     * comparison result in SCC across this statement */
    int m0_out;
    asm volatile("s_add_u32 m0, %2, %4\n\tbuffer_load_dwordx4 %1, %3, 0 offen lds"
                 : "={m0}"(m0_out)
                 : "v"(voffset), "s"(lds_base), "s"(rsrc), "n"(OFF)
                 : "memory", "scc");
    (void)m0_out;
}

/* One direct-to-LDS dword copy: lane l fetches 4 bytes at voffset and the
 * wavefront writes them to LDS at lds_addr + 4 l (256 bytes). */
__device__ __forceinline__ void dma4(const i32x4 &rsrc, uint32_t lds_addr_, uint32_t voffset)
{
    int m0_out;
    asm volatile("s_mov_b32 m0, %2\n\tbuffer_load_dword %1, %3, 0 offen lds"
                 : "={m0}"(m0_out)
                 : "v"(voffset), "s"(lds_addr_), "s"(rsrc)
                 : "memory");
    (void)m0_out;
}

/* The same from 64-bit addresses: lane l fetches 16 bytes (4, 1) at its own
 * address, written to LDS at lds_base + 16 l (+ 4 l; a byte as a dword).  A
 * global load to LDS may not follow a write of M0 at once. */
__device__ __forceinline__ void dma_global16(uint32_t lds_base, const void *ptr)
{
    int m0_out;
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off"
                 : "={m0}"(m0_out)
                 : "v"(ptr), "s"(lds_base)
                 : "memory");
    (void)m0_out;
}
__device__ __forceinline__ void dma_global4(uint32_t lds_base, const void *ptr)
{
    int m0_out;
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dword %1, off"
                 : "={m0}"(m0_out)
                 : "v"(ptr), "s"(lds_base)
                 : "memory");
    (void)m0_out;
}
__device__ __forceinline__ void dma_global1(uint32_t lds_base, const void *ptr)
{
    int m0_out;
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_ubyte %1, off"
                 : "={m0}"(m0_out)
                 : "v"(ptr), "s"(lds_base)
                 : "memory");
    (void)m0_out;
}

/* Wait until at most N vector-memory operations of this wave are
 * outstanding (loads complete in issue order). */
template <int N>
__device__ __forceinline__ void wait_vmcnt()
{
    static_assert(N >= 0 && N < 64, "vmcnt range");
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

} /* namespace */

} /* namespace g355 */

#endif
