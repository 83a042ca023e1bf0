// Copies from global memory straight into LDS, and the waits around them: what the
// matrix products share.  The copies are issued from inline asm, so that the compiler,
// which cannot tell them apart from the buffer being read, does not drain them before
// every LDS read; their completion is awaited explicitly before the barrier that
// publishes the buffer.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mxq {

// M0 is a register the compiler reserves (it may hold a live value of its own
// across this statement, e.g. for an LDS instruction it emitted), so the copy
// saves it into an SGPR of its own, points it at the LDS destination, and puts
// the saved value back before the statement ends.  The load takes M0 when it
// is issued, so the restore right behind it does not change the copy.  The
// build treats -Winline-asm as an error, so a reserved register can never sit
// on a clobber list unnoticed.
__device__ __forceinline__ void dma16(const uint8_t *g, const uint8_t *l)
{
    const uint32_t la = (uint32_t)(uintptr_t)((__attribute__((address_space(3))) const uint8_t *)l);
    uint32_t saved;
    asm volatile("s_mov_b32 %0, m0\n\t"
                 "s_mov_b32 m0, %2\n\t"
                 "s_nop 0\n\t"
                 "global_load_lds_dwordx4 %1, off\n\t"
                 "s_mov_b32 m0, %0"
                 : "=&s"(saved)
                 : "v"(g), "s"(__builtin_amdgcn_readfirstlane(la))
                 : "memory");
}

// The same copy with the global address split into a wave-uniform 64-bit base
// (scalar registers) and a 32-bit per-lane offset, so a step's new base is
// scalar arithmetic only.
__device__ __forceinline__ void dma16_so(const uint8_t *base, uint32_t off, const uint8_t *l)
{
    const uint32_t la = (uint32_t)(uintptr_t)((__attribute__((address_space(3))) const uint8_t *)l);
    uint32_t saved;
    asm volatile("s_mov_b32 %0, m0\n\t"
                 "s_mov_b32 m0, %3\n\t"
                 "s_nop 0\n\t"
                 "global_load_lds_dwordx4 %1, %2\n\t"
                 "s_mov_b32 m0, %0"
                 : "=&s"(saved)
                 : "v"(off), "s"(base), "s"(__builtin_amdgcn_readfirstlane(la))
                 : "memory");
}

__device__ __forceinline__ uint32_t lds_address(const void *l)
{
    return (uint32_t)(uintptr_t)((__attribute__((address_space(3))) const void *)l);
}

// The same to an LDS address held in a scalar register.  ONCE: what is not read again leaves
// the caches to what is.
template <bool ONCE>
__device__ __forceinline__ void copy16(const uint8_t *base, uint32_t off, uint32_t lds)
{
    uint32_t saved;
    if constexpr (ONCE)
        asm volatile("s_mov_b32 %0, m0\n\t"
                     "s_mov_b32 m0, %3\n\t"
                     "s_nop 0\n\t"
                     "global_load_lds_dwordx4 %1, %2 nt\n\t"
                     "s_mov_b32 m0, %0"
                     : "=&s"(saved)
                     : "v"(off), "s"(base), "s"(lds)
                     : "memory");
    else
        asm volatile("s_mov_b32 %0, m0\n\t"
                     "s_mov_b32 m0, %3\n\t"
                     "s_nop 0\n\t"
                     "global_load_lds_dwordx4 %1, %2\n\t"
                     "s_mov_b32 m0, %0"
                     : "=&s"(saved)
                     : "v"(off), "s"(base), "s"(lds)
                     : "memory");
}

// The same from an address of each lane's own.
__device__ __forceinline__ void copy16(const uint8_t *from, uint32_t lds)
{
    uint32_t saved;
    asm volatile("s_mov_b32 %0, m0\n\t"
                 "s_mov_b32 m0, %2\n\t"
                 "s_nop 0\n\t"
                 "global_load_lds_dwordx4 %1, off\n\t"
                 "s_mov_b32 m0, %0"
                 : "=&s"(saved)
                 : "v"(from), "s"(lds)
                 : "memory");
}

__device__ __forceinline__ void wait_all_vm()
{
    __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0), expcnt/lgkmcnt untouched
}

__device__ __forceinline__ void barrier_no_fence()
{
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

}  // namespace mxq
