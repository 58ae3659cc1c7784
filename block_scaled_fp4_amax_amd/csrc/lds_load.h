// lds_load.h -- loads from memory straight to LDS (device only).
#pragma once

#include "fp4q_device.h"

namespace fp4q {

// Loads of 16 bytes a lane straight to LDS at a wave-uniform base (lane l's go to base
// + 16 l), from per-lane addresses or through a descriptor.  They are written out, with the
// waits below, because the compiler's own waits cannot tell stages apart and would
// wait for every outstanding load before any read of LDS.  No other instruction
// here reads m0, so the reserved-register clobber warning is silenced.  The bytes are read
// once (non-temporal: 4 x 131072 cached keys 82 -> 71.5 us) unless a name says otherwise.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void lds_load(const void* p, uint32_t base)
{
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off nt" : : "v"(p), "s"(base) : "memory", "m0");
}

__device__ __forceinline__ void lds_load(rsrc_t r, uint32_t off, uint32_t base, uint32_t all = 0)
{
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %2, %3 offen nt lds" :
                 : "v"(off), "s"(base), "s"(r), "s"(all)
                 : "memory", "m0");
}

// Four bytes a lane, lane l's to base + 4 l.
__device__ __forceinline__ void lds_load4(rsrc_t r, uint32_t off, uint32_t base, uint32_t all = 0)
{
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tbuffer_load_dword %0, %2, %3 offen lds" :
                 : "v"(off), "s"(base), "s"(r), "s"(all)
                 : "memory", "m0");
}

// One byte a lane, lane l's to the word at base + 4 l.
__device__ __forceinline__ void lds_load1(rsrc_t r, uint32_t off, uint32_t base, uint32_t all = 0)
{
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tbuffer_load_ubyte %0, %2, %3 offen lds" :
                 : "v"(off), "s"(base), "s"(r), "s"(all)
                 : "memory", "m0");
}

// Two bytes a lane (2-byte aligned), lane l's to the word at base + 4 l.
__device__ __forceinline__ void lds_load2(rsrc_t r, uint32_t off, uint32_t base, uint32_t all = 0)
{
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tbuffer_load_ushort %0, %2, %3 offen lds" :
                 : "v"(off), "s"(base), "s"(r), "s"(all)
                 : "memory", "m0");
}

// Sixteen bytes a lane through the caches' ordinary policy, for bytes that other workgroups read again.
__device__ __forceinline__ void lds_load_kept(rsrc_t r, uint32_t off, uint32_t base, uint32_t all = 0)
{
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %2, %3 offen lds" :
                 : "v"(off), "s"(base), "s"(r), "s"(all)
                 : "memory", "m0");
}
#pragma clang diagnostic pop

// Waits until at most N vector-memory operations of the wave are outstanding; no read of
// LDS moves above it.
template <int N>
__device__ __forceinline__ void wait_loads()
{
    static_assert(N >= 0 && N < 64, "the counter holds 63");
    asm volatile("s_waitcnt vmcnt(%0)" : : "i"(N) : "memory");
}

// Waits for the wave's own reads of LDS, before a load overwrites the places that they read: the two are
// not ordered with each other.
__device__ __forceinline__ void wait_reads()
{
    asm volatile("s_waitcnt lgkmcnt(0)" : : : "memory");
}

typedef __attribute__((address_space(3))) unsigned char lds_t;

__device__ __forceinline__ uint32_t lds_address(const lds_t* p)
{
    return __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)p);
}

}  // namespace fp4q
