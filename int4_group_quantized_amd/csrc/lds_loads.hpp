// Loads that go straight from memory into LDS, and the waits for them.
#pragma once

#include "q4_device.hpp"

namespace q4 {

// 16 bytes per lane from memory into LDS: lane i's to byte `to` + 16 i.  In
// assembly because the compiler, which sees that images follow each other in
// one array, would let every LDS read wait for all such loads under way; the
// waits are wait_and_meet's.  The instruction has no destination register.  m0, a
// reserved register, cannot be declared as overwritten; nothing else in the kernels
// that call this uses it, which tests/test_attention_assembly.py and
// tests/test_latent_assembly.py check.
// First form: from base + the lane's offset in bytes, base the same in all lanes.
// A vector instruction may have written base just before (a value read from a
// lane, a spilled one too), and the compiler does not look into the assembly: the
// five wait states that a memory operation then needs are the move's and the
// no-operation's.  They cost 0.3% of 8,192 prompt tokens' time, 1.6% at dim 64.
__device__ __forceinline__ void load_lds(const uint16_t* base, uint32_t offset, uint32_t to) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\tglobal_load_lds_dwordx4 %1, %2"
                 :
                 : "s"(to), "v"(offset), "s"(base)
                 : "memory");
}
// A pointer that is the same in all lanes, in scalar registers.
__device__ __forceinline__ const uint16_t* uniform(const uint16_t* p) {
    const uint64_t v = (uint64_t)p;
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v), hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
    return (const uint16_t*)((uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ void load_lds(const uint16_t* p, uint32_t to) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" : : "s"(to), "v"(p) : "memory");
}

// Waits until at most NEWER of this wave's vector memory operations (which
// complete in order) and none of its LDS operations are under way, then for the
// workgroup.
template <int NEWER>
__device__ __forceinline__ void wait_for_loads() {
    static_assert(NEWER < 64, "the counter has six bits");
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt((NEWER & 15) | 0x70 | (NEWER >> 4) << 14);
    asm volatile("" ::: "memory");
}
template <int NEWER>
__device__ __forceinline__ void wait_and_meet() {
    wait_for_loads<NEWER>();
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// The same for LDS operations only.
__device__ __forceinline__ void lds_meet() {
    asm volatile("" ::: "memory");
    lds_barrier();
    asm volatile("" ::: "memory");
}

}  // namespace q4
