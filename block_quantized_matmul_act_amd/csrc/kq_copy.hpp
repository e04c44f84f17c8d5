// kq_copy.hpp -- copies from memory to LDS without registers (gfx950 only).
//
// 16 bytes of a lane, from base + voff or from `from`, to lds + 16 * lane.  Written as an
// instruction of our own: the compiler would make every read of LDS that follows wait
// for the newest copy.  The wave waits for its copies itself (arrived), before it reads
// what they brought or before the barrier after which others do.  The loads have no
// output registers; m0 is set right before each and used for nothing else.
#pragma once

#include "kq_device.hpp"

namespace kq {

__device__ __forceinline__ void copy16(uint32_t lds, const void *base, uint32_t voff) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(lds), "v"(voff), "s"(base) : "memory");
}
__device__ __forceinline__ void copy16(uint32_t lds, const void *from) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(lds), "v"(from) : "memory");
}
// All copies of the wave but the LEFT newest have arrived.
template <int LEFT>
__device__ __forceinline__ void arrived() {
    asm volatile("s_waitcnt vmcnt(%0)" ::"i"(LEFT) : "memory");
}
// The wave's reads of LDS are done: their places may be filled again.
__device__ __forceinline__ void reads_done() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

__device__ __forceinline__ uint32_t lds_offset(const void *p) {
    return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void *)p;
}

}  // namespace kq
