// Loads from memory straight to LDS.
#pragma once

#include "common.h"

namespace q4 {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void lds_void;

// Loads straight to LDS, 16 or 4 bytes per lane in lane order from LDS address
// `to` on.  Assembly, because around the builtin the compiler waits for every
// such load before any read of LDS, also of another stage; the kernels that use
// them wait by themselves (vmcnt, then a barrier).  Nothing is written to registers;
// the compiler puts `to` into m0 (a wait state before its use).  There is no
// memory clobber, which would bring those waits back: that LDS is not read before
// the load has ended, nor written while it is read, rests on the s_waitcnt and
// phase() (a barrier across which nothing moves) around it.
// The descriptor's check covers the sum of a lane's and the scalar offset and
// does not wrap (measured with both past it): what lies behind gives zeros.
__device__ __forceinline__ i32x4 rsrc_words(const void* base, uint32_t bytes) {
    const uint64_t b = reinterpret_cast<uintptr_t>(base);
    return i32x4{(int)(uint32_t)b, (int)(uint32_t)(b >> 32), (int)bytes, kBufferFlags};
}
__device__ __forceinline__ void to_lds16(i32x4 r, uint32_t off, uint32_t soff, uint32_t to) {
    asm volatile("s_nop 0\n\tbuffer_load_dwordx4 %0, %1, %2 offen lds" ::"v"(off), "s"(r), "s"(soff), "{m0}"(to));
}
__device__ __forceinline__ uint32_t lds_address(const uint8_t* p) { return (uint32_t)(uintptr_t)(lds_void*)p; }

// A barrier across which nothing moves; no wait is implied.
__device__ __forceinline__ void phase() {
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_barrier" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}

}  // namespace q4
