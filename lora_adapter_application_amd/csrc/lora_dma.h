// lora_dma.h -- direct-to-LDS loads of the kernels that stage operands in LDS.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace lora {

// One global_load_lds_dwordx4 with a wave-uniform 64-bit base and a 32-bit
// byte offset per lane, written as asm so that the compiler does not track it:
// its own tracking cannot tell the stages apart and would wait for every load
// in flight before each LDS read.  The waits for these loads are explicit
// (s_waitcnt vmcnt in the kernel); lane l writes the 16 bytes at LDS offset
// 16 l of the instruction's 1 KB, whose wave-uniform address is lds.  m0 is
// not named as clobbered: the compiler reserves it and sets it before each of
// its own uses.
__device__ __forceinline__ void dma16_off(const void *base, uint32_t off, uint32_t lds)
{
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(off), "s"(base), "s"(lds)
                 : "memory");
}

// The same with 4 bytes a lane: 256 bytes, lane l at LDS offset 4 l.
__device__ __forceinline__ void dma4_off(const void *base, uint32_t off, uint32_t lds)
{
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dword %0, %1" ::"v"(off), "s"(base), "s"(lds)
                 : "memory");
}

}  // namespace lora
