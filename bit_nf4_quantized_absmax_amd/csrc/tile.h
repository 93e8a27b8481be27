// Helpers of the MX4 kernels: wait counts, the operand tiles' swizzle and the
// workgroup barrier (matmul.hip, whose sources a recorded profile covers, has its
// own), block scales, DMA from a uniform base.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace qlora {

// s_waitcnt immediate (gfx9 encoding: vmcnt bits 3:0 and 15:14, expcnt 6:4,
// lgkmcnt 11:8); vm = 63 / lgkm = 15 do not wait.
constexpr int wait_imm(int vm, int lgkm) { return (vm & 15) | ((vm >> 4) << 14) | 0x70 | ((lgkm & 15) << 8); }

// 128-byte rows (64 bf16, 256 MX4 codes): 16-byte chunk c of row r at 16-byte position c ^ f(r).
__device__ __forceinline__ int swz128(int row, int chunk) {
  return row * 128 + 16 * (chunk ^ ((row & 7) ^ ((row >> 3) & 1)));
}
// Workgroup barrier without a memory-model fence (a fence would also wait for
// every outstanding DMA and prefetch): waits per kWait, then s_barrier.  The
// signal fences stop the compiler from moving memory accesses across it and
// the scheduling barriers keep each side its own scheduling region.
template <int kWait>
__device__ __forceinline__ void raw_barrier() {
  __builtin_amdgcn_sched_barrier(0);
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
  __builtin_amdgcn_s_waitcnt(kWait);
  __builtin_amdgcn_s_barrier();
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
  __builtin_amdgcn_sched_barrier(0);
}

// The scale 2^(byte - 127) of an MX4 block as the fp32 operand of the E2M1
// conversions (byte 0 is the subnormal 2^-127).
__device__ __forceinline__ float mx4_scale(uint32_t byte) {
  return __uint_as_float(byte == 0u ? 0x00400000u : byte << 23);
}

// dma16 of lds_dma.h from a uniform base and a 32-bit byte offset a lane; 4 bytes a lane.
__device__ __forceinline__ void dma16(const void *base, uint32_t off, uint32_t dst) {
  asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(off), "s"(base), "{m0}"(dst) : "memory");
}
__device__ __forceinline__ void dma4(const void *base, uint32_t off, uint32_t dst) {
  asm volatile("s_nop 0\n\tglobal_load_lds_dword %0, %1" ::"v"(off), "s"(base), "{m0}"(dst) : "memory");
}

}  // namespace qlora
