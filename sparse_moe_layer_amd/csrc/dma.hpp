// Direct loads to LDS and the waits around them: what the kernels that stage their operands
// by hand share.
#pragma once
#include "common.hpp"

namespace moe {

// Immediates of s_waitcnt: until at most n of this wave's vector memory accesses (loads to LDS
// among them) are under way; the second also until none of its LDS accesses is.
constexpr int vmcnt_imm(int n) { return 0xF70 | (n & 15) | (((n >> 4) & 3) << 14); }
constexpr int vmcnt_lgkm0_imm(int n) { return vmcnt_imm(n) & ~0xF00; }

// The raw barrier with a compiler-level fence on both sides (the builtin itself does not order
// memory accesses for the compiler).  It does not wait for this wave's LDS accesses: a
// wait for them (vmcnt_lgkm0_imm) comes first wherever another wave overwrites what this one
// read, or reads what it wrote.
__device__ __forceinline__ void block_sync() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// The same once this wave's LDS accesses are done.
__device__ __forceinline__ void lds_sync() {
  __builtin_amdgcn_s_waitcnt(vmcnt_lgkm0_imm(63));
  block_sync();
}

constexpr int kBufferFlags = 0x00020000;    // raw (untyped) 32-bit buffer access
constexpr uint32_t kNowhere = 0xFFFFFFF0u;  // past every buffer: the load writes zeros to LDS

// A 16-byte direct load (global memory to LDS, no registers) from base + voff + soff (voff the
// lane's, soff the wave's, below 2^32 together); past `records` bytes it writes zeros.  The
// compiler counts buffer loads to LDS apart from LDS reads, so fragment reads keep partial LDS
// waits; with the global_load_lds form in flight it waits for every outstanding LDS operation
// before each matrix instruction that consumes a fragment.  once (a constant): non-temporal.
__device__ __forceinline__ void dma16(const void* base, uint32_t records, uint32_t voff, uint32_t soff, void* l,
                                      bool once = false) {
  const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, records, kBufferFlags);
  if (once) __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)l, 16, voff, soff, 0, 2);
  else __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)l, 16, voff, soff, 0, 0);
}

}  // namespace moe
