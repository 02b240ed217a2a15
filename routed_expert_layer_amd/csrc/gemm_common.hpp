// What the prefill GEMM kernels share: wait counts and direct-to-LDS loads.
#pragma once
#include "dev_common.hpp"

namespace moe {
namespace {

// s_waitcnt immediate that waits for vmcnt <= n only (gfx9 encoding: vmcnt
// bits 3:0 and 15:14, expcnt 6:4, lgkmcnt 11:8 at their maxima).
constexpr int vmcnt_only(int n) { return (n & 15) | ((n >> 4) << 14) | (7 << 4) | (15 << 8); }
// ... and for lgkmcnt <= n only (vmcnt and expcnt at their maxima).
constexpr int lgkmcnt_only(int n) { return 15 | (3 << 14) | (7 << 4) | ((n & 15) << 8); }

// One 16-byte chunk per lane from base + off (a wave-uniform base, a 32-bit
// lane offset) straight into the wave's 1 KiB at `lds` (lane l at lds + 16 l),
// through a raw buffer resource (dword 3 = 0x00020000 for byte-addressed
// loads on gfx950, no bounds check).
__device__ __forceinline__ void buffer_load_lds16(const void* base, uint32_t off, char* lds) {
  const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, -1, 0x00020000);
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)lds, 16, off, 0, 0, 0);
}

}  // namespace
}  // namespace moe
