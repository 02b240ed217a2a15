// What the prefill GEMM kernels share: wait counts, direct-to-LDS loads and the super-tile shapes.
#pragma once
#include "dev_common.hpp"
#include "moe_kernels.hpp"

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

// Per expert, a super-tile is GM token tiles x GN weight tiles (GM*GN <= 32
// block slots): GM = the smallest power of two covering its token tiles, at
// most 8; GN = the largest power of two dividing the weight tiles that fits
// beside it. Super-tiles per expert: ceil(m tiles / GM) x (n tiles / GN).
// Returns that count for a group of `rows` rows (0 for none) and sets
// shape = GM | GN << 8. Host planner and device planner use the same rule.
__host__ __device__ inline int supertiles_of(int rows, int N, int tile_tokens, int& shape) {
  const int NTB = N / 256;
  int gn_div = 1;
  while (gn_div < 16 && NTB % (gn_div * 2) == 0) gn_div *= 2;
  const int mtiles = (rows + tile_tokens - 1) / tile_tokens;
  int GM = 8;
  while (GM > 1 && GM / 2 >= mtiles) GM /= 2;
  const int GN = (32 / GM) < gn_div ? 32 / GM : gn_div;
  shape = GM | (GN << 8);
  return rows > 0 ? (mtiles + GM - 1) / GM * (NTB / GN) : 0;
}

inline int supertile_blocks(int tot) { return (tot + 7) / 8 * 256; }  // 8 XCDs x 32 slots per round

}  // namespace
}  // namespace moe
