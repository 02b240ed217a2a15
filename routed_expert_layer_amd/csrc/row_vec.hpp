// Rows of fp32 or bf16 in registers: N elements at a time, as fp32.
#pragma once
#include <initializer_list>
#include <utility>

#include "dev_common.hpp"

namespace moe {
namespace {

template <bool BF16>
constexpr int kElem = BF16 ? 2 : 4;

// N elements at p (aligned to their size, or to 16 bytes where that is less).
template <bool BF16, int N>
struct RowVec {
  static constexpr int kBytes = N * kElem<BF16>;
  static constexpr int kWords = kBytes < 4 ? 1 : kBytes / 4;
  uint32_t w[kWords];

  // STREAM: past the caches, for rows that are read once.
  template <bool STREAM = false>
  __device__ __forceinline__ void load(const void* base, size_t elem) {
    const char* p = static_cast<const char*>(base) + elem * kElem<BF16>;
    if constexpr (kBytes >= 16) {
#pragma unroll
      for (int i = 0; i < kBytes / 16; ++i) {
        const u32x4_t v = STREAM ? ld16_nt(p + 16 * i) : ld16(p + 16 * i);
#pragma unroll
        for (int j = 0; j < 4; ++j) w[4 * i + j] = v[j];
      }
    } else if constexpr (kBytes == 8) {
      const u32x2_t v = *reinterpret_cast<const u32x2_t*>(p);
      w[0] = v[0];
      w[1] = v[1];
    } else if constexpr (kBytes == 4) {
      w[0] = *reinterpret_cast<const uint32_t*>(p);
    } else {
      w[0] = *reinterpret_cast<const uint16_t*>(p);
    }
  }
  // STREAM: past the caches, for rows that the experts' products read next: dispatching 4096 tokens to 6 of 64 experts
  // (201 MB of rows) takes 38 us so and 47 through the caches, where the end of the kernel waits for what they hold, and
  // with the product behind it (which is bound by its arithmetic) 847 and 854; 256 tokens 333 and 337.
  template <bool STREAM = false>
  __device__ __forceinline__ void store(void* base, size_t elem) const {
    char* p = static_cast<char*>(base) + elem * kElem<BF16>;
    if constexpr (kBytes >= 16) {
#pragma unroll
      for (int i = 0; i < kBytes / 16; ++i) {
        const u32x4_t v{w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]};
        if constexpr (STREAM) __builtin_nontemporal_store(v, reinterpret_cast<u32x4_t*>(p) + i);
        else reinterpret_cast<u32x4_t*>(p)[i] = v;
      }
    } else if constexpr (kBytes == 8) {
      *reinterpret_cast<u32x2_t*>(p) = u32x2_t{w[0], w[1]};
    } else if constexpr (kBytes == 4) {
      *reinterpret_cast<uint32_t*>(p) = w[0];
    } else {
      *reinterpret_cast<uint16_t*>(p) = (uint16_t)w[0];
    }
  }
  __device__ __forceinline__ float get(int i) const {
    if constexpr (!BF16) return __uint_as_float(w[i]);
    else return __uint_as_float((i & 1) ? (w[i >> 1] & 0xFFFF0000u) : (w[i >> 1] << 16));
  }
  // Rounded to nearest even; a NaN stays one.
  __device__ __forceinline__ void set(const float (&f)[N]) {
    if constexpr (!BF16) {
#pragma unroll
      for (int i = 0; i < N; ++i) w[i] = __float_as_uint(f[i]);
    } else if constexpr (N == 1) {
      w[0] = __builtin_bit_cast(uint16_t, (__bf16)f[0]);
    } else {
      typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
#pragma unroll
      for (int i = 0; i < N / 2; ++i)
        w[i] = __builtin_bit_cast(uint32_t, bf16x2_t{(__bf16)f[2 * i], (__bf16)f[2 * i + 1]});
    }
  }
};

// Elements a thread takes at a time of rows of `len` elements: the most (8 of
// bf16, 4 of fp32) that divide the row and that every buffer is aligned for.
// Buffers come with their element's bytes.
inline int row_vec_elems(size_t len, int most, std::initializer_list<std::pair<const void*, int>> bufs) {
  for (int n = most; n > 1; n >>= 1) {
    bool ok = len % n == 0;
    for (const auto& b : bufs) {
      const size_t a = (size_t)n * b.second < 16 ? (size_t)n * b.second : 16;
      ok = ok && (reinterpret_cast<uintptr_t>(b.first) % a) == 0;
    }
    if (ok) return n;
  }
  return 1;
}

}  // namespace
}  // namespace moe
