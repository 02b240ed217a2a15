// Rows of fp32 or bf16 in registers: N elements at a time, as fp32.
#pragma once
#include <type_traits>

#include "dev_common.hpp"

namespace moe {
namespace {

// Where the piece of N elements that begins at column c of a row of n is taken: the last one ends with the row, so that
// it is moved whole too; its first elements are then those of the piece before (the same values, written twice). Rows
// shorter than a piece begin at 0. (7754 tokens' sums of 6 rows of 219 bf16 values 7.5 us with a shorter last piece, 6.6
// so, their gradient 21.6 and 13.5, that of 4096 x 6 of 4095 120 and 95; copies are as fast with one, and have one.)
template <int N>
__device__ __forceinline__ int piece_start(int c, int n) {
  return min(c, max(n - N, 0));
}

template <bool BF16>
constexpr int kElem = BF16 ? 2 : 4;
template <bool BF16>
constexpr int kVecElems = 16 / kElem<BF16>;  // elements of 16 bytes

// N elements (8, 16 or 32 bytes) at any element of a row: global loads and stores of vectors need no more alignment than
// their elements on this GPU, so rows of odd lengths go in 16-byte pieces too, all but the last few elements. (With
// pieces of the widest size that divides the row instead, 7754 tokens x 6 rows of 219 bf16 values take 10.3 us to send out
// and 24.1 for the gradient, 7.0 and 13.5 so; 9949 rows of 2 x 1509 74.8 us through SwiGLU and back, 54 so.)
template <bool BF16, int N>
struct RowVec {
  using elem_t = std::conditional_t<BF16, uint16_t, uint32_t>;
  static constexpr int kWords = N * kElem<BF16> / 4;
  static_assert(N == 4 || N == 8, "a row's last piece goes in parts of four, two and one: up to seven elements");
  static constexpr int kPiece = kWords < 4 ? kWords : 4;  // words to a load
  typedef uint32_t piece_t __attribute__((ext_vector_type(kPiece), aligned(kElem<BF16>)));
  template <int M>  // M elements
  using part_t __attribute__((aligned(kElem<BF16>))) = uint32_t __attribute__((ext_vector_type(M * kElem<BF16> / 4)));
  uint32_t w[kWords];

  // `left` elements are left in the row: the ones past them are 0 and not read or written. STREAM: past the caches, for
  // rows that are read once.
  template <bool STREAM = false>
  __device__ __forceinline__ void load(const void* base, size_t elem, int left) {
    const elem_t* p = static_cast<const elem_t*>(base) + elem;
    if (left >= N) {
#pragma unroll
      for (int i = 0; i < kWords / kPiece; ++i) {
        const piece_t* q = reinterpret_cast<const piece_t*>(p) + i;
        piece_t v;
        if constexpr (STREAM) v = __builtin_nontemporal_load(q);
        else v = *q;
#pragma unroll
        for (int j = 0; j < kPiece; ++j) w[kPiece * i + j] = v[j];
      }
    } else {
      // four, two and one of them, wherever there are, moved to their places afterwards
      part_t<4> f = 0;
      part_t<2> t = 0;
      uint32_t o = 0;
      if (N > 4 && left >= 4) f = *reinterpret_cast<const part_t<4>*>(p);
      if (left & 2) t = *reinterpret_cast<const part_t<2>*>(p + (left & 4));
      if (left & 1) o = p[left & 6];
      constexpr int k2 = kElem<BF16> / 2;  // words of two elements
      uint32_t v[2 * k2] = {};
      if (left & 2) {
#pragma unroll
        for (int i = 0; i < k2; ++i) v[i] = t[i];
        v[k2] = o;
      } else {
        v[0] = o;
      }
#pragma unroll
      for (int i = 0; i < kWords; ++i) w[i] = 0;
      const bool four = N > 4 && left >= 4;
#pragma unroll
      for (int i = 0; i < 2 * k2; ++i) {
        w[i] = four ? f[i] : v[i];
        if constexpr (N > 4) w[2 * k2 + i] = four ? v[i] : 0;
      }
    }
  }
  // STREAM: past the caches, for rows that the experts' products read next: dispatching 4096 tokens to 6 of
  // 64 experts (201 MB of rows) takes 38 us so and 47 through the caches, where the end of the kernel waits for what they
  // hold, and with the product behind it (which is bound by its arithmetic) 847 and 854; 256 tokens 333 and 337.
  template <bool STREAM = false>
  __device__ __forceinline__ void store(void* base, size_t elem, int left) const {
    elem_t* p = static_cast<elem_t*>(base) + elem;
    if (left >= N) {
#pragma unroll
      for (int i = 0; i < kWords / kPiece; ++i) {
        piece_t v;
#pragma unroll
        for (int j = 0; j < kPiece; ++j) v[j] = w[kPiece * i + j];
        piece_t* q = reinterpret_cast<piece_t*>(p) + i;
        if constexpr (STREAM) __builtin_nontemporal_store(v, q);
        else *q = v;
      }
    } else {
      constexpr int k2 = kElem<BF16> / 2;  // words of two elements
      uint32_t v[2 * k2];
      const bool four = N > 4 && left >= 4;
      part_t<4> f;
      part_t<2> t;
#pragma unroll
      for (int i = 0; i < 2 * k2; ++i) {
        f[i] = w[i];
        v[i] = w[i];
        if constexpr (N > 4) v[i] = four ? w[2 * k2 + i] : w[i];
      }
#pragma unroll
      for (int i = 0; i < k2; ++i) t[i] = v[i];
      if (four) *reinterpret_cast<part_t<4>*>(p) = f;
      if (left & 2) *reinterpret_cast<part_t<2>*>(p + (left & 4)) = t;
      if (left & 1) p[left & 6] = (elem_t)((left & 2) ? v[k2] : v[0]);
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
    } else {
      typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
#pragma unroll
      for (int i = 0; i < N / 2; ++i)
        w[i] = __builtin_bit_cast(uint32_t, bf16x2_t{(__bf16)f[2 * i], (__bf16)f[2 * i + 1]});
    }
  }
};

}  // namespace
}  // namespace moe
