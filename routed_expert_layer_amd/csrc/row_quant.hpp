// Codes of a row (or of a part of one) in 8 bits with a scale.
#pragma once
#include "dev_common.hpp"

namespace moe {
namespace {

// What a row's codes are formed with, from the largest magnitude (as bits, so
// that infinities and NaN compare above every finite value). A code is
// rne(127 v / amax) exactly, without a branch (one for the values near a half
// costs more code than the rest together: 333 rows of 1280 took 6.5 us, 4.2
// so): the half that decides is c = floor(t) + 1/2 for t = 127 v / amax in
// fp32, on either side of an integer, and the side of 127 v - c amax moves it
// by a quarter before it is rounded. Both are scaled so that A = amax 2^B is in
// [2^32, 2^33): a difference that is not 0 is above a quarter then, and c A has
// 16 bits for bf16 v, so that its difference is rounded once; for fp32 v the
// part of c A below 24 bits is taken off too, behind a first difference that
// is exact wherever the sum's sign could depend on it (|t - c| < |t| / 127).
struct RowQuant {
  float amax, up, inv, k127, a32;
  __device__ __forceinline__ explicit RowQuant(uint32_t amax_bits) {
    amax = __uint_as_float(amax_bits);
    up = amax < 0x1p-80f ? 0x1p+100f : 1.f;  // a power of two that keeps 127 / amax and 2^B finite
    const float a = amax * up;
    const bool some = amax_bits - 1u < 0x7F800000u - 1u;  // else the codes are 0, or any: their scale is NaN
    const float b = __uint_as_float((286u - (__float_as_uint(a) >> 23)) << 23);
    inv = some ? 127.f / a : 0.f;
    k127 = some ? 127.f * b : 0.f;
    a32 = some ? a * b : 0.f;
  }
  // The scale: NaN for a row with an infinity or NaN (its products are then NaN), 0 for a row of zeros.
  __device__ __forceinline__ float scale() const {
    return __float_as_uint(amax) < 0x7F800000u ? amax / 127.f : __uint_as_float(0x7FC00000u);
  }
  // A word whose low byte is v's code.
  template <bool BF16>
  __device__ __forceinline__ uint32_t code(float v) const {
    v *= up;
    const float c = floorf(v * inv) + 0.5f, p = c * a32;
    float d = fmaf(v, k127, -p);
    if constexpr (!BF16) d -= fmaf(c, a32, -p);
    return __float_as_uint((c + __builtin_amdgcn_fmed3f(d, -0.25f, 0.25f)) + 12582912.f);  // 1.5 2^23
  }
  template <bool BF16>
  __device__ __forceinline__ uint32_t pack2(float a, float b) const {
    return __builtin_amdgcn_perm(code<BF16>(b), code<BF16>(a), 0x0c0c0400u);
  }
  template <bool BF16>
  __device__ __forceinline__ uint32_t pack4(float a, float b, float c, float d) const {
    return pack2<BF16>(a, b) | __builtin_amdgcn_perm(code<BF16>(d), code<BF16>(c), 0x04000c0cu);
  }
};

// bf16 of any value: a NaN stays one (f32_to_bf16 takes finite values).
__device__ __forceinline__ uint32_t bf16_bits(float f) {
  const uint32_t u = __float_as_uint(f);
  return isnan(f) ? (u >> 16 | 0x40u) : (uint32_t)f32_to_bf16(f);
}

}  // namespace
}  // namespace moe
