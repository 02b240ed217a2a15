// SwiGLU whose inputs are kept in 8 bits, and its backward pass from them.
//
//   g = gu[r, :I], u = gu[r, I:],  s(g) = 1 / (1 + e^-g),  h = g s(g) u
//   kept, for 128 columns of g or u at a time:  scale = max|v| / 127,  code = rne(127 v / max|v|)
//   backward, from g^, u^ = code * scale:
//     dg = dh u^ s (1 + g^ (1 - s)),  du = dh g^ s,  h^ = g^ s u^
//
// Sixteen lanes take 128 columns of g and the same of u, eight of each a lane,
// so a scale is one reduction over 16 lanes and every byte is moved once.
// Bytes bound both passes: 98304 bf16 rows of 2 x 2048 take 636 us, 3.65 GB at
// 5.7 TB/s (a copy reaches 4.9).
#include "dev_common.hpp"
#include "moe_kernels.hpp"
#include "row_quant.hpp"
#include "row_vec.hpp"

namespace moe {
namespace {

constexpr int kKeptGroup = 128;  // columns that share a scale
constexpr int kKeptLanes = 16, kKeptCols = 8;

// 1 / (1 + e^-g) and 1 - it, neither by a difference: both keep their last bits (a NaN stays one). For bf16 results by
// the hardware's exponential and reciprocal, a step of 2^-23 each and 1.5 |g| half steps from the exponent's argument
// (below 2^-8 by far): 98304 rows of 2 x 2048 take 636 us for both passes so, 708 with expf and a
// division.
template <bool FAST>
struct Sigmoid {
  float s, t;
  __device__ __forceinline__ explicit Sigmoid(float g) {
    const float e = FAST ? __expf(-fabsf(g)) : expf(-fabsf(g));
    const float r = FAST ? __builtin_amdgcn_rcpf(1.f + e) : 1.f / (1.f + e);
    s = g >= 0.f ? r : e * r;
    t = g >= 0.f ? e * r : r;
  }
};

// Where a thread works: a row and up to eight columns from c0 on, of a group of 128.
struct KeptAt {
  int64_t row;
  int group, c0, left;  // left: columns of g (and u) from c0 on, 0 for a thread past them
  bool on;
};

__device__ __forceinline__ KeptAt kept_at(int64_t rows, int I, int groups) {
  const int64_t q = ((int64_t)blockIdx.x * 256 + threadIdx.x) / kKeptLanes;
  KeptAt a;
  a.row = q / groups;
  a.group = (int)(q % groups);
  a.c0 = a.group * kKeptGroup + ((int)threadIdx.x & (kKeptLanes - 1)) * kKeptCols;
  a.on = a.row < rows;
  a.left = a.on ? max(0, I - a.c0) : 0;
  return a;
}

template <bool BF16>
__device__ __forceinline__ void load8(const void* p, size_t base, const KeptAt& a, float (&f)[kKeptCols]) {
  RowVec<BF16, kKeptCols> v;
  v.load(p, base + a.c0, a.left);
#pragma unroll
  for (int i = 0; i < kKeptCols; ++i) f[i] = v.get(i);
}

template <bool BF16>
__device__ __forceinline__ void store8(void* p, size_t base, const KeptAt& a, const float (&f)[kKeptCols]) {
  RowVec<BF16, kKeptCols> v;
  v.set(f);
  v.template store<true>(p, base + a.c0, a.left);
}

typedef uint32_t codes_t __attribute__((ext_vector_type(2), aligned(1)));  // eight codes at any byte

__device__ __forceinline__ uint32_t max16(uint32_t v) {
#pragma unroll
  for (int d = kKeptLanes / 2; d > 0; d >>= 1) v = max(v, (uint32_t)__shfl_xor((int)v, d, kKeptLanes));
  return v;
}

template <bool BF16>
__device__ __forceinline__ void keep8(const float (&f)[kKeptCols], const KeptAt& a, int8_t* codes, size_t base,
                                      float* scale) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < kKeptCols; ++i) m = max(m, __float_as_uint(f[i]) & 0x7FFFFFFFu);
  const RowQuant q(max16(m));
  if (!a.on) return;
  if ((threadIdx.x & (kKeptLanes - 1)) == 0) *scale = q.scale();
  const codes_t v{q.pack4<BF16>(f[0], f[1], f[2], f[3]), q.pack4<BF16>(f[4], f[5], f[6], f[7])};
  int8_t* p = codes + base + a.c0;
  if (a.left >= kKeptCols) {
    *reinterpret_cast<codes_t*>(p) = v;
  } else {
#pragma unroll
    for (int i = 0; i < kKeptCols - 1; ++i)
      if (i < a.left) p[i] = (int8_t)(v[i >> 2] >> (8 * (i & 3)));
  }
}

template <bool BF16>
__global__ __launch_bounds__(256) void swiglu_save_kernel(const void* __restrict__ gu, int64_t rows,
                                                          const int32_t* __restrict__ n_rows, int I, int groups,
                                                          void* __restrict__ h, int8_t* __restrict__ codes,
                                                          float* __restrict__ scales) {
  if (n_rows) rows = min(rows, (int64_t)*n_rows);
  const KeptAt a = kept_at(rows, I, groups);  // a thread past the rows stays for the reductions
  const size_t r = (size_t)a.row * 2 * I;
  float g[kKeptCols], u[kKeptCols], f[kKeptCols];
  load8<BF16>(gu, r, a, g);
  load8<BF16>(gu, r + I, a, u);
#pragma unroll
  for (int i = 0; i < kKeptCols; ++i) f[i] = g[i] * Sigmoid<BF16>(g[i]).s * u[i];
  store8<BF16>(h, (size_t)a.row * I, a, f);
  float* sc = scales + (size_t)a.row * 2 * groups + a.group;
  keep8<BF16>(g, a, codes, r, sc);
  keep8<BF16>(u, a, codes, r + I, sc + groups);
}

__device__ __forceinline__ void kept8(const int8_t* codes, size_t base, const KeptAt& a, float scale,
                                      float (&f)[kKeptCols]) {
  const int8_t* p = codes + base + a.c0;
  codes_t v{0, 0};
  if (a.left >= kKeptCols) {
    v = *reinterpret_cast<const codes_t*>(p);
  } else {
#pragma unroll
    for (int i = 0; i < kKeptCols - 1; ++i)
      if (i < a.left) v[i >> 2] |= (uint32_t)(uint8_t)p[i] << (8 * (i & 3));
  }
#pragma unroll
  for (int i = 0; i < kKeptCols; ++i) f[i] = (float)(int8_t)(v[i >> 2] >> (8 * (i & 3))) * scale;
}

template <bool BF16>
__global__ __launch_bounds__(256) void swiglu_backward_kernel(const int8_t* __restrict__ codes,
                                                              const float* __restrict__ scales,
                                                              const void* __restrict__ dh, int64_t rows,
                                                              const int32_t* __restrict__ n_rows, int I, int groups,
                                                              void* __restrict__ dgu, void* __restrict__ h) {
  if (n_rows) rows = min(rows, (int64_t)*n_rows);
  const KeptAt a = kept_at(rows, I, groups);
  if (a.left == 0) return;
  const size_t r = (size_t)a.row * 2 * I;
  const float* sc = scales + (size_t)a.row * 2 * groups + a.group;
  float g[kKeptCols], u[kKeptCols], d[kKeptCols], dg[kKeptCols], du[kKeptCols], f[kKeptCols];
  kept8(codes, r, a, sc[0], g);
  kept8(codes, r + I, a, sc[groups], u);
  load8<BF16>(dh, (size_t)a.row * I, a, d);
#pragma unroll
  for (int i = 0; i < kKeptCols; ++i) {
    const Sigmoid<BF16> s(g[i]);
    const float gs = g[i] * s.s;
    dg[i] = d[i] * u[i] * fmaf(gs, s.t, s.s);
    du[i] = d[i] * gs;
    f[i] = gs * u[i];
  }
  store8<BF16>(dgu, r, a, dg);
  store8<BF16>(dgu, r + I, a, du);
  if (h) store8<BF16>(h, (size_t)a.row * I, a, f);
}

}  // namespace

hipError_t launch_swiglu_save(const void* gu, bool bf16, int rows, const int32_t* n_rows, int I, void* h,
                              int8_t* codes, float* scales, hipStream_t s) {
  const int groups = (I + kKeptGroup - 1) / kKeptGroup;
  const dim3 grid((unsigned)(((int64_t)rows * groups * kKeptLanes + 255) / 256));
  if (bf16)
    hipLaunchKernelGGL(swiglu_save_kernel<true>, grid, dim3(256), 0, s, gu, (int64_t)rows, n_rows, I, groups, h, codes,
                       scales);
  else
    hipLaunchKernelGGL(swiglu_save_kernel<false>, grid, dim3(256), 0, s, gu, (int64_t)rows, n_rows, I, groups, h, codes,
                       scales);
  return hipGetLastError();
}

hipError_t launch_swiglu_backward(const int8_t* codes, const float* scales, const void* dh, bool bf16, int rows,
                                  const int32_t* n_rows, int I, void* dgu, void* h, hipStream_t s) {
  const int groups = (I + kKeptGroup - 1) / kKeptGroup;
  const dim3 grid((unsigned)(((int64_t)rows * groups * kKeptLanes + 255) / 256));
  if (bf16)
    hipLaunchKernelGGL(swiglu_backward_kernel<true>, grid, dim3(256), 0, s, codes, scales, dh, (int64_t)rows, n_rows, I,
                       groups, dgu, h);
  else
    hipLaunchKernelGGL(swiglu_backward_kernel<false>, grid, dim3(256), 0, s, codes, scales, dh, (int64_t)rows, n_rows, I,
                       groups, dgu, h);
  return hipGetLastError();
}

}  // namespace moe
