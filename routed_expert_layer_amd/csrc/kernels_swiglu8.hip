// SwiGLU whose inputs are kept in 8 bits, and its backward pass from them.
//
//   g = gu[r, :I], u = gu[r, I:],  s(g) = 1 / (1 + e^-g),  h = g s(g) u
//   kept, for 128 columns of g or u at a time:  scale = max|v| / 127,  code = rne(127 v / max|v|)
//   backward, from g^, u^ = code * scale:
//     dg = dh u^ s (1 + g^ (1 - s)),  du = dh g^ s,  h^ = g^ s u^
//
// A lane takes 16 bytes of g and the same columns of u, so that a wave's loads
// and stores are whole lines: 16 lanes 128 columns of bf16, 32 of fp32 (eight
// columns a lane there too: 16384 rows of 2 x 2048 fp32 back in 146 us, 86 so).
// A scale is one reduction over those lanes, and every byte is moved once.
// Bytes bound both passes: 98304 bf16 rows of 2 x 2048 take 668 us, 3.65 GB at
// 5.5 TB/s (a copy reaches 4.9).
#include <type_traits>

#include "dev_common.hpp"
#include "moe_kernels.hpp"
#include "row_quant.hpp"
#include "row_vec.hpp"

namespace moe {
namespace {

constexpr int kKeptGroup = 128;  // columns that share a scale

// s(g) = 1 / (1 + e^-g), t = 1 - s and g s, none by a difference that loses bits. The exponent's argument has 48 bits,
// the reciprocal is corrected by what 1 + e and it were rounded by, and for g >= 0 g s = g - g t is rounded once, so that
// all are off by some half steps of 2^-24 at any g. That shows in bf16 results too: g u often lies next to a tie, and the
// last bits of s decide. By the hardware's exponential and reciprocal as they are 1.7e-5 of 8192 x 2048 values of h went
// to the other side, 0.5e-5 so (most of them of one value of g); both passes of 98304 rows 642 us and 668.
// FAR: of gates below -64 s and g s are 2^64 times as large, and `down` takes products with them back: e^g then is a
// normal number down to e^-131, and what the hardware's exponential loses below 2^-126 is not lost to a large u or dh.
// An infinity or NaN in g reaches every result.
template <bool FAR>
struct Silu {
  float s, t, gs, down;
  __device__ __forceinline__ explicit Silu(float g) {
#pragma clang fp contract(off)  // p is rounded: its residue is `low`
    constexpr float kLog2E = 1.44269504f, kLog2ELow = 1.92596299e-8f, kLn2 = 0.693147181f;
    const bool far = FAR && g < -64.f;
    const float x = fminf(fabsf(g), 512.f);
    const float p = x * -kLog2E, low = fmaf(x, -kLog2ELow, fmaf(x, -kLog2E, -p));
    const float w = __builtin_amdgcn_exp2f(far ? p + 64.f : p);  // the sum is exact
    const float e = fmaf(w, low * kLn2, w);                      // far: below 2^-27, 1 + e is 1 either way
    const float q = __builtin_amdgcn_rcpf(1.f + e), r = fmaf(fmaf(-q, e, 1.f - q), q, q), er = e * r;
    const bool up = g >= 0.f;
    s = up ? r : er;
    t = up ? er : r;
    gs = fmaf(up ? -x : g, er, up ? g : 0.f);
    down = far ? 0x1p-64f : 1.f;
  }
};

// f with Silu's form for these gates: most threads have none far out, and the same bits by either.
template <int N, typename F>
__device__ __forceinline__ void with_silu(const float (&g)[N], const F& f) {
  float least = g[0];
#pragma unroll
  for (int i = 1; i < N; ++i) least = fminf(least, g[i]);
  if (least < -64.f) f(std::true_type{});
  else f(std::false_type{});
}

// Where a thread works: a row and the columns from c on.
struct KeptAt {
  int64_t row;
  int c, left;  // left: columns of g (and u) from c on, 0 for a thread without any
};

template <bool BF16, int N>
__device__ __forceinline__ void load(const void* p, size_t base, const KeptAt& a, float (&f)[N]) {
  RowVec<BF16, N> v;
  v.load(p, base + a.c, a.left);
#pragma unroll
  for (int i = 0; i < N; ++i) f[i] = v.get(i);
}

// Past the caches at any length, though pieces may lie across lines: 60000 bf16 rows of 2 x 645 75 us out and 66 back, 86
// and 72 through the caches; fp32 112 and 116, 114 and 136; 98304 bf16 rows of 2 x 2048 back 333 and 345.
template <bool BF16, int N>
__device__ __forceinline__ void store(void* p, size_t base, const KeptAt& a, const float (&f)[N]) {
  RowVec<BF16, N> v;
  v.set(f);
  v.template store<true>(p, base + a.c, a.left);
}

template <int N>
using codes_t __attribute__((aligned(1))) = uint32_t __attribute__((ext_vector_type(N / 4)));  // N codes at any byte

template <bool BF16, int N>
__device__ __forceinline__ void keep(const float (&f)[N], const KeptAt& a, bool first, int8_t* codes, size_t base,
                                     float* scale) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) m = max(m, __float_as_uint(f[i]) & 0x7FFFFFFFu);
#pragma unroll
  for (int d = kKeptGroup / N / 2; d > 0; d >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, d, 64));
  const RowQuant q(m);
  if (a.left == 0) return;
  if (first) *scale = q.scale();
  codes_t<N> v;
#pragma unroll
  for (int i = 0; i < N / 4; ++i) v[i] = q.pack4<BF16>(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
  int8_t* p = codes + base + a.c;
  if (a.left >= N) {
    *reinterpret_cast<codes_t<N>*>(p) = v;
  } else {
    typedef uint16_t half_t __attribute__((aligned(1)));
    typedef uint32_t word_t __attribute__((aligned(1)));
    uint32_t rest = v[0];  // four, two and one of them
    if (N > 4 && a.left >= 4) {
      *reinterpret_cast<word_t*>(p) = rest;
      rest = v[N / 4 - 1];
      p += 4;
    }
    if (a.left & 2) {
      *reinterpret_cast<half_t*>(p) = (uint16_t)rest;
      rest >>= 16;
      p += 2;
    }
    if (a.left & 1) *p = (int8_t)rest;
  }
}

template <bool BF16>
__global__ __launch_bounds__(256) void swiglu_save_kernel(const void* __restrict__ gu, int64_t rows,
                                                          const int32_t* __restrict__ n_rows, int I, int groups,
                                                          void* __restrict__ h, int8_t* __restrict__ codes,
                                                          float* __restrict__ scales) {
  if (n_rows) rows = min(rows, (int64_t)*n_rows);
  constexpr int N = kVecElems<BF16>, kLanes = kKeptGroup / N;
  const uint32_t q = (blockIdx.x * 256u + threadIdx.x) / kLanes;  // rows * groups is 2^26 at most
  const int group = (int)(q % (uint32_t)groups), lane = (int)threadIdx.x & (kLanes - 1);
  const int c0 = group * kKeptGroup + lane * N;
  KeptAt a{(int64_t)(q / (uint32_t)groups), c0, 0};
  a.left = a.row < rows ? max(0, I - c0) : 0;  // a thread without columns stays for the reductions
  const size_t r = (size_t)a.row * 2 * I;
  float g[N], u[N], f[N];
  load<BF16>(gu, r, a, g);
  load<BF16>(gu, r + I, a, u);
  with_silu(g, [&](auto far) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const Silu<decltype(far)::value> v(g[i]);
      f[i] = v.gs * u[i] * v.down;
    }
  });
  store<BF16>(h, (size_t)a.row * I, a, f);
  float* sc = scales + (size_t)a.row * 2 * groups + group;
  keep<BF16>(g, a, lane == 0, codes, r, sc);
  keep<BF16>(u, a, lane == 0, codes, r + I, sc + groups);
}

// sc: the row's scales. The row's last piece may begin in the group before the last.
template <int N>
__device__ __forceinline__ void kept(const int8_t* codes, size_t base, const KeptAt& a, const float* sc, float (&f)[N]) {
  const int8_t* p = codes + base + a.c;
  const int g0 = a.c / kKeptGroup, g1 = (a.c + min(a.left, N) - 1) / kKeptGroup;
  const int turn = g1 * kKeptGroup - a.c;  // the columns from here on have the second scale
  const float s0 = sc[g0], s1 = sc[g1];
  codes_t<N> v = 0;
  if (a.left >= N) {
    v = *reinterpret_cast<const codes_t<N>*>(p);
  } else {
#pragma unroll
    for (int i = 0; i < N - 1; ++i)
      if (i < a.left) v[i >> 2] |= (uint32_t)(uint8_t)p[i] << (8 * (i & 3));
  }
#pragma unroll
  for (int i = 0; i < N; ++i) f[i] = (float)(int8_t)(v[i >> 2] >> (8 * (i & 3))) * (i < turn ? s0 : s1);
}

template <bool BF16>
__global__ __launch_bounds__(256) void swiglu_backward_kernel(const int8_t* __restrict__ codes,
                                                              const float* __restrict__ scales,
                                                              const void* __restrict__ dh, int64_t rows,
                                                              const int32_t* __restrict__ n_rows, int I, int groups,
                                                              void* __restrict__ dgu, void* __restrict__ h) {
  if (n_rows) rows = min(rows, (int64_t)*n_rows);
  constexpr int N = kVecElems<BF16>;
  const uint32_t q = blockIdx.x * 256u + threadIdx.x, pieces = (uint32_t)(I + N - 1) / N;
  KeptAt a{(int64_t)(q / pieces), piece_start<N>((int)(q % pieces) * N, I), 0};
  if (a.row >= rows) return;
  a.left = I - a.c;
  const size_t r = (size_t)a.row * 2 * I;
  const float* sc = scales + (size_t)a.row * 2 * groups;
  float g[N], u[N], d[N], dg[N], du[N], f[N];
  kept(codes, r, a, sc, g);
  kept(codes, r + I, a, sc + groups, u);
  load<BF16>(dh, (size_t)a.row * I, a, d);
  with_silu(g, [&](auto far) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const Silu<decltype(far)::value> v(g[i]);
      // s's derivative is 1.1 at most: half of it times the larger factor stays in range, and so does what follows where
      // the result does (dh u alone may not)
      const float a = fabsf(d[i]) > fabsf(u[i]) ? d[i] : u[i], b = fabsf(d[i]) > fabsf(u[i]) ? u[i] : d[i];
      dg[i] = a * (0.5f * fmaf(v.gs, v.t, v.s)) * b * (2.f * v.down);
      du[i] = d[i] * v.gs * v.down;
      f[i] = v.gs * u[i] * v.down;
    }
  });
  store<BF16>(dgu, r, a, dg);
  store<BF16>(dgu, r + I, a, du);
  if (h) store<BF16>(h, (size_t)a.row * I, a, f);
}

}  // namespace

hipError_t launch_swiglu_save(const void* gu, bool bf16, int rows, const int32_t* n_rows, int I, void* h,
                              int8_t* codes, float* scales, hipStream_t s) {
  const int groups = (I + kKeptGroup - 1) / kKeptGroup;
  const int lanes = kKeptGroup / (bf16 ? kVecElems<true> : kVecElems<false>);
  const dim3 grid((unsigned)(((int64_t)rows * groups * lanes + 255) / 256));
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
  const int each = bf16 ? kVecElems<true> : kVecElems<false>, pieces = (I + each - 1) / each;
  const dim3 grid((unsigned)(((int64_t)rows * pieces + 255) / 256));
  if (bf16)
    hipLaunchKernelGGL(swiglu_backward_kernel<true>, grid, dim3(256), 0, s, codes, scales, dh, (int64_t)rows, n_rows, I,
                       groups, dgu, h);
  else
    hipLaunchKernelGGL(swiglu_backward_kernel<false>, grid, dim3(256), 0, s, codes, scales, dh, (int64_t)rows, n_rows, I,
                       groups, dgu, h);
  return hipGetLastError();
}

}  // namespace moe
