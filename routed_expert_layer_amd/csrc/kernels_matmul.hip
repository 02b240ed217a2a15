// The experts' products over their groups of rows, on row-major weights, and
// their gradients:
//
//   rows:    c[r, :] = a[r, :] W_e          (or W_e^T: the gradient of the rows)
//   weights: dW_e = sum over the rows r of e of a[r, :]^T dc[r, :]   (0 for an expert without rows)
//
// Every block finds its tile from counts and offsets in GPU memory.
#include <algorithm>

#include "dev_common.hpp"
#include "moe_kernels.hpp"

namespace moe {
namespace {

constexpr int kTile = 64, kDepth = 16;

// c[m, n] = sum_k A(m, k) B(k, n) for one 64 x 64 tile; A(m, k) at a[m sam + k sak] and so on.
template <bool OUT_BF16>
__device__ __forceinline__ void tile_product(const uint16_t* __restrict__ a, size_t sam, size_t sak,
                                             const uint16_t* __restrict__ b, size_t sbk, size_t sbn, int M, int N,
                                             int K, void* __restrict__ c, size_t ldc) {
  __shared__ float la[kDepth][kTile + 1], lb[kDepth][kTile + 1];
  const int tid = threadIdx.x, tm = (tid / 16) * 4, tn = (tid % 16) * 4;
  float acc[4][4] = {};
  for (int k0 = 0; k0 < K; k0 += kDepth) {
    __syncthreads();
    for (int i = tid; i < kTile * kDepth; i += 256) {
      const int m = i % kTile, k = i / kTile;
      la[k][m] = m < M && k0 + k < K ? bf16_to_f32(a[m * sam + (k0 + k) * sak]) : 0.f;
      lb[k][m] = m < N && k0 + k < K ? bf16_to_f32(b[(k0 + k) * sbk + m * sbn]) : 0.f;
    }
    __syncthreads();
    for (int k = 0; k < kDepth; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(la[k][tm + i], lb[k][tn + j], acc[i][j]);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (tm + i < M && tn + j < N) {
        const size_t at = (size_t)(tm + i) * ldc + tn + j;
        if constexpr (OUT_BF16) reinterpret_cast<__bf16*>(c)[at] = (__bf16)acc[i][j];
        else reinterpret_cast<float*>(c)[at] = acc[i][j];
      }
}

// The rows of expert e, or none where they pass rows_max.
__device__ __forceinline__ int group_of(const int32_t* counts, const int32_t* offsets, int e, int rows_max, int& first) {
  const int n = counts[e];
  first = offsets[e];
  return n > 0 && first >= 0 && n <= rows_max && first <= rows_max - n ? n : 0;
}

template <bool TRANSPOSED, bool OUT_BF16>
__global__ __launch_bounds__(256) void matmul_rows_kernel(const uint16_t* __restrict__ a, const uint16_t* __restrict__ w,
                                                          const int32_t* __restrict__ counts,
                                                          const int32_t* __restrict__ offsets, int E, int rows_max,
                                                          int K, int N, void* __restrict__ c) {
  int left = blockIdx.x, first = 0, n = 0, e = 0;
  for (; e < E; ++e) {
    n = group_of(counts, offsets, e, rows_max, first);
    const int tiles = (n + kTile - 1) / kTile;
    if (left < tiles) break;
    left -= tiles;
  }
  if (e == E) return;
  const int m0 = left * kTile, n0 = blockIdx.y * kTile;
  const int depth = TRANSPOSED ? N : K, width = TRANSPOSED ? K : N;
  const size_t row = (size_t)first + m0;
  const uint16_t* b = w + (size_t)e * K * N + (TRANSPOSED ? (size_t)n0 * N : (size_t)n0);
  char* out = static_cast<char*>(c) + (row * width + n0) * (OUT_BF16 ? 2 : 4);
  tile_product<OUT_BF16>(a + row * depth, depth, 1, b, TRANSPOSED ? 1 : N, TRANSPOSED ? N : 1, n - m0, width - n0,
                         depth, out, width);
}

template <bool OUT_BF16>
__global__ __launch_bounds__(256) void matmul_dw_kernel(const uint16_t* __restrict__ a, const uint16_t* __restrict__ dc,
                                                        const int32_t* __restrict__ counts,
                                                        const int32_t* __restrict__ offsets, int rows_max, int K, int N,
                                                        void* __restrict__ dw) {
  const int e = blockIdx.z, k0 = blockIdx.y * kTile, n0 = blockIdx.x * kTile;
  int first;
  const int n = group_of(counts, offsets, e, rows_max, first);
  if (n == 0) first = 0;
  char* out = static_cast<char*>(dw) + ((size_t)e * K * N + (size_t)k0 * N + n0) * (OUT_BF16 ? 2 : 4);
  tile_product<OUT_BF16>(a + (size_t)first * K + k0, 1, K, dc + (size_t)first * N + n0, N, 1, K - k0, N - n0, n, out, N);
}

}  // namespace

hipError_t launch_matmul_grouped(const void* a, const void* w, const int32_t* counts, const int32_t* offsets, int E,
                                 int rows_max, int K, int N, bool transposed, void* c, bool out_bf16, hipStream_t s) {
  const auto* pa = static_cast<const uint16_t*>(a);
  const auto* pw = static_cast<const uint16_t*>(w);
  const int width = transposed ? K : N;
  const dim3 grid(rows_max / kTile + std::min(E, rows_max), (width + kTile - 1) / kTile);
  const auto run = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, dim3(256), 0, s, pa, pw, counts, offsets, E, rows_max, K, N, c);
  };
  if (transposed) out_bf16 ? run(matmul_rows_kernel<true, true>) : run(matmul_rows_kernel<true, false>);
  else out_bf16 ? run(matmul_rows_kernel<false, true>) : run(matmul_rows_kernel<false, false>);
  return hipGetLastError();
}

hipError_t launch_matmul_grouped_dw(const void* a, const void* dc, const int32_t* counts, const int32_t* offsets, int E,
                                    int rows_max, int K, int N, void* dw, bool out_bf16, hipStream_t s) {
  const auto* pa = static_cast<const uint16_t*>(a);
  const auto* pd = static_cast<const uint16_t*>(dc);
  const dim3 grid((N + kTile - 1) / kTile, (K + kTile - 1) / kTile, E);
  const auto run = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, dim3(256), 0, s, pa, pd, counts, offsets, rows_max, K, N, dw);
  };
  out_bf16 ? run(matmul_dw_kernel<true>) : run(matmul_dw_kernel<false>);
  return hipGetLastError();
}

}  // namespace moe
