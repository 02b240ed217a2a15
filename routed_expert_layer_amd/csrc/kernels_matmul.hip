// The experts' products over their groups of rows, on row-major weights, and
// their gradients:
//
//   rows:    c[r, :] = a[r, :] W_e          (or W_e^T: the gradient of the rows)
//   weights: dW_e = sum over the rows r of e of a[r, :]^T dc[r, :]   (0 for an expert without rows)
//
// One tile kernel: BM x 256 results, 32 steps of the sum per stage, operands
// straight from global memory into LDS (16 bytes a lane, no registers), NS
// stages in flight, one barrier per stage; a wave reads the next stage's
// fragments into a second register set while its matrix-core instructions use
// the current one. Operands stay as they lie in memory: one whose sum index is
// the fast one (rows of a, W^T) is read as 16-byte pieces of its rows, one
// whose sum index is the slow one (W, and both sides of the weight gradient)
// through the transposing LDS read (four 16-bit values down a column for each
// of 16 lanes). Both are stored with their pieces exchanged by an XOR of the
// row, so that the reads of a wave fall on all banks.
#include <algorithm>
#include <type_traits>

#include "dev_common.hpp"
#include "gemm_common.hpp"
#include "moe_kernels.hpp"

namespace moe {
namespace {

typedef short s16x4_t __attribute__((ext_vector_type(4)));

constexpr int kBN = 256;     // columns of a tile
constexpr int kStep = 32;    // sum steps of a stage
constexpr uint32_t kNone = 0x80000000u;  // a lane offset past every buffer: the load returns zeros

// One operand of a tile: SIZE rows or columns of results, kStep of the sum per
// stage. SLOW: the sum index is the slow one in memory.
template <bool SLOW, int SIZE>
struct Side {
  static constexpr int kLoads = SIZE / 16;           // 1 KiB loads per stage
  static constexpr int kBytes = SIZE * kStep * 2;    // LDS bytes per stage
  // Fast: LDS holds SIZE rows of four 16-byte pieces, piece c of row r in slot c ^ (r / 2 % 4): eight rows' pieces of
  // one c, which a wave reads together, lie in 128 different bytes of the banks.
  // Slow: LDS holds kStep rows of SIZE columns; the 32-byte pair of pieces p of row k in place p ^ turn(k).
  static __device__ __forceinline__ int turn(int k) {
    return SIZE >= 128 ? (k & 3) | ((k >> 3) & 1) << 2 : ((k >> 1) & 1) | ((k >> 3) & 1) << 1;
  }
  // Byte offset of what this lane fetches with load f of a stage, from the tile's first element; `lim` results are in
  // the operand from there on (past them the last ones are fetched, for results that are not stored). ld in elements.
  static __device__ __forceinline__ uint32_t fetch(int f, int lane, int ld, int lim) {
    if constexpr (SLOW) {
      constexpr int kLanes = SIZE / 8;  // lanes per row
      const int k = f * (64 / kLanes) + lane / kLanes, slot = lane % kLanes;
      const int col = ((((slot >> 1) ^ turn(k)) << 1) | (slot & 1)) * 8;
      return (uint32_t)(k * ld + min(col, lim - 8)) * 2u;
    } else {
      const int r = f * 16 + lane / 4;
      return (uint32_t)min(r, lim - 1) * (uint32_t)ld * 2u + (uint32_t)((lane & 3) ^ ((r >> 1) & 3)) * 16u;
    }
  }
  // The first of the eight sum steps (of a stage's 32) that this lane fetches; fast operands only.
  static __device__ __forceinline__ int step_of(int lane) { return ((lane & 3) ^ ((lane >> 3) & 3)) * 8; }
};

// Fragments of 16 results x 32 steps: lane l holds result l % 16, steps 8 (l / 16) .. + 7.
template <bool SLOW, int SIZE, int N>
struct Reader {
  uint32_t at[SLOW ? N : 1];
  __device__ __forceinline__ Reader(int first, int lane) {
    if constexpr (SLOW) {
      const int k = 8 * (lane >> 4) + ((lane & 15) >> 2), q = lane & 3;
#pragma unroll
      for (int i = 0; i < N; ++i) at[i] = k * SIZE * 2 + (((first + i) ^ Side<SLOW, SIZE>::turn(k)) << 5) + q * 8;
    } else {
      const int r = lane & 15;
      at[0] = (first * 16 + r) * 64 + (((lane >> 4) ^ ((r >> 1) & 3)) << 4);
    }
  }
  __device__ __forceinline__ u32x4_t read(const char* stage, int i) const {
    if constexpr (SLOW) {
      using P = __attribute__((address_space(3))) s16x4_t*;
      const char* p = stage + at[i];
      const s16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((P)p);
      const s16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((P)(p + 4 * SIZE * 2));
      const u32x2_t a = __builtin_bit_cast(u32x2_t, lo), b = __builtin_bit_cast(u32x2_t, hi);
      return u32x4_t{a[0], a[1], b[0], b[1]};
    } else {
      return *reinterpret_cast<const u32x4_t*>(stage + at[0] + i * 1024);
    }
  }
};

// One 16-byte piece per lane from base + off straight into the wave's 1 KiB at LDS byte `lds`; a lane offset of `bytes` or
// more fetches zeros. In assembly, because the compiler waits for every load to LDS it knows of before a transposing read
// (s_waitcnt vmcnt(0) in each stage); nothing is returned in registers, and the waits for the data are the explicit ones
// of the loop below. Five wait states stand between a vector instruction that may have written a scalar operand and the
// load, one between the write of m0 (which nothing else in these kernels uses) and the load.
__device__ __forceinline__ void load_lds16(const void* base, uint32_t bytes, uint32_t off, uint32_t lds) {
  const uint64_t p = reinterpret_cast<uint64_t>(base);
  const u32x4_t r{(uint32_t)p, (uint32_t)(p >> 32) & 0xFFFFu, bytes, 0x00020000u};
  asm volatile("s_nop 4\n\ts_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds"
               :
               : "v"(off), "s"(r), "s"(lds)
               : "memory");
}

// What one tile works on. a and b point at the tile's first element; lda and ldb are elements per row of memory; m and n
// results are left from the tile's first on, `depth` sum steps.
struct Tile {
  const uint16_t* a;
  const uint16_t* b;
  char* c;
  int lda, ldb, ldc, m, n, depth;
};

template <int BM, int WAVES_M, int WAVES_N, int NS, bool SLOW_A, bool SLOW_B, bool OUT_BF16>
__device__ __forceinline__ void tile_product(const Tile& t, char* lds) {
  constexpr int kWaves = WAVES_M * WAVES_N;
  using A = Side<SLOW_A, BM>;
  using B = Side<SLOW_B, kBN>;
  constexpr int kStage = A::kBytes + B::kBytes;
  constexpr int MF = BM / WAVES_M / 16, NF = kBN / WAVES_N / 16;  // fragments per wave
  constexpr int LA = A::kLoads / kWaves, LB = B::kLoads / kWaves, L = LA + LB;
  static_assert(A::kLoads % kWaves == 0 && B::kLoads % kWaves == 0, "loads split over the waves");
  const int tid = (int)threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)lds;
  const int wm = wave % WAVES_M, wn = wave / WAVES_M;
  const int stages = (t.depth + kStep - 1) / kStep, tail = t.depth % kStep;

  uint32_t off[L];
#pragma unroll
  for (int q = 0; q < LA; ++q) off[q] = A::fetch(wave + kWaves * q, lane, t.lda, t.m);
#pragma unroll
  for (int q = 0; q < LB; ++q) off[LA + q] = B::fetch(wave + kWaves * q, lane, t.ldb, t.n);
  const bool none = tail != 0 && A::step_of(lane) >= tail;  // past the sum's end in the last stage

  // Stage s -> LDS buffer `buf`. Steps past the sum's end are zeros on both sides: of a slow operand by the buffer's
  // size, of a fast one by the lane offset.
  auto issue = [&](int s, int buf) {
    const uint32_t base = lds0 + buf * kStage;
    const bool last = s == stages - 1;
    const uint32_t left = (uint32_t)min(kStep, t.depth - s * kStep);
    const uint16_t* pa = t.a + (SLOW_A ? (size_t)s * kStep * t.lda : (size_t)s * kStep);
    const uint16_t* pb = t.b + (SLOW_B ? (size_t)s * kStep * t.ldb : (size_t)s * kStep);
    const uint32_t na = SLOW_A ? left * (uint32_t)t.lda * 2u : kNone;
    const uint32_t nb = SLOW_B ? left * (uint32_t)t.ldb * 2u : kNone;
#pragma unroll
    for (int q = 0; q < LA; ++q)
      load_lds16(pa, na, !SLOW_A && last && none ? kNone : off[q], base + (wave + kWaves * q) * 1024);
#pragma unroll
    for (int q = 0; q < LB; ++q)
      load_lds16(pb, nb, !SLOW_B && last && none ? kNone : off[LA + q], base + A::kBytes + (wave + kWaves * q) * 1024);
  };

  const Reader<SLOW_A, BM, MF> ra(wm * MF, lane);
  const Reader<SLOW_B, kBN, NF> rb(wn * NF, lane);
  f32x4_t acc[NF][MF];
#pragma unroll
  for (int i = 0; i < NF; ++i)
#pragma unroll
    for (int j = 0; j < MF; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  struct Frags {
    u32x4_t a[MF], b[NF];
  };

  // JM: this wave's fragments of rows that hold any result (uniform per wave).
  auto sum = [&](auto jm_const) {
    constexpr int JM = decltype(jm_const)::value;
    auto read = [&](int s, Frags& f) {
      const char* base = lds + (s % NS) * kStage;
      if constexpr (JM > 0) {
#pragma unroll
        for (int j = 0; j < JM; ++j) f.a[j] = ra.read(base, j);
#pragma unroll
        for (int i = 0; i < NF; ++i) f.b[i] = rb.read(base + A::kBytes, i);
      }
    };
    auto compute = [&](const Frags& f) {
#pragma unroll
      for (int i = 0; i < NF; ++i)
#pragma unroll
        for (int j = 0; j < JM; ++j) acc[i][j] = mfma_bf16(f.b[i], f.a[j], acc[i][j]);
    };
    auto step = [&](int s, Frags& cur, Frags& nxt) {
      // this wave's loads of stage s + 1 have landed, and its reads of stage s
      if (s + NS - 1 < stages) {
        __builtin_amdgcn_s_waitcnt(vmcnt_only(L * (NS - 2)));
      } else {
        __builtin_amdgcn_s_waitcnt(vmcnt_only(0));
      }
      __builtin_amdgcn_s_waitcnt(lgkmcnt_only(0));
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
      if (s + NS < stages) issue(s + NS, s % NS);
      read(min(s + 1, stages - 1), nxt);
      compute(cur);
      if constexpr (JM > 0) {
        constexpr int kReads = JM * (SLOW_A ? 2 : 1) + NF * (SLOW_B ? 2 : 1);
        constexpr int kPer = (NF * JM) / kReads > 0 ? (NF * JM) / kReads : 1;
#pragma unroll
        for (int q = 0; q < kReads; ++q) {
          __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
          __builtin_amdgcn_sched_group_barrier(0x008, kPer, 0);
        }
      }
    };
    for (int s = 0; s < NS && s < stages; ++s) issue(s, s);
    if (stages >= NS) {
      __builtin_amdgcn_s_waitcnt(vmcnt_only(L * (NS - 1)));
    } else {
      __builtin_amdgcn_s_waitcnt(vmcnt_only(0));
    }
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    Frags f0, f1;
    read(0, f0);
    int s = 0;
    for (; s + 1 < stages; s += 2) {
      step(s, f0, f1);
      step(s + 1, f1, f0);
    }
    if (s < stages) step(s, f0, f1);
  };
  static_assert(MF % 4 == 0, "the dispatch below takes quarters");
  const int rows_here = t.m - wm * MF * 16;
  const int quarter = rows_here <= 0 ? 0 : min(4, (rows_here + MF * 4 - 1) / (MF * 4));
  if (stages > 0) switch (quarter) {
    case 0: sum(std::integral_constant<int, 0>{}); break;
    case 1: sum(std::integral_constant<int, MF / 4>{}); break;
    case 2: sum(std::integral_constant<int, MF / 2>{}); break;
    case 3: sum(std::integral_constant<int, MF / 4 * 3>{}); break;
    default: sum(std::integral_constant<int, MF>{}); break;
  }

  // Lane l holds row l % 16 of a fragment and its columns 4 (l / 16) .. + 3.
  const int g = lane >> 4;
#pragma unroll
  for (int j = 0; j < MF; ++j) {
    const int m = (wm * MF + j) * 16 + (lane & 15);
#pragma unroll
    for (int i = 0; i < NF; ++i) {
      const int n = (wn * NF + i) * 16 + 4 * g;
      if (m >= t.m || n >= t.n) continue;
      const f32x4_t v = acc[i][j];
      if constexpr (OUT_BF16) {
        typedef __bf16 bf16x4_t __attribute__((ext_vector_type(4)));
        *reinterpret_cast<u32x2_t*>(t.c + ((size_t)m * t.ldc + n) * 2) =
            __builtin_bit_cast(u32x2_t, bf16x4_t{(__bf16)v[0], (__bf16)v[1], (__bf16)v[2], (__bf16)v[3]});
      } else {
        *reinterpret_cast<f32x4_t*>(t.c + ((size_t)m * t.ldc + n) * 4) = v;
      }
    }
  }
}

// The rows of expert e, or none where they pass rows_max.
__device__ __forceinline__ int group_of(const int32_t* counts, const int32_t* offsets, int e, int rows_max, int& first) {
  const int n = counts[e];
  first = offsets[e];
  return n > 0 && first >= 0 && n <= rows_max && first <= rows_max - n ? n : 0;
}

struct RowTile {
  int e, first, rows, m, n;  // expert, its first row and rows, tile indexes; e < 0: none
};

// Tile number `index` of all experts' tiles (expert, then column tile, then row tile), BM rows and kBN columns each; the
// blocks of one XCD (equal index modulo 8) take consecutive ones, so that the blocks that run together on it share an
// expert's rows and columns in its L2.
template <int BM, int THREADS>
__device__ __forceinline__ RowTile find_tile(const int32_t* __restrict__ counts, const int32_t* __restrict__ offsets,
                                             int E, int rows_max, int col_tiles, int* sums, RowTile* found) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int per = (E + THREADS - 1) / THREADS, e0 = tid * per, e1 = min(E, e0 + per);
  int mine = 0, first;
  for (int e = e0; e < e1; ++e) mine += (group_of(counts, offsets, e, rows_max, first) + BM - 1) / BM;
  int s = mine;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(s, d, 64);
    if (lane >= d) s += o;
  }
  if (lane == 63) sums[wave] = s;
  if (tid == 0) found->e = -1;
  __syncthreads();
  int before = s - mine, total = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 64; ++w) {
    before += w < wave ? sums[w] : 0;
    total += sums[w];
  }
  const int64_t all = (int64_t)total * col_tiles, share = (all + 7) / 8;
  const int64_t at = (int64_t)(blockIdx.x >> 3), index = (blockIdx.x & 7) * share + at;
  if (at < share && index < all) {
    int64_t left = index - (int64_t)before * col_tiles;
    if (left >= 0 && left < (int64_t)mine * col_tiles)
      for (int e = e0; e < e1; ++e) {
        const int n = group_of(counts, offsets, e, rows_max, first), tiles = (n + BM - 1) / BM;
        if (left < (int64_t)tiles * col_tiles) {
          *found = RowTile{e, first, n, (int)(left % tiles), (int)(left / tiles)};
          break;
        }
        left -= (int64_t)tiles * col_tiles;
      }
  }
  __syncthreads();
  return *found;
}

template <int BM, int WAVES_M, int WAVES_N, int NS, bool TRANSPOSED, bool OUT_BF16>
__global__ __launch_bounds__(64 * WAVES_M * WAVES_N, BM == 64 ? 2 : 1) void matmul_rows_kernel(
    const uint16_t* __restrict__ a, const uint16_t* __restrict__ w, const int32_t* __restrict__ counts,
    const int32_t* __restrict__ offsets, int E, int rows_max, int K, int N, char* __restrict__ c) {
  __shared__ __attribute__((aligned(1024))) char lds[NS * (BM + kBN) * kStep * 2];
  const int depth = TRANSPOSED ? N : K, width = TRANSPOSED ? K : N;
  const int col_tiles = (width + kBN - 1) / kBN;
  const RowTile f = find_tile<BM, 64 * WAVES_M * WAVES_N>(counts, offsets, E, rows_max, col_tiles,
                                                          reinterpret_cast<int*>(lds),
                                                          reinterpret_cast<RowTile*>(lds + 256));
  __syncthreads();  // the stages overwrite what was found
  const int e = __builtin_amdgcn_readfirstlane(f.e);
  if (e < 0) return;
  const int m0 = __builtin_amdgcn_readfirstlane(f.m) * BM, n0 = __builtin_amdgcn_readfirstlane(f.n) * kBN;
  const size_t row = (size_t)__builtin_amdgcn_readfirstlane(f.first) + m0;
  Tile t;
  t.a = a + row * depth;
  t.b = w + (size_t)e * K * N + (TRANSPOSED ? (size_t)n0 * N : (size_t)n0);
  t.c = c + (row * width + n0) * (OUT_BF16 ? 2 : 4);
  t.lda = depth;
  t.ldb = N;
  t.ldc = width;
  t.m = __builtin_amdgcn_readfirstlane(f.rows) - m0;
  t.n = width - n0;
  t.depth = depth;
  tile_product<BM, WAVES_M, WAVES_N, NS, false, !TRANSPOSED, OUT_BF16>(t, lds);
}

template <int BM, int WAVES_M, int WAVES_N, int NS, bool OUT_BF16>
__global__ __launch_bounds__(64 * WAVES_M * WAVES_N, BM == 64 ? 2 : 1) void matmul_dw_kernel(
    const uint16_t* __restrict__ a, const uint16_t* __restrict__ dc, const int32_t* __restrict__ counts,
    const int32_t* __restrict__ offsets, int rows_max, int K, int N, char* __restrict__ dw) {
  __shared__ __attribute__((aligned(1024))) char lds[NS * (BM + kBN) * kStep * 2];
  const int row_tiles = (K + BM - 1) / BM, col_tiles = (N + kBN - 1) / kBN, tiles = row_tiles * col_tiles;
  // as in find_tile: consecutive tiles to the blocks of one XCD
  const unsigned share = gridDim.x / 8, extra = gridDim.x % 8, x = blockIdx.x & 7;
  const unsigned index = x * share + min(x, extra) + (blockIdx.x >> 3);
  const int e = (int)(index / tiles), left = (int)(index % tiles);
  const int k0 = (left % row_tiles) * BM, n0 = (left / row_tiles) * kBN;
  int first;
  const int n = group_of(counts, offsets, e, rows_max, first);
  if (n == 0) first = 0;
  Tile t;
  t.a = a + (size_t)first * K + k0;
  t.b = dc + (size_t)first * N + n0;
  t.c = dw + ((size_t)e * K * N + (size_t)k0 * N + n0) * (OUT_BF16 ? 2 : 4);
  t.lda = K;
  t.ldb = N;
  t.ldc = N;
  t.m = K - k0;
  t.n = N - n0;
  t.depth = n;
  tile_product<BM, WAVES_M, WAVES_N, NS, true, true, OUT_BF16>(t, lds);
}

}  // namespace

hipError_t launch_matmul_grouped(const void* a, const void* w, const int32_t* counts, const int32_t* offsets, int E,
                                 int rows_max, int K, int N, bool transposed, void* c, bool out_bf16, hipStream_t s) {
  const auto* pa = static_cast<const uint16_t*>(a);
  const auto* pw = static_cast<const uint16_t*>(w);
  const int64_t col_tiles = ((transposed ? K : N) + kBN - 1) / kBN;
  const auto run = [&](auto kernel, int bm, int threads) {
    const int64_t blocks = ((rows_max / bm + std::min(E, rows_max)) * col_tiles + 7) / 8 * 8;
    hipLaunchKernelGGL(kernel, dim3((unsigned)blocks), dim3(threads), 0, s, pa, pw, counts, offsets, E, rows_max, K, N,
                       static_cast<char*>(c));
  };
  const auto sized = [&](auto t, auto o) {
    constexpr bool T = decltype(t)::value, O = decltype(o)::value;
    const int64_t mean = rows_max / E;
    if (mean <= 64) run(matmul_rows_kernel<64, 1, 4, 4, T, O>, 64, 256);
    else if (mean <= 512) run(matmul_rows_kernel<128, 2, 4, 6, T, O>, 128, 512);
    else run(matmul_rows_kernel<256, 2, 4, 4, T, O>, 256, 512);
  };
  if (transposed) out_bf16 ? sized(std::true_type{}, std::true_type{}) : sized(std::true_type{}, std::false_type{});
  else out_bf16 ? sized(std::false_type{}, std::true_type{}) : sized(std::false_type{}, std::false_type{});
  return hipGetLastError();
}

hipError_t launch_matmul_grouped_dw(const void* a, const void* dc, const int32_t* counts, const int32_t* offsets, int E,
                                    int rows_max, int K, int N, void* dw, bool out_bf16, hipStream_t s) {
  const auto* pa = static_cast<const uint16_t*>(a);
  const auto* pd = static_cast<const uint16_t*>(dc);
  const auto run = [&](auto kernel, int bm, int threads) {
    const int64_t blocks = (int64_t)((N + kBN - 1) / kBN) * ((K + bm - 1) / bm) * E;
    hipLaunchKernelGGL(kernel, dim3((unsigned)blocks), dim3(threads), 0, s, pa, pd, counts, offsets, rows_max, K, N,
                       static_cast<char*>(dw));
  };
  if (rows_max / E <= 64) out_bf16 ? run(matmul_dw_kernel<64, 1, 4, 4, true>, 64, 256) : run(matmul_dw_kernel<64, 1, 4, 4, false>, 64, 256);
  else out_bf16 ? run(matmul_dw_kernel<256, 2, 4, 4, true>, 256, 512) : run(matmul_dw_kernel<256, 2, 4, 4, false>, 256, 512);
  return hipGetLastError();
}

}  // namespace moe
