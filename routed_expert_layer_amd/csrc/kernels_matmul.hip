// The experts' products over their groups of rows, on row-major weights, and
// their gradients:
//
//   rows:    c[r, :] = a[r, :] W_e          (or W_e^T: the gradient of the rows)
//   weights: dW_e = sum over the rows r of e of a[r, :]^T dc[r, :]   (0 for an expert without rows)
//
// One tile kernel: BM x 256 results, the sum in parts of 32 steps, operands
// straight from global memory into LDS (16 bytes a lane, no registers), one
// barrier per part; a wave reads the fragments of the next part into a second
// register set while its matrix-core instructions use the current one.
// Operands stay as they lie in memory: one whose sum index is the fast one
// (rows of a, W^T) is read as 16-byte pieces of its rows, one whose sum index
// is the slow one (W, and both sides of the weight gradient) through the
// transposing LDS read (four 16-bit values down a column for each of 16
// lanes). Both are stored with their pieces exchanged by an XOR of the row, so
// that the reads of a wave fall on all banks. Each operand has a ring of its
// own in LDS: of parts for a slow one, of pairs of parts for a fast one, whose
// rows then come in whole cache lines.
//
// What bounds them: long groups the operands' way from the memory-side cache,
// at a clock that the power limit holds at 1.8 to 2.0 GHz of 2.4 (1536 rows an
// expert of 4096 x 4096: 1165 to 1245 TFLOP/s, W^T 1180 to 1230, weight
// gradients 1100 to 1165; the library's dense products 1277, 1484, 1172; matrix
// cores busy 65, 63 and 54% of the cycles), few rows the weights' bytes (3 rows
// an expert 6.3 to 6.6 TB/s), short weight gradients their stores (5.2 TB/s).
#include <algorithm>
#include <type_traits>

#include "dev_common.hpp"
#include "gemm_common.hpp"
#include "moe_kernels.hpp"

namespace moe {
namespace {

typedef short s16x4_t __attribute__((ext_vector_type(4)));

constexpr int kBN = 256;     // columns of a tile
constexpr int kPart = 32;    // sum steps of a part
constexpr uint32_t kNone = 0x80000000u;  // a lane offset past every buffer: the load returns zeros

template <typename T>
struct type_of {
  using type = T;
};

// One operand of a tile: SIZE rows or columns of results. SLOW: the sum index
// is the slow one in memory. A slot of its ring holds kStep of the sum.
template <bool SLOW, int SIZE>
struct Side {
  static constexpr int kParts = SLOW ? 1 : 2, kStep = kPart * kParts;
  static constexpr int kBytes = SIZE * kStep * 2;    // of a slot
  static constexpr int kLoads = kBytes / 1024;       // 1 KiB loads per slot
  // Fast: a slot holds SIZE rows of eight 16-byte pieces, piece c of row r in place c ^ turn(r): eight rows' pieces of
  // one c, which a wave reads together, lie in 128 different bytes of the banks.
  // Slow: a slot holds 32 rows of SIZE columns; the 32-byte pair of pieces p of row k in place p ^ turn(k).
  static __device__ __forceinline__ int turn(int r) {
    if constexpr (!SLOW) return r & 7;
    return SIZE >= 128 ? (r & 3) | ((r >> 3) & 1) << 2 : ((r >> 1) & 1) | ((r >> 3) & 1) << 1;
  }
  // Byte offset of what this lane fetches with load f of a slot, from the tile's first element; `lim` results are in
  // the operand from there on (nothing is fetched for those past them). ld in elements.
  static __device__ __forceinline__ uint32_t fetch(int f, int lane, int ld, int lim) {
    if constexpr (SLOW) {
      constexpr int kLanes = SIZE / 8;  // lanes per row
      const int k = f * (64 / kLanes) + lane / kLanes, slot = lane % kLanes;
      const int col = ((((slot >> 1) ^ turn(k)) << 1) | (slot & 1)) * 8;
      return col < lim ? (uint32_t)(k * ld + col) * 2u : kNone;
    } else {
      const int r = f * 8 + lane / 8;
      return r < lim ? (uint32_t)r * (uint32_t)ld * 2u + (uint32_t)((lane & 7) ^ turn(r)) * 16u : kNone;
    }
  }
  // The first of the eight sum steps (of a slot's) that this lane fetches; fast operands only.
  static __device__ __forceinline__ int step_of(int lane) { return ((lane & 7) ^ turn(lane / 8)) * 8; }
};

// Fragments of 16 results x 32 steps, part h of a slot: lane l holds result l % 16, steps 8 (l / 16) .. + 7.
template <bool SLOW, int SIZE, int N>
struct Reader {
  using S = Side<SLOW, SIZE>;
  uint32_t at[SLOW ? N : 2];
  __device__ __forceinline__ Reader(int first, int lane) {
    if constexpr (SLOW) {
      const int k = 8 * (lane >> 4) + ((lane & 15) >> 2), q = lane & 3;
#pragma unroll
      for (int i = 0; i < N; ++i) at[i] = k * SIZE * 2 + (((first + i) ^ S::turn(k)) << 5) + q * 8;
    } else {
      const int r = lane & 15;
#pragma unroll
      for (int h = 0; h < 2; ++h) at[h] = (first * 16 + r) * (S::kStep * 2) + (((4 * h + (lane >> 4)) ^ S::turn(r)) << 4);
    }
  }
  __device__ __forceinline__ u32x4_t read(const char* slot, int h, int i) const {
    if constexpr (SLOW) {
      using P = __attribute__((address_space(3))) s16x4_t*;
      const char* p = slot + at[i];
      const s16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((P)p);
      const s16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((P)(p + 4 * SIZE * 2));
      const u32x2_t a = __builtin_bit_cast(u32x2_t, lo), b = __builtin_bit_cast(u32x2_t, hi);
      return u32x4_t{a[0], a[1], b[0], b[1]};
    } else {
      return *reinterpret_cast<const u32x4_t*>(slot + at[h] + i * (16 * S::kStep * 2));
    }
  }
};

__device__ __forceinline__ uint32_t uniform(uint32_t v) { return (uint32_t)__builtin_amdgcn_readfirstlane((int)v); }

// N times 1 KiB, 16 bytes a lane, from base + off[i] straight into LDS at byte lds + i * APART; a lane offset of `bytes` or
// more fetches zeros. In assembly, because the compiler waits for every load to LDS it knows of before a transposing read
// (s_waitcnt vmcnt(0) in each part); nothing is returned in registers, and the waits for the data are the explicit ones
// of the loop below. Five wait states stand between a vector instruction that may have written a scalar operand and the
// first load, one between a write of m0 (which nothing else in these kernels uses) and the load.
template <int N, int APART>
__device__ __forceinline__ void load_lds(const void* base, uint32_t bytes, const uint32_t (&off)[N], uint32_t lds) {
  const uint64_t p = reinterpret_cast<uint64_t>(base);
  const u32x4_t r{uniform((uint32_t)p), uniform((uint32_t)(p >> 32) & 0xFFFFu), uniform(bytes), 0x00020000u};
  lds = uniform(lds);
  static_assert(N == 1 || N == 2 || N == 4 || N == 8, "loads of an operand per wave");
  if constexpr (N == 8) {
    const uint32_t lo[4] = {off[0], off[1], off[2], off[3]}, hi[4] = {off[4], off[5], off[6], off[7]};
    load_lds<4, APART>(base, bytes, lo, lds);
    load_lds<4, APART>(base, bytes, hi, lds + 4 * APART);
    return;
  }
  if constexpr (N == 1)
    asm volatile("s_nop 4\n\ts_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds"
                 :
                 : "v"(off[0]), "s"(r), "s"(lds)
                 : "memory");
  else if constexpr (N == 2)
    asm volatile("s_nop 4\n\ts_mov_b32 m0, %3\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %2, 0 offen lds\n\t"
                 "s_add_u32 m0, m0, %4\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
                 :
                 : "v"(off[0]), "v"(off[1]), "s"(r), "s"(lds), "i"(APART)
                 : "memory", "scc");
  else if constexpr (N == 4)
    asm volatile("s_nop 4\n\ts_mov_b32 m0, %5\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %4, 0 offen lds\n\t"
                 "s_add_u32 m0, m0, %6\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %4, 0 offen lds\n\t"
                 "s_add_u32 m0, m0, %6\n\ts_nop 0\n\tbuffer_load_dwordx4 %2, %4, 0 offen lds\n\t"
                 "s_add_u32 m0, m0, %6\n\ts_nop 0\n\tbuffer_load_dwordx4 %3, %4, 0 offen lds"
                 :
                 : "v"(off[0]), "v"(off[1]), "v"(off[2]), "v"(off[3]), "s"(r), "s"(lds), "i"(APART)
                 : "memory", "scc");
}

// What one tile works on. a and b point at the tile's first element, lda, ldb and ldc are elements per row of memory; m
// and n results are left from the tile's first on, `depth` sum steps.
struct Tile {
  const uint16_t* a;
  const uint16_t* b;
  char* c;
  int lda, ldb, ldc, m, n, depth;
};

// Turn p of the loop below waits for what part p + 1 needs, and sends for what goes into the slots that part p used for
// the last time: part p + ring of a slow operand, the pair p / 2 + ring of a fast one behind an odd part. LA, LB loads
// each. What may still be under way behind turn p's wait: the loads sent after the last one that part p + 1 needs.
constexpr int loads_ahead(bool slow_a, int ring_a, int la, bool slow_b, int ring_b, int lb, int parity) {
  const int p = 64 + parity;
  int after = 0;
  for (int q = 0; q < p; ++q) {
    if (slow_a || q % 2 == 1) {
      after += la;
      if (slow_a ? q + ring_a == p + 1 : (q - 1) / 2 + ring_a == (p + 1) / 2) after = 0;
    }
    if (slow_b || q % 2 == 1) {
      after += lb;
      if (slow_b ? q + ring_b == p + 1 : (q - 1) / 2 + ring_b == (p + 1) / 2) after = 0;
    }
  }
  return after;
}

template <int BM, int RA, int RB, bool SLOW_A, bool SLOW_B>
constexpr int kLdsBytes = RA * Side<SLOW_A, BM>::kBytes + RB * Side<SLOW_B, kBN>::kBytes;

template <int BM, int WAVES_M, int WAVES_N, int RA, int RB, bool SLOW_A, bool SLOW_B, bool OUT_BF16>
__device__ __forceinline__ void tile_product(const Tile& t, char* lds) {
  constexpr int kWaves = WAVES_M * WAVES_N;
  using A = Side<SLOW_A, BM>;
  using B = Side<SLOW_B, kBN>;
  constexpr int MF = BM / WAVES_M / 16, NF = kBN / WAVES_N / 16;  // fragments per wave
  constexpr int LA = A::kLoads / kWaves, LB = B::kLoads / kWaves;
  static_assert(A::kLoads % kWaves == 0 && B::kLoads % kWaves == 0, "loads split over the waves");
  constexpr int kAhead[2] = {loads_ahead(SLOW_A, RA, LA, SLOW_B, RB, LB, 0),
                             loads_ahead(SLOW_A, RA, LA, SLOW_B, RB, LB, 1)};
  static_assert(kAhead[0] < 64 && kAhead[1] < 64, "vmcnt counts to 63");
  const int lane = (int)threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)lds;
  const int wm = wave % WAVES_M, wn = wave / WAVES_M;
  const int parts = (t.depth + kPart - 1) / kPart;

  uint32_t off_a[LA], off_b[LB];  // lane offsets of a slot's loads
#pragma unroll
  for (int q = 0; q < LA; ++q) off_a[q] = A::fetch(wave + kWaves * q, lane, t.lda, t.m);
#pragma unroll
  for (int q = 0; q < LB; ++q) off_b[q] = B::fetch(wave + kWaves * q, lane, t.ldb, t.n);
  // Slot number s of an operand (s kStep of the sum before it) -> LDS byte `to`. Steps past the sum's end are zeros on
  // both sides, without a fetch: of a slow operand by the buffer's size, of a fast one by the lane offset.
  auto send = [&](auto side, auto& off, const uint16_t* p, int ld, int s, uint32_t to) {
    using S = typename decltype(side)::type;
    constexpr int n = sizeof(off) / sizeof(off[0]);
    const int left = t.depth - s * S::kStep;
    if constexpr (S::kParts == 1) {
      load_lds<n, kWaves * 1024>(p + (int64_t)s * S::kStep * ld, (uint32_t)max(0, min(S::kStep, left)) * (uint32_t)ld * 2u,
                                 off, to + wave * 1024);
    } else if (left >= S::kStep) {
      load_lds<n, kWaves * 1024>(p + (int64_t)s * S::kStep, kNone, off, to + wave * 1024);
    } else {
      uint32_t part[n];
#pragma unroll
      for (int q = 0; q < n; ++q) part[q] = S::step_of(lane) < left ? off[q] : kNone;
      load_lds<n, kWaves * 1024>(p + (int64_t)s * S::kStep, kNone, part, to + wave * 1024);
    }
  };
  constexpr type_of<A> side_a{};
  constexpr type_of<B> side_b{};
  // Turn p: the slots (by number modulo the ring) that part p leaves, filled again.
  auto refill = [&](int p, int parity, int slot_a, int slot_b) {
    if (SLOW_A || parity == 1)
      send(side_a, off_a, t.a, t.lda, (SLOW_A ? p : (p - 1) / 2) + RA, lds0 + slot_a * A::kBytes);
    if (SLOW_B || parity == 1)
      send(side_b, off_b, t.b, t.ldb, (SLOW_B ? p : (p - 1) / 2) + RB, lds0 + RA * A::kBytes + slot_b * B::kBytes);
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
    auto read = [&](int slot_a, int slot_b, int parity, Frags& f) {
      const char* pa = lds + slot_a * A::kBytes;
      const char* pb = lds + RA * A::kBytes + slot_b * B::kBytes;
      if constexpr (JM > 0) {
#pragma unroll
        for (int j = 0; j < JM; ++j) f.a[j] = ra.read(pa, parity, j);
#pragma unroll
        for (int i = 0; i < NF; ++i) f.b[i] = rb.read(pb, parity, i);
      }
    };
    auto compute = [&](const Frags& f) {
#pragma unroll
      for (int i = 0; i < NF; ++i)
#pragma unroll
        for (int j = 0; j < JM; ++j) acc[i][j] = mfma_bf16(f.b[i], f.a[j], acc[i][j]);
      // one LDS read, then a share of the matrix-core instructions, in turn
      if constexpr (JM > 0) {
        constexpr int kReads = JM * (SLOW_A ? 2 : 1) + NF * (SLOW_B ? 2 : 1);
        constexpr int kEach = (NF * JM) / kReads > 0 ? (NF * JM) / kReads : 1;
#pragma unroll
        for (int q = 0; q < kReads; ++q) {
          __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
          __builtin_amdgcn_sched_group_barrier(0x008, kEach, 0);
        }
      }
    };
    int slot_a = 0, slot_b = 0;  // of the part that is read next
    auto advance = [&](int parity) {
      if (SLOW_A || parity == 1) slot_a = slot_a + 1 == RA ? 0 : slot_a + 1;
      if (SLOW_B || parity == 1) slot_b = slot_b + 1 == RB ? 0 : slot_b + 1;
    };
    // This wave's loads for part p + 1 have landed and its reads of part p are done; behind the barrier every wave's.
    auto meet = [&](auto parity) {
      asm volatile("" ::: "memory");
      __builtin_amdgcn_s_waitcnt(vmcnt_only(kAhead[decltype(parity)::value]));
      __builtin_amdgcn_s_waitcnt(lgkmcnt_only(0));
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
    };
    constexpr std::integral_constant<int, 0> even{};
    constexpr std::integral_constant<int, 1> odd{};
    // the first parts, in the order of the turns that would have sent for them
    constexpr int kFirst = (SLOW_A ? RA : 2 * RA) > (SLOW_B ? RB : 2 * RB) ? (SLOW_A ? RA : 2 * RA) : (SLOW_B ? RB : 2 * RB);
#pragma unroll
    for (int q = -kFirst; q < 0; ++q) {
      if (q == -1) meet(odd);
      if ((SLOW_A || (q & 1)) && (SLOW_A ? q : (q - 1) / 2) + RA >= 0) {
        const int n = (SLOW_A ? q : (q - 1) / 2) + RA;
        send(side_a, off_a, t.a, t.lda, n, lds0 + n * A::kBytes);
      }
      if ((SLOW_B || (q & 1)) && (SLOW_B ? q : (q - 1) / 2) + RB >= 0) {
        const int n = (SLOW_B ? q : (q - 1) / 2) + RB;
        send(side_b, off_b, t.b, t.ldb, n, lds0 + RA * A::kBytes + n * B::kBytes);
      }
    }
    Frags f0, f1;
    read(0, 0, 0, f0);
    int p = 0;
    for (; p + 1 < parts; p += 2) {
      meet(even);
      refill(p, 0, slot_a, slot_b);
      advance(0);
      read(slot_a, slot_b, 1, f1);
      compute(f0);
      meet(odd);
      refill(p + 1, 1, slot_a, slot_b);
      advance(1);
      read(slot_a, slot_b, 0, f0);
      compute(f1);
    }
    if (p < parts) compute(f0);
    __builtin_amdgcn_s_waitcnt(vmcnt_only(0));  // no load to LDS outlives the tile
  };
  static_assert(MF % 4 == 0, "the dispatch below takes quarters");
  const int rows_here = t.m - wm * MF * 16;
  const int quarter = rows_here <= 0 ? 0 : min(4, (rows_here + MF * 4 - 1) / (MF * 4));
  if (parts > 0) switch (quarter) {
    case 0: sum(std::integral_constant<int, 0>{}); break;
    case 1: sum(std::integral_constant<int, MF / 4>{}); break;
    case 2: sum(std::integral_constant<int, MF / 2>{}); break;
    case 3: sum(std::integral_constant<int, MF / 4 * 3>{}); break;
    default: sum(std::integral_constant<int, MF>{}); break;
  }

  // Lane l holds row l % 16 of a fragment and its columns 4 (l / 16) .. + 3. Of fp32 results four lanes then store 64 bytes
  // of a row. Of bf16 results two fragments exchange halves between neighbouring rows of 16 lanes, so that a lane has eight
  // columns, and the tile goes through LDS (16-byte pieces exchanged by an XOR of the row, as above), so that a wave stores
  // whole rows: the lanes' own stores of 64 bytes a row took 1145 us for the weight gradients of 4096 tokens x 6 of 64
  // experts of 4096 x 4096 and 531 for 512 tokens, where the stores are most of the work, whole rows past the caches 1106
  // and 421. (fp32 gains as much where stores are most of the work, 512 tokens of 4096 x 2048 421 and 400, and loses it
  // where they are not, 4096 tokens 716 and 730; it stays as it is.) Weight gradients are read much later; rows are read
  // next and stay in the caches.
  const int g = lane >> 4;
  if constexpr (OUT_BF16) {
    typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
    static_assert(BM * kBN * 2 <= kLdsBytes<BM, RA, RB, SLOW_A, SLOW_B>, "the tile fits where the operands were");
    auto pack = [](float x, float y) { return __builtin_bit_cast(uint32_t, bf16x2_t{(__bf16)x, (__bf16)y}); };
    __syncthreads();  // every wave is done with the operands
#pragma unroll
    for (int j = 0; j < MF; ++j) {
      const int m = (wm * MF + j) * 16 + (lane & 15);
#pragma unroll
      for (int i = 0; i < NF; i += 2) {
        const f32x4_t v = acc[i][j], w = acc[i + 1][j];
        const auto lo = __builtin_amdgcn_permlane16_swap(pack(v[0], v[1]), pack(w[0], w[1]), false, false);
        const auto hi = __builtin_amdgcn_permlane16_swap(pack(v[2], v[3]), pack(w[2], w[3]), false, false);
        const int piece = (wn * NF + i + (g & 1)) * 2 + (g >> 1);
        *reinterpret_cast<u32x4_t*>(lds + m * kBN * 2 + ((piece ^ (m & 15)) << 4)) = u32x4_t{lo[0], hi[0], lo[1], hi[1]};
      }
    }
    __syncthreads();
#pragma unroll 4
    for (int r = 0; r < BM / (2 * kWaves); ++r) {
      const int m = (r * kWaves + wave) * 2 + (lane >> 5), piece = lane & 31;
      const u32x4_t v = *reinterpret_cast<const u32x4_t*>(lds + m * kBN * 2 + ((piece ^ (m & 15)) << 4));
      if (m < t.m && piece * 8 < t.n) {
        u32x4_t* to = reinterpret_cast<u32x4_t*>(t.c + ((size_t)m * t.ldc + piece * 8) * 2);
        if constexpr (SLOW_A) __builtin_nontemporal_store(v, to);
        else *to = v;
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < MF; ++j) {
      const int m = (wm * MF + j) * 16 + (lane & 15);
#pragma unroll
      for (int i = 0; i < NF; ++i) {
        const int n = (wn * NF + i) * 16 + 4 * g;
        if (m < t.m && n < t.n) *reinterpret_cast<f32x4_t*>(t.c + ((size_t)m * t.ldc + n) * 4) = acc[i][j];
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

// The tile of this block among `total`, or -1. The blocks of one XCD (equal block index modulo 8) run 32 at a time, on 32
// consecutive tiles, which share operands in its L2; the next 32 go to the next XCD, so that an expert with many tiles is
// spread over all of them. Fewer than 256 tiles are spread evenly.
constexpr int kRun = 32;
__device__ __forceinline__ int64_t tile_index(int64_t total) {
  const int x = (int)(blockIdx.x & 7), q = (int)(blockIdx.x >> 3);
  const int run = (int)min((int64_t)kRun, (total + 7) / 8), slot = q % kRun;
  const int64_t at = ((int64_t)(q / kRun) * 8 + x) * run + slot;
  return slot < run && at < total ? at : -1;
}
unsigned tile_blocks(int64_t tiles) { return (unsigned)((tiles + 8 * kRun - 1) / (8 * kRun) * 8 * kRun); }

// Place of tile number `left` of `rows` x `cols`: bands of eight rows, in them column by column, so that 32 tiles are
// eight by four (bands of 4 and 16 and runs of 16 and 64 tiles: weight gradients of 16384 tokens 2980, 3040, 3020 and 3110
// us, 2970 so).
__device__ __forceinline__ void tile_place(int left, int rows, int cols, int& m, int& n) {
  const int band = left / (8 * cols), in = left - band * 8 * cols, high = min(8, rows - band * 8);
  m = band * 8 + in % high;
  n = in / high;
}

template <int BM, int WAVES_M, int WAVES_N, int RA, int RB, int OCC, bool TRANSPOSED, bool OUT_BF16>
__global__ __launch_bounds__(64 * WAVES_M * WAVES_N, OCC) void matmul_rows_kernel(
    const uint16_t* __restrict__ a, const uint16_t* __restrict__ w, const int32_t* __restrict__ counts,
    const int32_t* __restrict__ offsets, int E, int rows_max, int K, int N, char* __restrict__ c) {
  constexpr int kThreads = 64 * WAVES_M * WAVES_N;
  __shared__ __attribute__((aligned(1024))) char lds[kLdsBytes<BM, RA, RB, false, !TRANSPOSED>];
  const int depth = TRANSPOSED ? N : K, width = TRANSPOSED ? K : N;
  const int cols = (width + kBN - 1) / kBN;
  // Which expert's tile this is: every thread counts the tiles of a few experts, and one of them finds it among its own.
  struct Found {
    int e, first, rows, m, n;
  };
  int* sums = reinterpret_cast<int*>(lds);
  Found* found = reinterpret_cast<Found*>(lds + 64 * sizeof(int));
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int each = (E + kThreads - 1) / kThreads, e0 = tid * each, e1 = min(E, e0 + each);
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
  int before = s - mine, all = 0;
#pragma unroll
  for (int v = 0; v < kThreads / 64; ++v) {
    before += v < wave ? sums[v] : 0;
    all += sums[v];
  }
  const int64_t index = tile_index((int64_t)all * cols);
  int64_t left = index - (int64_t)before * cols;
  if (index >= 0 && left >= 0 && left < (int64_t)mine * cols)
    for (int e = e0; e < e1; ++e) {
      const int n = group_of(counts, offsets, e, rows_max, first), tiles = (n + BM - 1) / BM;
      if (left < (int64_t)tiles * cols) {
        Found f{e, first, n, 0, 0};
        tile_place((int)left, tiles, cols, f.m, f.n);
        *found = f;
        break;
      }
      left -= (int64_t)tiles * cols;
    }
  __syncthreads();
  const Found f = *found;
  __syncthreads();  // the operands overwrite it
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
  tile_product<BM, WAVES_M, WAVES_N, RA, RB, false, !TRANSPOSED, OUT_BF16>(t, lds);
}

template <int BM, int WAVES_M, int WAVES_N, int RA, int RB, int OCC, bool OUT_BF16>
__global__ __launch_bounds__(64 * WAVES_M * WAVES_N, OCC) void matmul_dw_kernel(
    const uint16_t* __restrict__ a, const uint16_t* __restrict__ dc, const int32_t* __restrict__ counts,
    const int32_t* __restrict__ offsets, int E, int rows_max, int K, int N, char* __restrict__ dw) {
  __shared__ __attribute__((aligned(1024))) char lds[kLdsBytes<BM, RA, RB, true, true>];
  const int rows = (K + BM - 1) / BM, cols = (N + kBN - 1) / kBN;
  const int64_t index = tile_index((int64_t)E * rows * cols);
  if (index < 0) return;
  const int e = (int)(index / (rows * cols));
  int m, n, first;
  tile_place((int)(index - (int64_t)e * (rows * cols)), rows, cols, m, n);
  Tile t;
  t.depth = group_of(counts, offsets, e, rows_max, first);
  if (t.depth == 0) first = 0;
  t.a = a + (size_t)first * K + m * BM;
  t.b = dc + (size_t)first * N + n * kBN;
  t.c = dw + ((size_t)e * K * N + (size_t)m * BM * N + n * kBN) * (OUT_BF16 ? 2 : 4);
  t.lda = K;
  t.ldb = N;
  t.ldc = N;
  t.m = K - m * BM;
  t.n = N - n * kBN;
  tile_product<BM, WAVES_M, WAVES_N, RA, RB, true, true, OUT_BF16>(t, lds);
}

// Rows of a tile. 256 where that leaves work for most CUs (190 tiles, counted as half an empty tile for each expert), less
// where it does not: 1500 tokens x 2 of 8 experts of 2048 x 2048 take 50 us in 256s, 35 in 128s and 40 in 64s, 333 tokens
// 42, 29 and 22, 3000 tokens 52, 67 and 66. Groups of few rows leave most of a large tile empty and read the weights
// alone: up to 8 rows an expert 64s read them as fast or faster (48 tokens x 8 of 128 experts of 2048 x 1536 116 us, 125 in
// 256s; at 12 rows 144 and 141). W^T comes in 128-byte pieces of 256 rows, which more and smaller blocks fetch better: up
// to 32 rows 64s (64 tokens x 6 of 64 experts of 2048 x 4096 174 us, 221 in 128s, 232 in 256s), up to 256 rows 128s (187
// rows 289 us, 354 in 64s, 336 in 256s; at 375 rows 475 and 464).
int tile_rows(bool transposed, int rows_max, int E, int64_t cols) {
  const int mean = rows_max / E;
  const auto enough = [&](int bm) { return cols * std::max(rows_max / bm + E / 2, std::min(E, rows_max)) >= 190; };
  if (mean <= (transposed ? 32 : 8)) return 64;
  if (enough(256) && !(transposed && mean <= 256)) return 256;
  return enough(128) ? 128 : 64;
}

}  // namespace

hipError_t launch_matmul_grouped(const void* a, const void* w, const int32_t* counts, const int32_t* offsets, int E,
                                 int rows_max, int K, int N, bool transposed, void* c, bool out_bf16, hipStream_t s) {
  const auto* pa = static_cast<const uint16_t*>(a);
  const auto* pw = static_cast<const uint16_t*>(w);
  const int64_t cols = ((transposed ? K : N) + kBN - 1) / kBN;
  const auto run = [&](auto kernel, int bm, int threads) {
    const int64_t tiles = (rows_max / bm + std::min(E, rows_max)) * cols;
    hipLaunchKernelGGL(kernel, dim3(tile_blocks(tiles)), dim3(threads), 0, s, pa, pw, counts, offsets, E, rows_max, K, N,
                       static_cast<char*>(c));
  };
  const auto sized = [&](auto t, auto o) {
    constexpr bool T = decltype(t)::value, O = decltype(o)::value;
    // LDS: 80 KiB, two blocks to a CU, for 64 rows; 144 for 128; 128 and, with W^T, 160 for 256
    switch (tile_rows(T, rows_max, E, cols)) {
      case 64: run(matmul_rows_kernel<64, 1, 4, 2, T ? 2 : 4, 2, T, O>, 64, 256); break;
      case 128: run(matmul_rows_kernel<128, 2, 4, 3, T ? 3 : 6, 1, T, O>, 128, 512); break;
      default: run(matmul_rows_kernel<256, 2, 4, 2, T ? 3 : 4, 1, T, O>, 256, 512);
    }
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
    const int64_t tiles = (int64_t)((N + kBN - 1) / kBN) * ((K + bm - 1) / bm) * E;
    hipLaunchKernelGGL(kernel, dim3(tile_blocks(tiles)), dim3(threads), 0, s, pa, pd, counts, offsets, E, rows_max, K, N,
                       static_cast<char*>(dw));
  };
  // 256 rows of dW to a tile, unless the last round of 256 blocks is mostly empty: every tile is as much work as its
  // expert has rows, and 300 tiles take two rounds (333 tokens x 5 of 20 experts of 1280 x 648 19.0 us, 15.8 in 64s; 128
  // tiles of 32 experts of 512 x 512 10.7 and 8.5; 256 tiles of 16 experts of 1024 x 1024 11.4 and 12.6). Long sums are no
  // exception, though 64s read 2.5 times the operands: 4096 rows for each of 8 experts of 1536 x 1536 (288 tiles) 198 us
  // in 256s and 195 in 64s, of 1024 x 1024 (128 tiles) 93 and 88, 20 experts of 1280 x 648 with 1024 rows each 59 and 52.
  const int64_t tiles = (int64_t)((N + kBN - 1) / kBN) * ((K + 255) / 256) * E;
  if (10 * tiles >= 7 * ((tiles + 255) / 256 * 256))
    out_bf16 ? run(matmul_dw_kernel<256, 2, 4, 4, 4, 1, true>, 256, 512)
             : run(matmul_dw_kernel<256, 2, 4, 4, 4, 1, false>, 256, 512);
  else
    out_bf16 ? run(matmul_dw_kernel<64, 1, 4, 4, 4, 2, true>, 64, 256)
             : run(matmul_dw_kernel<64, 1, 4, 4, 4, 2, false>, 64, 256);
  return hipGetLastError();
}

}  // namespace moe
