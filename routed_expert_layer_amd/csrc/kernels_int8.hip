// Experts in 8-bit integers, a scale per token on one side and per output
// channel on the other (MOE_W_INT8).
//
//   sx = max|x| / 127 over a token,  xq = rne(127 x / max|x|)
//   g = (xq W1) sx s1,  u = (xq W3) sx s3,  h = silu(g) u
//   sh, hq = the same of a row of h,  y = (hq W2) sh s2
//
// The integer products run on v_mfma_i32_16x16x64_i8 and are exact (32-bit
// sums: |sum| <= 127^2 K, so K may reach 133000). A 16 x 64 operand fragment
// is 1 KiB, as a 16 x 32 fragment in bf16 is, so the blobs, the streaming of
// weights in decode steps and the staging of prefill tiles have the same byte
// geometry as the bf16 experts at half the K.
//
// A row's scale needs the whole row of h, which no tile of the gate/up product
// holds: h goes to memory in fp32 (a rounding to 16 bits here would move one
// code in some hundreds by a step, more than all other roundings together)
// and the down projection's side turns it into codes: decode blocks for
// themselves, prefill in a pass of its own between the products.
#include <algorithm>
#include <cstring>

#include "dev_common.hpp"
#include "gemm_common.hpp"
#include "int8_layout.hpp"
#include "moe_kernels.hpp"
#include "row_quant.hpp"

namespace moe {
namespace {

using i32x4_t = int32_t __attribute__((ext_vector_type(4)));

__device__ __forceinline__ i32x4_t mfma_i8(u32x4_t a, u32x4_t b, i32x4_t c) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4_t, a), __builtin_bit_cast(i32x4_t, b), c, 0, 0,
                                               0);
}

// silu(g) u for g, u three roundings off already, which move it by 3 (1 + |g|) + 3
// half steps of 2^-24 at most: the hardware's exponential and reciprocal (a step
// each; the exponent's argument carries |g| half steps) add 1.5 |g| + 5. The
// tests count both where a code is near a half. (expf and a division moved as many
// codes and cost 1 to 3%: 4096 tokens x 6 of 256 experts of 4096 x 2048 1467 us
// a call, not 1453, 16384 x 6 of 64 3250, not 3155.)
__device__ __forceinline__ float swiglu(float g, float u) {
  return g * __builtin_amdgcn_rcpf(1.0f + __expf(-g)) * u;
}

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) {
    const uint32_t o = __shfl_xor(v, d, 64);
    v = o > v ? o : v;
  }
  return v;
}

// One wave: the codes and the scale of a row of K bf16 values (K a multiple
// of 16). NC: 16-value pieces a lane keeps in registers (K <= 1024 NC).
template <int NC>
__device__ __forceinline__ void quantise_row(const uint16_t* __restrict__ row, int K, uint8_t* __restrict__ codes,
                                             float* __restrict__ scale, int lane) {
  const int pieces = K / 16;
  u32x4_t raw[NC][2];
  uint32_t m = 0;
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int p = lane + 64 * c;
    raw[c][0] = raw[c][1] = u32x4_t{0u, 0u, 0u, 0u};
    if (p < pieces) {
      raw[c][0] = ld16(row + (size_t)p * 16);
      raw[c][1] = ld16(row + (size_t)p * 16 + 8);
    }
  }
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const uint32_t lo = (raw[c][q][w] << 16) & 0x7FFFFFFFu, hi = raw[c][q][w] & 0x7FFF0000u;
        m = lo > m ? lo : m;
        m = hi > m ? hi : m;
      }
  const RowQuant rq(wave_max_u32(m));
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int p = lane + 64 * c;
    if (p < pieces) {
      u32x4_t o;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const uint32_t a = raw[c][w >> 1][2 * (w & 1)], b = raw[c][w >> 1][2 * (w & 1) + 1];
        o[w] = rq.pack4<true>(__uint_as_float(a << 16), __uint_as_float(a & 0xFFFF0000u), __uint_as_float(b << 16),
                              __uint_as_float(b & 0xFFFF0000u));
      }
      *reinterpret_cast<u32x4_t*>(codes + (size_t)p * 16) = o;
    }
  }
  if (lane == 0) *scale = rq.scale();
}

// Where a launch finds its work items {slot, row_begin, rows, expert}: in the kernel arguments or in device memory
// (*n of them, the grid sized for the most there can be).
struct ArgItems {
  WorkArgs wa;
  __device__ __forceinline__ bool get(int i, int4& it) const {
    it = wa.item[i];
    return true;
  }
};
struct DevItems {
  const int32_t* n;
  const int4* items;
  __device__ __forceinline__ int count() const { return *n; }
  __device__ __forceinline__ bool get(int i, int4& it) const {
    if (i >= *n) return false;
    const int4 v = items[i];
    it = make_int4(__builtin_amdgcn_readfirstlane(v.x), __builtin_amdgcn_readfirstlane(v.y),
                   __builtin_amdgcn_readfirstlane(v.z), __builtin_amdgcn_readfirstlane(v.w));
    return true;
  }
};

// What a layer's kernels run over, planned by one block of 256 threads from a
// routing's counts and offsets, or from a listed group a thread. Groups that
// reach past rows_max and experts without a slot are left out.
//   tile_rows 0: decode, the groups with rows as items {slot, row_begin, rows,
//     expert}, in ascending order, and their number;
//   else: prefill, an entry for each tile of tile_rows rows, and their number.
//     Up to kSuper tiles of a group make a super-row; an entry is {slot, first
//     row of the super-row, its rows, tiles in it | this one's index << 8}.
// At most `cap` are written, however the counts overlap.
constexpr int kSuper = 8;
struct Plan {
  const int32_t *counts, *offsets, *slot_of;
  int E, n_slots, rows_max, tile_rows, cap;
  int32_t* n;  // nullptr: no plan
  int4* items;
  uint32_t* zero;  // `zeros` words are cleared besides
  int zeros;
};

// Thread's group `it` of a list of 256 (`base` entries before it); returns the new number of entries. E, lds: LDS.
__device__ __forceinline__ int plan_groups(int4 it, bool ok, int base, int tile_rows, int cap, int4* items,
                                           int (*lds)[256], int4* group) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int mine = !ok ? 0 : tile_rows ? (it.z + tile_rows - 1) / tile_rows : 1;
  int x = mine;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(x, d, 64);
    if (lane >= d) x += o;
  }
  if (lane == 63) lds[0][wave] = x;
  __syncthreads();
  int before = 0, all = 0;
  for (int w = 0; w < 4; ++w) {
    before += w < wave ? lds[0][w] : 0;
    all += lds[0][w];
  }
  lds[1][tid] = before + x;  // inclusive
  group[tid] = it;
  __syncthreads();
  for (int q = tid; q < min(all, cap - base); q += 256) {
    int lo = 0, hi = 255;  // the group of entry q: the first whose inclusive count is above q
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (lds[1][mid] > q) hi = mid; else lo = mid + 1;
    }
    const int4 g = group[lo];
    int4 e = g;
    if (tile_rows) {
      const int tiles = (g.z + tile_rows - 1) / tile_rows, t = q - (lds[1][lo] - tiles), s0 = t / kSuper * kSuper;
      const int in = min(kSuper, tiles - s0);
      e = make_int4(g.x, g.y + s0 * tile_rows, min(g.z - s0 * tile_rows, kSuper * tile_rows), in | (t - s0) << 8);
    }
    items[base + q] = e;
  }
  __syncthreads();
  return min(base + all, cap);
}

__device__ __forceinline__ void run_plan(const Plan& p) {
  for (int q = threadIdx.x; q < p.zeros; q += 256) p.zero[q] = 0u;
  __shared__ int lds[2][256];
  __shared__ int4 group[256];
  int base = 0;
  for (int e0 = 0; e0 < p.E; e0 += 256) {
    const int e = e0 + (int)threadIdx.x;
    int4 it = make_int4(0, 0, 0, e);
    bool ok = false;
    if (e < p.E) {
      it.z = p.counts[e];
      it.y = p.offsets[e];
      it.x = p.slot_of ? p.slot_of[e] : e;
      ok = it.z > 0 && it.y >= 0 && (long long)it.y + it.z <= p.rows_max && it.x >= 0 && it.x < p.n_slots;
    }
    base = plan_groups(it, ok, base, p.tile_rows, p.cap, p.items, lds, group);
  }
  if (threadIdx.x == 0) *p.n = base;
}

// Prefill entries of up to kMaxItems groups listed on the host.
__global__ __launch_bounds__(256) void plan_list(const ArgItems wk, int tile_rows, int cap, int32_t* __restrict__ n,
                                                 int4* __restrict__ items) {
  __shared__ int lds[2][256];
  __shared__ int4 group[256];
  const bool ok = (int)threadIdx.x < wk.wa.n;
  const int all = plan_groups(ok ? wk.wa.item[threadIdx.x] : make_int4(0, 0, 0, 0), ok, 0, tile_rows, cap, items, lds, group);
  if (threadIdx.x == 0) *n = all;
}

// T token rows to codes, four rows a block (one a wave); with a plan, block 0
// plans the layer's work items instead. Bound by memory: 2 bytes in, 1 out
// (16384 rows of 4096 33.5 us, 6.0 TB/s).
template <int NC>
__global__ __launch_bounds__(256) void quantise_tokens(const uint16_t* __restrict__ x, int T, int H,
                                                       uint8_t* __restrict__ xq, float* __restrict__ sx,
                                                       const Plan plan) {
  int block = blockIdx.x;
  if (plan.n != nullptr) {
    if (block == 0) {
      run_plan(plan);
      return;
    }
    --block;
  }
  const int r = block * 4 + (threadIdx.x >> 6);
  if (r < T) quantise_row<NC>(x + (size_t)r * H, H, xq + (size_t)r * H, sx + r, threadIdx.x & 63);
}

// The rows of listed work items through perm_src: grouped row r of xq and sx.
template <int NC>
__global__ __launch_bounds__(256) void quantise_items(const uint16_t* __restrict__ x,
                                                      const int32_t* __restrict__ perm_src, const ArgItems wk, int H,
                                                      uint8_t* __restrict__ xq, float* __restrict__ sx) {
  int4 it;
  if (!wk.get(blockIdx.y, it)) return;
  const int m = blockIdx.x * 4 + (threadIdx.x >> 6);
  if (m >= it.z) return;
  const size_t r = (size_t)(it.y + m);
  quantise_row<NC>(x + (size_t)perm_src[r] * H, H, xq + r * H, sx + r, threadIdx.x & 63);
}

// ---------------------------------------------------------------------------
// Packing: fragment order as in the bf16 blobs, 16 K bytes a lane.
// ---------------------------------------------------------------------------
__global__ __launch_bounds__(256) void pack_int8_kernel(const int8_t* __restrict__ Q1, const int8_t* __restrict__ Q3,
                                                        const int8_t* __restrict__ Q2, const float* __restrict__ S1,
                                                        const float* __restrict__ S3, const float* __restrict__ S2,
                                                        int H, int I, char* __restrict__ blob, const Int8Layout L) {
  const size_t q = (size_t)blockIdx.x * 256 + threadIdx.x;
  const int KC1 = H / 64, KC2 = I / 64;
  const size_t c1 = (size_t)(2 * I / 16) * KC1 * 64, c2 = (size_t)(H / 16) * KC2 * 64;
  union {
    int8_t b[16];
    uint4 v;
  } o;
  if (q < c1) {
    const int l = (int)(q % 64), c = (int)((q / 64) % KC1), t = (int)(q / (64 * (size_t)KC1));
    int mat, i;
    p1_row_source(16 * t + (l % 16), mat, i);
    const int8_t* Q = mat ? Q3 : Q1;
    const int k0 = 64 * c + 16 * (l / 16);
    for (int j = 0; j < 16; ++j) o.b[j] = Q[(size_t)(k0 + j) * I + i];
    *reinterpret_cast<uint4*>(blob + L.p1 + q * 16) = o.v;
    return;
  }
  size_t r = q - c1;
  if (r < c2) {
    const int l = (int)(r % 64), c = (int)((r / 64) % KC2), t = (int)(r / (64 * (size_t)KC2));
    const int n = 16 * t + (l % 16);
    for (int j = 0; j < 16; ++j) o.b[j] = Q2[(size_t)int8_k2_source(c, l / 16, j) * H + n];
    *reinterpret_cast<uint4*>(blob + L.p2 + r * 16) = o.v;
    return;
  }
  r -= c2;
  if (r < (size_t)2 * I) {
    int mat, i;
    p1_row_source((int)r, mat, i);
    reinterpret_cast<float*>(blob + L.p1s)[r] = mat ? S3[i] : S1[i];
    return;
  }
  r -= (size_t)2 * I;
  if (r < (size_t)H) reinterpret_cast<float*>(blob + L.p2s)[r] = S2[r];
}

// ---------------------------------------------------------------------------
// Decode: every weight byte is read once, straight from memory into matrix
// instructions whose other operand holds up to 16 tokens' codes. Bound by the
// weights' bytes: 8 tokens x 6 of 64 experts of 4096 x 2048 (28 chosen) 71 us
// in gate/up and 38 in down, 6.5 TB/s; one token 18.5 and 13.3 us, 5.4 and 3.8.
// ---------------------------------------------------------------------------
// A wave's fragments [c0, c1) of a 16-row tile, 1 KiB apart. Up to NF of them
// are held: loaded before anything that they wait for (a down projection's
// codes), and used again for every 16 rows of a group, so weights are read
// once however long the group is. Past NF (MORE) they are streamed, kStream in
// flight.
constexpr int kStream = 8;
template <int NF, bool MORE>
struct Held {
  u32x4_t a[NF];
  int n;  // fragments held: the first n
  __device__ __forceinline__ void load(const char* wp, int c0, int c1) {
    n = min(NF, c1 - c0);
    if (n == NF) {
#pragma unroll
      for (int u = 0; u < NF; ++u) a[u] = ld16_nt(wp + (size_t)(c0 + u) * 1024);
    } else {
#pragma unroll
      for (int u = 0; u < NF; ++u) {
        a[u] = u32x4_t{0u, 0u, 0u, 0u};
        if (u < n) a[u] = ld16_nt(wp + (size_t)(c0 + u) * 1024);
      }
    }
  }
  // the sum over all of [c0, c1) times the token fragments bload(c)
  template <typename BLoad>
  __device__ __forceinline__ i32x4_t dot(const char* wp, int c0, int c1, BLoad bload) const {
    i32x4_t acc = {0, 0, 0, 0};
#pragma unroll
    for (int u0 = 0; u0 < NF; u0 += kStream) {
      u32x4_t b[kStream];
#pragma unroll
      for (int u = 0; u < kStream; ++u)
        if (u0 + u < NF) b[u] = bload(min(c0 + u0 + u, c1 - 1));  // past n: against zeros
#pragma unroll
      for (int u = 0; u < kStream; ++u)
        if (u0 + u < NF) acc = mfma_i8(a[u0 + u], b[u], acc);
    }
    if constexpr (!MORE) return acc;
    for (int c = c0 + NF; c < c1; c += kStream) {
      u32x4_t w[kStream], b[kStream];
#pragma unroll
      for (int u = 0; u < kStream; ++u) {
        const int cu = min(c + u, c1 - 1);
        w[u] = ld16_nt(wp + (size_t)cu * 1024);
        b[u] = bload(cu);
        if (c + u >= c1) b[u] = u32x4_t{0u, 0u, 0u, 0u};
      }
#pragma unroll
      for (int u = 0; u < kStream; ++u) acc = mfma_i8(w[u], b[u], acc);
    }
    return acc;
  }
};

// Gate/up: a block is one 16-row tile of P1 (8 gate and 8 up columns) of an
// item, its four waves splitting K. src: the token of each grouped row
// (nullptr: xq holds the grouped rows). h: fp32, row-major.
template <typename W, int NF, bool MORE>
__global__ __launch_bounds__(256) void int8_decode_up(const uint8_t* __restrict__ xq, const float* __restrict__ sx,
                                                      const int32_t* __restrict__ src, const W wk,
                                                      const char* __restrict__ slot_base, size_t slot_stride,
                                                      const Int8Layout L, int H, int I, float* __restrict__ h) {
  const int NT = I / 8;
  const int item = blockIdx.x / NT, tile = blockIdx.x - item * NT;
  int4 it;
  if (!wk.get(item, it)) return;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6)), lane = threadIdx.x & 63;
  const int KC = H / 64, c0 = (KC * wave) >> 2, c1 = (KC * (wave + 1)) >> 2;
  const char* blob = slot_base + (size_t)it.x * slot_stride;
  const char* wp = blob + L.p1 + (size_t)tile * KC * 1024 + lane * 16;
  Held<NF, MORE> w;
  w.load(wp, c0, c1);
  __shared__ i32x4_t red[4][64];
  for (int m0 = 0; m0 < it.z; m0 += 16) {
    const int m = m0 + (lane & 15);
    const bool valid = m < it.z;
    // lanes past the group read its first row again: their columns are not stored
    const int r = it.y + (valid ? m : 0), t = src ? src[r] : r;
    const uint8_t* xr = xq + (size_t)t * H + 16 * (lane >> 4);
    red[wave][lane] = c0 < c1 ? w.dot(wp, c0, c1, [&](int c) { return ld16(xr + (size_t)c * 64); }) : i32x4_t{0, 0, 0, 0};
    __syncthreads();
    if (wave == 0 && valid) {
      const i32x4_t s = red[0][lane] + red[1][lane] + red[2][lane] + red[3][lane];
      const f32x4_t sw = *reinterpret_cast<const f32x4_t*>(blob + L.p1s + (size_t)(16 * tile + 4 * (lane >> 4)) * 4);
      const float st = sx[t];
      const float g0 = (float)s[0] * (st * sw[0]), u0 = (float)s[1] * (st * sw[1]);
      const float g1 = (float)s[2] * (st * sw[2]), u1 = (float)s[3] * (st * sw[3]);
      *reinterpret_cast<float2*>(h + (size_t)r * I + 8 * tile + 2 * (lane >> 4)) =
          make_float2(swiglu(g0, u0), swiglu(g1, u1));
    }
    __syncthreads();
  }
}

// Four columns of row m's codes into LDS in the order of P2's K (int8_k2_source): fragment c at 1024 c, lane (column
// group, row) at 16 bytes each, columns 2q and 2q + 1 of every 8 beside each other.
__device__ __forceinline__ void put_h_codes(char* lds, int m, int col, const RowQuant& rq, const f32x4_t& v) {
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    const int c = col + 2 * p;
    *reinterpret_cast<uint16_t*>(lds + (c >> 6) * 1024 + (((c >> 1) & 3) * 16 + m) * 16 + 2 * ((c >> 3) & 7)) =
        (uint16_t)rq.pack2<false>(v[2 * p], v[2 * p + 1]);
  }
}

// The codes of rows [r0, r0 + n) of h (n <= 16) into LDS by a block of 256
// threads: a row's maximum over the block, then its codes, kQuantRows rows at a
// time in registers (rows of up to 1024 P; longer ones are read twice). Columns
// of rows past n are left as they are: they are other tokens' columns of the
// products, which are not stored. mx: LDS of 16 x 4 words.
constexpr int kQuantRows = 4;
template <int P>
__device__ __forceinline__ void quantise_h_rows(const float* __restrict__ h, int r0, int n, int I, char* lds,
                                                float* scales, uint32_t (*mx)[4]) {
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  for (int m0 = 0; m0 < n; m0 += kQuantRows) {
    f32x4_t v[kQuantRows][P];
#pragma unroll
    for (int r = 0; r < kQuantRows; ++r) {
      const float* row = h + (size_t)(r0 + m0 + r) * I;
#pragma unroll
      for (int p = 0; p < P; ++p) {
        const int i = 4 * tid + 1024 * p;
        v[r][p] = f32x4_t{0.f, 0.f, 0.f, 0.f};
        if (m0 + r < n && i < I) v[r][p] = *reinterpret_cast<const f32x4_t*>(row + i);
      }
    }
#pragma unroll
    for (int r = 0; r < kQuantRows; ++r) {
      if (m0 + r >= n) break;
      uint32_t m = 0;
#pragma unroll
      for (int p = 0; p < P; ++p)
#pragma unroll
        for (int w = 0; w < 4; ++w) m = max(m, abs_bits(v[r][p][w]));
      if (I > 1024 * P) {
        const float* row = h + (size_t)(r0 + m0 + r) * I;
        for (int i = 4 * tid + 1024 * P; i < I; i += 1024) {
          const f32x4_t q = *reinterpret_cast<const f32x4_t*>(row + i);
#pragma unroll
          for (int w = 0; w < 4; ++w) m = max(m, abs_bits(q[w]));
        }
      }
      m = wave_max_u32(m);
      if (lane == 0) mx[m0 + r][wave] = m;
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kQuantRows; ++r) {
      if (m0 + r >= n) break;
      const RowQuant rq(max(max(mx[m0 + r][0], mx[m0 + r][1]), max(mx[m0 + r][2], mx[m0 + r][3])));
#pragma unroll
      for (int p = 0; p < P; ++p)
        if (4 * tid + 1024 * p < I) put_h_codes(lds, m0 + r, 4 * tid + 1024 * p, rq, v[r][p]);
      if (I > 1024 * P) {
        const float* row = h + (size_t)(r0 + m0 + r) * I;
        for (int i = 4 * tid + 1024 * P; i < I; i += 1024)
          put_h_codes(lds, m0 + r, i, rq, *reinterpret_cast<const f32x4_t*>(row + i));
      }
      if (tid == 0) scales[m0 + r] = rq.scale();
    }
  }
}

// A float of y to or from other blocks of the same launch: at device scope (sc1), whichever XCDs they are on. base:
// wave-uniform, p within 2^32 bytes above it.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t device_rows(const float* base) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<float*>(base), (short)0, -1, 0x00020000);
}
__device__ __forceinline__ f32x4_t device_load4(const float* base, const float* p) {
  return __builtin_bit_cast(f32x4_t, __builtin_amdgcn_raw_buffer_load_b128(
                                         device_rows(base), (uint32_t)((const char*)p - (const char*)base), 0, 16));
}
__device__ __forceinline__ void device_store4(float* base, float* p, const f32x4_t& v) {
  __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, v), device_rows(base),
                                         (uint32_t)((char*)p - (char*)base), 0, 16);
}

// What a short step's down projection forms its output from: each block, once
// its part of y is stored, counts itself at its columns (`done`, zeroed by the
// launch before), and the one that comes last there adds the tokens' rows up in
// the combine's order, so the result does not depend on which block that is;
// no block waits for another. Saves a launch, but y goes past the L2s and the
// last blocks work alone, so up to kSumRows rows only. Calls in us, without /
// with: one token x 6 of 64 experts of 4096 x 2048 36.4 / 34.9, 4 x 6 85.5 /
// 85.0, 8 x 6 117 / 118; 4 x 2 of 96 of 1024 x 512 19.0 / 16.0, 16 x 2 19.2 /
// 20.8; 4 x 8 of 128 of 2048 x 768 31.2 / 32.9.
constexpr int kSumRows = 24;
struct SumArgs {
  const int32_t *topk_idx, *perm_pos, *slot_of;
  const float* topk_w;
  int T, k, n_slots;
  void* out;
  int out_bf16;
  uint32_t* done;  // [H / (16 R)]
};

template <int COLS>
__device__ __forceinline__ void sum_columns(const SumArgs& f, const float* y, int H, int col0) {
  for (int q = threadIdx.x; q < f.T * (COLS / 4); q += 256) {
    const int t = q / (COLS / 4), col = col0 + 4 * (q - t * (COLS / 4));
    f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
    for (int j0 = 0; j0 < f.k; j0 += 8) {
      f32x4_t v[8];
      float w[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        w[u] = 0.f;
        v[u] = f32x4_t{0.f, 0.f, 0.f, 0.f};
        if (j0 + u >= f.k) continue;
        const int e = f.topk_idx[t * f.k + j0 + u];
        const int slot = f.slot_of ? f.slot_of[e] : e;
        if (slot < 0 || slot >= f.n_slots) continue;
        w[u] = f.topk_w[t * f.k + j0 + u];
        v[u] = device_load4(y, y + (size_t)f.perm_pos[t * f.k + j0 + u] * H + col);
      }
#pragma unroll
      for (int u = 0; u < 8; ++u)
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[c] = fmaf(w[u], v[u][c], acc[c]);
    }
    if (f.out_bf16)
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(f.out) + (size_t)t * H + col) =
          make_uint2(bf16_bits(acc[0]) | bf16_bits(acc[1]) << 16, bf16_bits(acc[2]) | bf16_bits(acc[3]) << 16);
    else
      *reinterpret_cast<f32x4_t*>(static_cast<float*>(f.out) + (size_t)t * H + col) = acc;
  }
}

// Down projection: a block is R 16-row tiles of P2 (16 R output columns) of an
// item; it forms the codes of the item's rows of h itself, while its weights
// are on their way.
template <typename W, int NF, bool MORE, int R, bool SUM>
__global__ __launch_bounds__(256) void int8_decode_down(const float* __restrict__ h, const W wk,
                                                        const char* __restrict__ slot_base, size_t slot_stride,
                                                        const Int8Layout L, int H, int I, float* y, const SumArgs f) {
  const int NB = H / (16 * R);
  const int item = blockIdx.x / NB, tile0 = (blockIdx.x - item * NB) * R;
  int4 it;
  if (!wk.get(item, it)) {
    if constexpr (SUM)
      if (item == 0) sum_columns<16 * R>(f, y, H, 16 * tile0);  // no expert of the step has a slot: zeros
    return;
  }
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6)), lane = threadIdx.x & 63;
  const int KC = I / 64, c0 = (KC * wave) >> 2, c1 = (KC * (wave + 1)) >> 2;
  const char* blob = slot_base + (size_t)it.x * slot_stride;
  const char* wp = blob + L.p2 + (size_t)tile0 * KC * 1024 + lane * 16;
  Held<NF, MORE> w[R];
#pragma unroll
  for (int t = 0; t < R; ++t) w[t].load(wp + (size_t)t * KC * 1024, c0, c1);
  extern __shared__ __attribute__((aligned(16))) char codes[];  // 16 rows of I bytes
  __shared__ i32x4_t red[4][R][64];
  __shared__ float sh[16];
  __shared__ uint32_t mx[16][4];
  for (int m0 = 0; m0 < it.z; m0 += 16) {
    quantise_h_rows<(NF > 4 ? 2 : 1)>(h, it.y + m0, min(16, it.z - m0), I, codes, sh, mx);
    __syncthreads();
#pragma unroll
    for (int t = 0; t < R; ++t)
      red[wave][t][lane] = c0 < c1 ? w[t].dot(wp + (size_t)t * KC * 1024, c0, c1,
                                              [&](int c) { return ld16(codes + (size_t)c * 1024 + lane * 16); })
                                   : i32x4_t{0, 0, 0, 0};
    __syncthreads();
    const int m = m0 + (lane & 15);
    if (wave < R && m < it.z) {
      const i32x4_t s = red[0][wave][lane] + red[1][wave][lane] + red[2][wave][lane] + red[3][wave][lane];
      const int n0 = 16 * (tile0 + wave) + 4 * (lane >> 4);
      const f32x4_t sw = *reinterpret_cast<const f32x4_t*>(blob + L.p2s + (size_t)n0 * 4);
      const float st = sh[lane & 15];
      f32x4_t o;
#pragma unroll
      for (int c = 0; c < 4; ++c) o[c] = (float)s[c] * (st * sw[c]);
      float* row = y + (size_t)(it.y + m) * H + n0;
      if constexpr (SUM)
        device_store4(y, row, o);
      else
        *reinterpret_cast<f32x4_t*>(row) = o;
    }
    __syncthreads();
  }
  if constexpr (SUM) {
    __shared__ int last;
    __builtin_amdgcn_s_waitcnt(0);  // this wave's stores have completed
    __syncthreads();                // ... and every wave's
    if (threadIdx.x == 0)
      last = __hip_atomic_fetch_add(f.done + tile0 / R, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) + 1u ==
             (uint32_t)wk.count();
    __syncthreads();
    if (last) sum_columns<16 * R>(f, y, H, 16 * tile0);
  }
}

// ---------------------------------------------------------------------------
// Prefill: grouped GEMM, 16 BN_T weight rows x 16 BM_T tokens a block and 64 of
// K a stage, both operands straight into LDS in fragment order; eight waves of
// 32 x 64 (128 x 128), 64 x 64 (256 x 128) or 128 x 64 (256 x 256).
// Short groups are bound by the weights' bytes (4096 tokens x 6 of 256 experts
// of 4096 x 2048: 862 + 462 us, 5.0 TB/s), long ones by the operands' way
// through L2 and the matrix cores together (16384 x 6 of 64: 1577 + 1017 us,
// 1908 TOPS, the cores busy for 53 and 41% of the cycles; the products without
// their loads 1.7 ms, the loads without the products 2.2).
// ---------------------------------------------------------------------------
// h of prefill: 16-row tiles, 8 columns a piece, the two columns of a lane
// together: the gate/up product's store of a fragment is 512 contiguous bytes
// and lane (q, row) of the pass below reads what it wrote.
__device__ __forceinline__ size_t h_tile_at(size_t row, int piece, int q, int I) {
  return ((row >> 4) * (size_t)(I / 8) + piece) * 128 + (q * 16 + (row & 15)) * 2;
}

// Tile t of the launch: entry t / NTB's super-row, in which the tiles go in
// groups of kGroupN weight tiles over all its token tiles, so that the blocks
// that run together on an XCD share 8 x 4 tiles' operands in its L2.
constexpr int kGroupN = 4;

// PHASE 1: gate/up from tokens' codes (rows through src) to h, tiled as above.
// PHASE 2: the down projection from h's codes to fp32 rows of y, as the decode
// kernels leave them: a token's rows may cancel, and what fewer bits take from
// them is then no longer below the rounding of their sum. (fp16 rows with a
// factor each, for bf16 outputs, made 16384 tokens x 6 of 64 experts of 4096 x
// 2048 2.93 ms, not 3.15, but lost 2^-12 of the rows: 9e-4 relative on mixed
// inputs, all of the sum where rows cancel.)
template <int PHASE, int BM_T, int BN_T = 16>
__global__ __launch_bounds__(512, 1) void int8_gemm(const uint8_t* __restrict__ bsrc, const float* __restrict__ bscale,
                                                    const int32_t* __restrict__ src, const int32_t* __restrict__ n_entries,
                                                    const int4* __restrict__ entries,
                                                    const char* __restrict__ slot_base, size_t slot_stride,
                                                    size_t mat_off, size_t scale_off, int N, int K, int H, int I,
                                                    float* __restrict__ hout, float* __restrict__ yout) {
  // stages: 128 KiB for one block a CU, or 64 and 72 KiB for two (with 6, so one block a CU, 2048 tokens x 4 of 90
  // experts of 1024 x 512 took 69.7 us, not 63.4, 8192 x 6 of 256 of 4096 x 2048 2212, not 2101)
  constexpr int NS = BM_T == 16 || BN_T == 8 ? 4 : 3;
  constexpr int WN = BN_T * BM_T / 32;
  constexpr int WM = 4;
  constexpr int WAVES_N = BN_T / WN;
  static_assert(WAVES_N * (BM_T / WM) == 8, "wave grid");
  constexpr int FA = BN_T, FB = BM_T;
  constexpr int FPW = (FA + FB) / 8;
  constexpr int STAGE = (FA + FB) * 1024;
  __shared__ __attribute__((aligned(1024))) char lds[NS][STAGE];

  // an eighth of the tiles for each XCD (blocks b with the same b % 8), in order
  const int NTB = (N / 16 + BN_T - 1) / BN_T, last = N / 16 - 1, total = *n_entries * NTB, share = (total + 7) / 8;
  const int in_share = (int)(blockIdx.x >> 3), t = (int)(blockIdx.x & 7) * share + in_share;
  if (in_share >= share || t >= total) return;
  const int ent = t / NTB;
  const int4 en = entries[ent];
  const int gm = en.w & 0xFF;
  const int li = (en.w >> 8) * NTB + (t - ent * NTB);
  const int whole = NTB / kGroupN * kGroupN * gm;  // tiles in whole groups of weight tiles
  const int width = li < whole ? kGroupN : NTB % kGroupN, lg = li < whole ? li : li - whole;
  const int ng = lg / (gm * width), rem = lg - ng * gm * width;
  const int mt = rem / width, nt = (li < whole ? ng * kGroupN : NTB / kGroupN * kGroupN) + rem % width;
  const int4 it = make_int4(__builtin_amdgcn_readfirstlane(en.x), __builtin_amdgcn_readfirstlane(en.y),
                            __builtin_amdgcn_readfirstlane(en.z), 0);
  const int tid = (int)threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int wn = wave % WAVES_N, wm = wave / WAVES_N;
  const int KC = K / 64;
  const char* blob = slot_base + (size_t)it.x * slot_stride;
  const char* wbase = blob + mat_off;

  constexpr int QW = FA / 8;  // weight fragments a wave loads per stage; the others are token fragments
  uint32_t off[FPW], kstep[FPW];
#pragma unroll
  for (int q = 0; q < FPW; ++q) {
    const int f = wave + 8 * q;
    if (q < QW) {
      off[q] = (uint32_t)(min(nt * BN_T + f, last) * KC) * 1024u + lane * 16;  // past N: not stored
      kstep[q] = 1024;
    } else {
      int mloc = mt * (16 * BM_T) + (f - FA) * 16 + (lane & 15);
      if (mloc >= it.z) mloc = it.z - 1;  // a valid row; its columns are not stored
      if constexpr (PHASE == 2) {
        const uint32_t row = (uint32_t)(it.y + mloc);
        off[q] = (row >> 4) * (uint32_t)KC * 1024u + ((row & 15) + 16 * (lane >> 4)) * 16;
        kstep[q] = 1024;
      } else {
        const uint32_t row = (uint32_t)(src ? src[it.y + mloc] : it.y + mloc);
        off[q] = row * (uint32_t)H + (lane >> 4) * 16;
        kstep[q] = 64;
      }
    }
  }
  auto issue = [&](int stage, int buf) {
    char* base = lds[buf];
#pragma unroll
    for (int q = 0; q < FPW; ++q)
      buffer_load_lds16(q < QW ? static_cast<const void*>(wbase) : static_cast<const void*>(bsrc),
                        off[q] + (uint32_t)stage * kstep[q], base + (wave + 8 * q) * 1024);
  };

  i32x4_t acc[WN][WM];
#pragma unroll
  for (int i = 0; i < WN; ++i)
#pragma unroll
    for (int j = 0; j < WM; ++j) acc[i][j] = i32x4_t{0, 0, 0, 0};
  struct Frags {
    u32x4_t a[WN], b[WM];
  };
  // JM: this wave's token fragments that hold rows of the group
  auto k_loop = [&](auto jm_const) {
    constexpr int JM = decltype(jm_const)::value;
    auto read_stage = [&](int kt, Frags& f) {
      const char* b = lds[kt % NS];
#pragma unroll
      for (int j = 0; j < JM; ++j) f.b[j] = ld16(b + (FA + wm * WM + j) * 1024 + lane * 16);
      if constexpr (JM > 0) {
#pragma unroll
        for (int i = 0; i < WN; ++i) f.a[i] = ld16(b + (wn * WN + i) * 1024 + lane * 16);
      }
    };
    auto compute = [&](const Frags& f) {
#pragma unroll
      for (int i = 0; i < WN; ++i)
#pragma unroll
        for (int j = 0; j < JM; ++j) acc[i][j] = mfma_i8(f.a[i], f.b[j], acc[i][j]);
    };
    // step kt computes on stage kt's registers while it reads stage kt + 1's fragments; after its barrier every
    // wave has finished reading stage kt, whose buffer is then refilled with stage kt + NS
    auto step = [&](int kt, Frags& cur, Frags& nxt) {
      if (kt + NS - 1 < KC) {
        __builtin_amdgcn_s_waitcnt(vmcnt_only(FPW * (NS - 2)));
      } else {
        __builtin_amdgcn_s_waitcnt(vmcnt_only(0));
      }
      __builtin_amdgcn_s_waitcnt(lgkmcnt_only(0));
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
      if (kt + NS < KC) issue(kt + NS, kt % NS);
      read_stage(min(kt + 1, KC - 1), nxt);
      compute(cur);
      if constexpr (JM > 0) {
#pragma unroll
        for (int q = 0; q < WN + JM; ++q) {
          __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
          __builtin_amdgcn_sched_group_barrier(0x008, (WN * JM) / (WN + JM), 0);
        }
      }
    };
    for (int s0 = 0; s0 < NS && s0 < KC; ++s0) issue(s0, s0);
    if (KC >= NS) {
      __builtin_amdgcn_s_waitcnt(vmcnt_only(FPW * (NS - 1)));
    } else {
      __builtin_amdgcn_s_waitcnt(vmcnt_only(0));
    }
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    Frags f0, f1;
    read_stage(0, f0);
    int kt = 0;
    for (; kt + 1 < KC; kt += 2) {
      step(kt, f0, f1);
      step(kt + 1, f1, f0);
    }
    if (kt < KC) step(kt, f0, f1);
  };
  static_assert(WM == 4, "the dispatch below covers 0 .. 4 fragments");
  const int rows_here = it.z - (mt * 16 * BM_T + wm * WM * 16);
  const int jm = rows_here <= 0 ? 0 : min(WM, (rows_here + 15) / 16);
  switch (jm) {
    case 0: k_loop(std::integral_constant<int, 0>{}); break;
    case 1: k_loop(std::integral_constant<int, 1>{}); break;
    case 2: k_loop(std::integral_constant<int, 2>{}); break;
    case 3: k_loop(std::integral_constant<int, 3>{}); break;
    default: k_loop(std::integral_constant<int, 4>{}); break;
  }

  const float* wscale = reinterpret_cast<const float*>(blob + scale_off);
  // every scale first, so that their loads are in flight together
  f32x4_t sw[WN];
#pragma unroll
  for (int i = 0; i < WN; ++i)
    sw[i] = *reinterpret_cast<const f32x4_t*>(wscale + 16 * min(nt * BN_T + wn * WN + i, last) + 4 * (lane >> 4));
  float st[WM];
#pragma unroll
  for (int j = 0; j < WM; ++j) {
    const int mloc = mt * (16 * BM_T) + (wm * WM + j) * 16 + (lane & 15);
    const size_t row = (size_t)(it.y + min(mloc, it.z - 1));
    st[j] = bscale[(PHASE == 1 && src) ? (size_t)src[row] : row];
  }
#pragma unroll
  for (int j = 0; j < WM; ++j) {
    const int mloc = mt * (16 * BM_T) + (wm * WM + j) * 16 + (lane & 15);
    if (mloc >= it.z) continue;
    const size_t row = (size_t)(it.y + mloc);
#pragma unroll
    for (int i = 0; i < WN; ++i) {
      const int ntile = nt * BN_T + wn * WN + i;
      if (ntile > last) break;
      const i32x4_t s = acc[i][j];
      f32x4_t v;
#pragma unroll
      for (int c = 0; c < 4; ++c) v[c] = (float)s[c] * (st[j] * sw[i][c]);
      if constexpr (PHASE == 1)
        *reinterpret_cast<float2*>(hout + h_tile_at(row, ntile, lane >> 4, I)) =
            make_float2(swiglu(v[0], v[1]), swiglu(v[2], v[3]));
      else
        *reinterpret_cast<f32x4_t*>(yout + row * H + 16 * ntile + 4 * (lane >> 4)) = v;
    }
  }
}

// h to codes between the products: a block is one 16-row tile; lane (q, row)
// of a wave reads its two columns of each of a 64-wide piece's eight 8-wide
// parts and has the 16 code bytes of its place in the token fragment (the
// order P2 is packed in, int8_k2_source). Up to kHeld pieces a wave stay in
// registers between the row maximum and the codes; wider rows are read again.
// Bound by memory: 98304 rows of 2048 183 us, 5.5 TB/s.
constexpr int kHeld = 4, kReqWaves = 8;
__global__ __launch_bounds__(64 * kReqWaves) void requantise_h(const float* __restrict__ h, int I,
                                                               uint8_t* __restrict__ hq, float* __restrict__ sh) {
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const size_t tile = blockIdx.x;
  const int pieces = I / 64;
  const float* base = h + tile * 16 * (size_t)I + lane * 2;
  __shared__ uint32_t mx[kReqWaves][16];
  float2 v[kHeld][8];
  uint32_t m = 0;
  auto load = [&](int c, float2 (&o)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = *reinterpret_cast<const float2*>(base + (size_t)(8 * c + j) * 128);
  };
  auto take = [&](const float2 (&o)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, max(abs_bits(o[j].x), abs_bits(o[j].y)));
  };
#pragma unroll
  for (int u = 0; u < kHeld; ++u)
    if (wave + kReqWaves * u < pieces) {
      load(wave + kReqWaves * u, v[u]);
      take(v[u]);
    }
  for (int c = wave + kReqWaves * kHeld; c < pieces; c += kReqWaves) {
    float2 o[8];
    load(c, o);
    take(o);
  }
  m = max(m, (uint32_t)__shfl_xor((int)m, 16, 64));
  m = max(m, (uint32_t)__shfl_xor((int)m, 32, 64));
  if (lane < 16) mx[wave][lane] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kReqWaves; ++w) m = max(m, mx[w][lane & 15]);
  const RowQuant rq(m);
  auto store = [&](int c, const float2 (&o)[8]) {
    u32x4_t b;
#pragma unroll
    for (int w = 0; w < 4; ++w) b[w] = rq.pack4<false>(o[2 * w].x, o[2 * w].y, o[2 * w + 1].x, o[2 * w + 1].y);
    *reinterpret_cast<u32x4_t*>(hq + (tile * pieces + c) * 1024 + lane * 16) = b;
  };
#pragma unroll
  for (int u = 0; u < kHeld; ++u)
    if (wave + kReqWaves * u < pieces) store(wave + kReqWaves * u, v[u]);
  for (int c = wave + kReqWaves * kHeld; c < pieces; c += kReqWaves) {
    float2 o[8];
    load(c, o);
    store(c, o);
  }
  if (wave == 0 && lane < 16) sh[tile * 16 + lane] = rq.scale();
}

// out[t] = sum over j of w[t, j] y[pos[t, j]], j ascending, over the experts that have a slot.
// A thread takes 8 columns, all of a token's rows in flight together (up to kAhead of them).
// Bound by memory: 16384 tokens x 6 rows of 4096 371 us, 4.7 TB/s.
constexpr int kAhead = 8;
template <bool OUT_BF16, bool UNIFORM>
__global__ __launch_bounds__(256) void int8_combine(const float* __restrict__ y, const int32_t* __restrict__ perm_pos,
                                                    const int32_t* __restrict__ topk_idx,
                                                    const float* __restrict__ topk_w,
                                                    const int32_t* __restrict__ slot_of, int n_slots, int k, int H,
                                                    int T, void* __restrict__ out) {
  const int per = H / 8;  // threads a token; a block may hold several tokens, or a part of one
  const size_t id = (size_t)blockIdx.x * 256 + threadIdx.x;
  size_t t = id / per;
  const int n = (int)(id - t * per) * 8;
  if constexpr (UNIFORM) t = (size_t)__builtin_amdgcn_readfirstlane((int)t);  // a wave is within one token: scalar loads
  if (t >= (size_t)T) return;
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int j0 = 0; j0 < k; j0 += kAhead) {
    f32x4_t v[kAhead][2];
    float w[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      w[u] = 0.f;
      v[u][0] = v[u][1] = f32x4_t{0.f, 0.f, 0.f, 0.f};
      if (j0 + u >= k) continue;
      const int e = topk_idx[t * k + j0 + u];
      const int slot = slot_of ? slot_of[e] : e;
      if (slot < 0 || slot >= n_slots) continue;
      const float* row = y + (size_t)perm_pos[t * k + j0 + u] * H + n;
      w[u] = topk_w[t * k + j0 + u];
      v[u][0] = *reinterpret_cast<const f32x4_t*>(row);
      v[u][1] = *reinterpret_cast<const f32x4_t*>(row + 4);
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (j0 + u < k) {
#pragma unroll
        for (int c = 0; c < 8; ++c) acc[c] = fmaf(w[u], v[u][c >> 2][c & 3], acc[c]);
      }
  }
  if constexpr (OUT_BF16) {
    u32x4_t o;
#pragma unroll
    for (int c = 0; c < 4; ++c) o[c] = bf16_bits(acc[2 * c]) | bf16_bits(acc[2 * c + 1]) << 16;
    *reinterpret_cast<u32x4_t*>(static_cast<uint16_t*>(out) + t * H + n) = o;
  } else {
    float* o = static_cast<float*>(out) + t * H + n;
    *reinterpret_cast<f32x4_t*>(o) = f32x4_t{acc[0], acc[1], acc[2], acc[3]};
    *reinterpret_cast<f32x4_t*>(o + 4) = f32x4_t{acc[4], acc[5], acc[6], acc[7]};
  }
}

hipError_t launch_quantise_tokens(const uint16_t* x, int T, int H, uint8_t* xq, float* sx, const Plan& plan,
                                  hipStream_t s) {
  const dim3 grid((T + 3) / 4 + (plan.n != nullptr ? 1 : 0));
  if (H <= 1024) hipLaunchKernelGGL(quantise_tokens<1>, grid, dim3(256), 0, s, x, T, H, xq, sx, plan);
  else if (H <= 2048) hipLaunchKernelGGL(quantise_tokens<2>, grid, dim3(256), 0, s, x, T, H, xq, sx, plan);
  else if (H <= 4096) hipLaunchKernelGGL(quantise_tokens<4>, grid, dim3(256), 0, s, x, T, H, xq, sx, plan);
  else if (H <= 8192) hipLaunchKernelGGL(quantise_tokens<8>, grid, dim3(256), 0, s, x, T, H, xq, sx, plan);
  else hipLaunchKernelGGL(quantise_tokens<16>, grid, dim3(256), 0, s, x, T, H, xq, sx, plan);
  return hipGetLastError();
}

template <typename W, int NF, bool MORE>
hipError_t decode_down(const W& wk, int n_items, const char* slot_base, size_t slot_stride, int H, int I,
                       const float* h, float* y, const SumArgs* sum, hipStream_t s) {
  constexpr int R = 2;  // H is a multiple of 64
  const auto run = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3(n_items * (H / (16 * R))), dim3(256), (size_t)16 * I, s, h, wk, slot_base,
                       slot_stride, int8_layout(H, I), H, I, y, sum != nullptr ? *sum : SumArgs{});
    return hipGetLastError();
  };
  if constexpr (std::is_same_v<W, DevItems>)
    if (sum != nullptr) return run(int8_decode_down<W, NF, MORE, R, true>);
  return run(int8_decode_down<W, NF, MORE, R, false>);
}

template <typename W>
hipError_t decode_products(const W& wk, int n_items, const uint8_t* xq, const float* sx, const int32_t* src,
                           const char* slot_base, size_t slot_stride, int H, int I, float* h, float* y,
                           hipStream_t s, const SumArgs* sum = nullptr) {
  const Int8Layout L = int8_layout(H, I);
  const auto up = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3(n_items * (I / 8)), dim3(256), 0, s, xq, sx, src, wk, slot_base, slot_stride, L, H,
                       I, h);
  };
  // Held fragments a wave: a quarter of K / 64, up to 8. (H 4096: 16 held took 40 us a token's call and 128 us of eight
  // tokens, 8 held and 8 streamed 37.5 and 121, having more waves resident.)
  if (H <= 1024) up(int8_decode_up<W, 4, false>);
  else if (H <= 2048) up(int8_decode_up<W, 8, false>);
  else up(int8_decode_up<W, 8, true>);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (I <= 1024) return decode_down<W, 4, false>(wk, n_items, slot_base, slot_stride, H, I, h, y, sum, s);
  if (I <= 2048) return decode_down<W, 8, false>(wk, n_items, slot_base, slot_stride, H, I, h, y, sum, s);
  return decode_down<W, 8, true>(wk, n_items, slot_base, slot_stride, H, I, h, y, sum, s);
}

// Rows a prefill tile holds: 256 when groups have 384 on average, else 128, of which two blocks fit on a CU. Calls in us,
// 128 / 256 rows: 16 experts of 2048 x 768 with 256 rows each 59 / 68 (most groups need a second tile then), 8 of
// 3968 x 1920 with 256 78 / 100, with 512 150 / 128; 64 of 4096 x 2048 with 384 922 / 895, with 768 1745 / 1640.
int tile_rows_for(int rows, int groups) { return (long long)rows >= 384ll * groups ? 256 : 128; }

// The two products and the pass between them over planned entries (at most rows / tile + groups).
hipError_t gemm_products(const uint8_t* xq, const float* sx, const int32_t* src, int rows, int groups, int tile_rows,
                         const int32_t* n, const int4* entries, const char* slot_base, size_t slot_stride, int H, int I,
                         float* h, uint8_t* hq, float* sh, float* y, hipStream_t s) {
  const Int8Layout L = int8_layout(H, I);
  const size_t most = rows / tile_rows + groups;  // entries
  // Less than a block a CU: 128 weight rows a block, twice the blocks (a call of 333 tokens x 5 of 20 experts of
  // 1280 x 640 39.5 -> 34.4 us; with blocks for 256 to 1024, 64 x 8 of 128 experts of 2048 x 768, 113 -> 115 us).
  const auto narrow = [&](int N) { return tile_rows == 128 && most * ((N + 255) / 256) < 256; };
  const auto product = [&](auto kernel, int columns, int N, int K, const uint8_t* b, const float* bs,
                           const int32_t* from, size_t mat, size_t scales) {
    const dim3 grid((unsigned)((most * ((N + columns - 1) / columns) + 7) / 8 * 8));
    hipLaunchKernelGGL(kernel, grid, dim3(512), 0, s, b, bs, from, n, entries, slot_base, slot_stride, mat, scales, N,
                       K, H, I, h, y);
    return hipGetLastError();
  };
  const auto up = [&](auto kernel, int columns) {
    return product(kernel, columns, 2 * I, H, xq, sx, src, L.p1, L.p1s);
  };
  const auto down = [&](auto kernel, int columns) {
    return product(kernel, columns, H, I, hq, sh, nullptr, L.p2, L.p2s);
  };
  hipError_t e = tile_rows == 256 ? up(int8_gemm<1, 16>, 256)
                 : narrow(2 * I)  ? up(int8_gemm<1, 8, 8>, 128)
                                  : up(int8_gemm<1, 8>, 256);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(requantise_h, dim3((rows + 15) / 16), dim3(64 * kReqWaves), 0, s, h, I, hq, sh);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  return tile_rows == 256 ? down(int8_gemm<2, 16>, 256)
         : narrow(H)      ? down(int8_gemm<2, 8, 8>, 128)
                          : down(int8_gemm<2, 8>, 256);
}

}  // namespace

hipError_t launch_pack_int8(int H, int I, const void* Q1, const void* Q3, const void* Q2, const void* S1,
                            const void* S3, const void* S2, void* blob, hipStream_t s) {
  const Int8Layout L = int8_layout(H, I);
  const size_t n = (size_t)(2 * I / 16) * (H / 64) * 64 + (size_t)(H / 16) * (I / 64) * 64 + (size_t)2 * I + H;
  hipLaunchKernelGGL(pack_int8_kernel, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, s,
                     static_cast<const int8_t*>(Q1), static_cast<const int8_t*>(Q3), static_cast<const int8_t*>(Q2),
                     static_cast<const float*>(S1), static_cast<const float*>(S3), static_cast<const float*>(S2), H, I,
                     static_cast<char*>(blob), L);
  return hipGetLastError();
}

hipError_t launch_ffn_int8_list(const void* x, const int32_t* perm_src, const int4* items, int n, int rows_total,
                                bool gemm, const char* slot_base, size_t slot_stride, int H, int I, float* y, void* ws,
                                hipStream_t s) {
  if (n <= 0) return hipSuccess;
  const Int8Ws w = int8_ws(rows_total, rows_total, H, I);
  char* b = static_cast<char*>(ws);
  uint8_t* xq = reinterpret_cast<uint8_t*>(b + w.xq);
  float *sx = reinterpret_cast<float*>(b + w.sx), *h = reinterpret_cast<float*>(b + w.h);
  const uint16_t* xb = static_cast<const uint16_t*>(x);
  WorkArgs wa;
  for (int base = 0; base < n; base += kMaxItems) {
    std::memset(&wa, 0, sizeof wa);
    wa.n = std::min(kMaxItems, n - base);
    int most = 0, rows = 0;
    for (int i = 0; i < wa.n; ++i) {
      wa.item[i] = items[base + i];
      most = std::max(most, wa.item[i].z);
      rows += wa.item[i].z;
    }
    const dim3 grid((most + 3) / 4, wa.n);
    const ArgItems wk{wa};
    if (H <= 1024) hipLaunchKernelGGL(quantise_items<1>, grid, dim3(256), 0, s, xb, perm_src, wk, H, xq, sx);
    else if (H <= 2048) hipLaunchKernelGGL(quantise_items<2>, grid, dim3(256), 0, s, xb, perm_src, wk, H, xq, sx);
    else if (H <= 4096) hipLaunchKernelGGL(quantise_items<4>, grid, dim3(256), 0, s, xb, perm_src, wk, H, xq, sx);
    else if (H <= 8192) hipLaunchKernelGGL(quantise_items<8>, grid, dim3(256), 0, s, xb, perm_src, wk, H, xq, sx);
    else hipLaunchKernelGGL(quantise_items<16>, grid, dim3(256), 0, s, xb, perm_src, wk, H, xq, sx);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (!gemm) {
      e = decode_products(wk, wa.n, xq, sx, nullptr, slot_base, slot_stride, H, I, h, y, s);
    } else {
      const int tile = tile_rows_for(rows, wa.n);
      int32_t* count = reinterpret_cast<int32_t*>(b + w.plan);
      int4* entries = reinterpret_cast<int4*>(b + w.plan + 256);
      hipLaunchKernelGGL(plan_list, dim3(1), dim3(256), 0, s, wk, tile, w.entries, count, entries);
      if ((e = hipGetLastError()) == hipSuccess)
        // rows_total: the pass between the products covers every row of the workspace, listed or not
        e = gemm_products(xq, sx, nullptr, rows_total, wa.n, tile, count, entries, slot_base, slot_stride, H, I, h,
                          reinterpret_cast<uint8_t*>(b + w.hq), reinterpret_cast<float*>(b + w.sh), y, s);
    }
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_ffn_int8_dev(const void* x, int T, const int32_t* perm_src, const int32_t* n_items,
                               const int4* items, int max_items, int rows_total, const char* slot_base,
                               size_t slot_stride, int H, int I, float* y, void* ws, hipStream_t s) {
  if (max_items <= 0 || T <= 0) return hipSuccess;
  const Int8Ws w = int8_ws(rows_total, rows_total, H, I);
  char* b = static_cast<char*>(ws);
  uint8_t* xq = reinterpret_cast<uint8_t*>(b + w.xq);
  float* sx = reinterpret_cast<float*>(b + w.sx);
  hipError_t e = launch_quantise_tokens(static_cast<const uint16_t*>(x), T, H, xq, sx, Plan{}, s);
  if (e != hipSuccess) return e;
  return decode_products(DevItems{n_items, items}, max_items, xq, sx, perm_src, slot_base, slot_stride, H, I,
                         reinterpret_cast<float*>(b + w.h), y, s);
}

hipError_t launch_experts_int8(const void* x, int T, int k, int E, const int32_t* topk_idx, const float* topk_w,
                               const int32_t* perm_src, const int32_t* perm_pos, const int32_t* counts,
                               const int32_t* offsets, const int32_t* slot_of, int n_slots, const char* slot_base,
                               size_t slot_stride, int H, int I, void* out, bool out_bf16, void* ws, float* y,
                               hipStream_t s) {
  if (T <= 0) return hipSuccess;
  const int rows = T * k;
  const Int8Ws w = int8_ws(rows, T, H, I);
  char* b = static_cast<char*>(ws);
  uint8_t* xq = reinterpret_cast<uint8_t*>(b + w.xq);
  float *sx = reinterpret_cast<float*>(b + w.sx), *h = reinterpret_cast<float*>(b + w.h);
  const uint16_t* xb = static_cast<const uint16_t*>(x);
  const bool gemm = int8_gemm_supported(H, I) && int8_gemm_pays(rows, E);
  const int groups = std::min(E, rows), tile = gemm ? tile_rows_for(rows, groups) : 0;
  int32_t* n = reinterpret_cast<int32_t*>(b + w.plan);
  int4* entries = reinterpret_cast<int4*>(b + w.plan + 256);
  const bool sums = !gemm && rows <= kSumRows;
  uint32_t* done = reinterpret_cast<uint32_t*>(b + w.done);
  hipError_t e = launch_quantise_tokens(xb, T, H, xq, sx,
                                        Plan{counts, offsets, slot_of, E, n_slots, rows, tile, w.entries, n, entries, done,
                                             sums ? H / 32 : 0},
                                        s);
  if (e != hipSuccess) return e;
  if (sums) {
    const SumArgs f{topk_idx, perm_pos, slot_of, topk_w, T, k, n_slots, out, (int)out_bf16, done};
    return decode_products(DevItems{n, entries}, groups, xq, sx, perm_src, slot_base, slot_stride, H, I, h, y, s, &f);
  }
  if (gemm)
    e = gemm_products(xq, sx, perm_src, rows, groups, tile, n, entries, slot_base, slot_stride, H, I, h,
                      reinterpret_cast<uint8_t*>(b + w.hq), reinterpret_cast<float*>(b + w.sh), y, s);
  else
    e = decode_products(DevItems{n, entries}, groups, xq, sx, perm_src, slot_base, slot_stride, H, I, h, y, s);
  if (e != hipSuccess) return e;
  const dim3 grid((unsigned)(((size_t)T * (H / 8) + 255) / 256));
  const auto combine = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, dim3(256), 0, s, y, perm_pos, topk_idx, topk_w, slot_of, n_slots, k, H, T, out);
    return hipGetLastError();
  };
  if (!out_bf16) return combine(int8_combine<false, false>);
  return gemm && H % 512 == 0 ? combine(int8_combine<true, true>) : combine(int8_combine<true, false>);
}

}  // namespace moe
