// Selection of experts from given logits (or from the router products'
// partial sums) under a gate, and the grouping of the rows by expert.
//
// Up to 64 tokens: one block does all. Up to kFewTokens: two launches, blocks
// of 16 to 64 tokens that choose and count their choices by expert (one byte
// an expert), then blocks of 64 tokens that add the counts up, each for
// itself, and place their rows. Longer batches add the counts up in a launch
// of its own (each block reading every count would be the longer way: 512
// chunks x 256 experts are 128 KiB a block). Captured calls in us, one block / two launches: 32 tokens of 128 experts 10.6
// / 12.5, 64 13.2 / 12.5, 64 of 64 experts 8.4 / 9.7; two / three: 16384 of 64 14.0 / 17.9, of 256 30.3 / 35.3.
#include "dev_common.hpp"
#include "dev_select.hpp"
#include "moe_kernels.hpp"

namespace moe {
namespace {

constexpr int kOneBlock = 64, kFewTokens = 16384;
constexpr int kMaxTokensPerBlock = 64;

// Where a token's logits come from: nsplit slabs of partial sums, `slab`
// floats apart, added in order, plus a bias; nsplit 1 and no bias for logits
// as given. The sums go to `keep` when it is set.
struct LogitSource {
  const float* p;
  int nsplit;
  size_t slab;
  const float* bias;
  float* keep;
  __device__ __forceinline__ void load(int t, int E, int lane, float* lds) const {
    for (int e = lane; e < E; e += 64) {
      const size_t at = (size_t)t * E + e;
      float x = p[at];
      for (int z = 1; z < nsplit; ++z) x += p[(size_t)z * slab + at];
      if (bias) x += bias[e];
      if (keep) keep[at] = x;
      lds[e] = x;
    }
  }
};

// A block's LDS: 16 waves' logits, the balance, then the masks of the block's tokens by expert.
inline size_t select_lds(int E) { return (size_t)16 * E * 4 + align_up((size_t)E * 4, 16) + (size_t)E * 8; }
struct SelectLds {
  float *logits, *balance;
  unsigned long long* masks;
  __device__ __forceinline__ SelectLds(char* base, int E, int wave) {
    logits = reinterpret_cast<float*>(base) + (size_t)wave * E;
    balance = reinterpret_cast<float*>(base) + (size_t)16 * E;
    masks = reinterpret_cast<unsigned long long*>(base + (size_t)16 * E * 4 + (((size_t)E * 4 + 15) & ~(size_t)15));
  }
};

// Exclusive prefix over a block of 1024 threads of v; `wsum` is LDS of 16 ints.
__device__ __forceinline__ int block_prefix(int v, int* wsum) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int x = v;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int n = __shfl_up(x, d, 64);
    if (lane >= d) x += n;
  }
  if (lane == 63) wsum[wave] = x;
  __syncthreads();
  int before = 0;
  for (int w = 0; w < wave; ++w) before += wsum[w];
  return before + x - v;
}

// Blocks of `chunk` tokens (16 waves, one token at a time each): the choice and the weights, and the masks in LDS.
template <int VE>
__device__ __forceinline__ void choose(const LogitSource& src, const GateArgs& g, int lanes, int t0, int n, int E,
                                       int k, int32_t* __restrict__ topk_idx, float* __restrict__ topk_w,
                                       const SelectLds& s) {
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int per = E / g.n_group;
  for (int e = threadIdx.x; e < E; e += 1024) {
    s.masks[e] = 0ull;
    if (g.balance != nullptr) s.balance[e] = g.balance[e];
  }
  if (wave < n) src.load(t0 + wave, E, lane, s.logits);
  __syncthreads();
  for (int i = wave; i < n; i += 16) {
    const size_t t = (size_t)(t0 + i);
    int e, at;
    float w;
    select_token<VE>(s.logits, g.balance != nullptr ? s.balance : nullptr, per, k, g, lanes, lane, e, w, at);
    if (i + 16 < n) {  // the wave's own logits: its LDS accesses are in order
      __builtin_amdgcn_wave_barrier();
      src.load(t0 + i + 16, E, lane, s.logits);
      __builtin_amdgcn_wave_barrier();
    }
    if (lane < k) {
      topk_idx[t * k + at] = e;
      topk_w[t * k + at] = w;
      atomicOr(&s.masks[e], 1ull << i);
    }
  }
  __syncthreads();
}

// The same with a row of 16 lanes a token, RVE experts a lane: wave w takes tokens 4 w .. 4 w + 3. Tokens that 32-bit
// scores do not decide go through select_token, one after another.
template <int VE, int RVE>
__device__ __forceinline__ void choose_rows(const float* __restrict__ logits, const GateArgs& g, int lanes,
                                            int row_lanes, int t0, int n, int E, int k, int32_t* __restrict__ topk_idx,
                                            float* __restrict__ topk_w, const SelectLds& s) {
  __shared__ int pick[16][64];
  __shared__ double score[16][64];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int per = E / g.n_group;
  // a row past the end repeats the last token, and writes nothing
  const int i = min(4 * wave + (lane >> 4), n - 1);
  const bool here = 4 * wave + (lane >> 4) < n;
  const size_t t = (size_t)(t0 + i);
  float l[RVE];
  load_row<RVE>(logits + t * E, ((reinterpret_cast<uintptr_t>(logits) & 15) | (E & 3) | (per & 3)) == 0, per, g.n_group,
                row_lanes, lane, l);
  for (int e = threadIdx.x; e < E; e += blockDim.x) {
    s.masks[e] = 0ull;
    if (g.balance != nullptr) s.balance[e] = fmaxf(g.balance[e], -INFINITY);  // a NaN is -inf
  }
  __syncthreads();
  const float* bal = g.balance != nullptr ? s.balance : nullptr;
  if (4 * wave < n) {
    int e, at;
    float w;
    const bool sure = select_row<RVE>(l, logits + t * E, bal, per, k, g, row_lanes, lane, pick[wave], score[wave], e, w,
                                      at);
    if (sure && here && (lane & 15) < k) {
      topk_idx[t * k + at] = e;
      topk_w[t * k + at] = w;
      atomicOr(&s.masks[e], 1ull << i);
    }
    uint64_t again = __ballot(!sure && here);
    while (again) {  // uniform
      const int j = 4 * wave + ((__ffsll((unsigned long long)again) - 1) >> 4);
      again &= ~(0xFFFFull << (16 * (j - 4 * wave)));
      const size_t tj = (size_t)(t0 + j);
      __builtin_amdgcn_wave_barrier();
      for (int q = lane; q < E; q += 64) s.logits[q] = logits[tj * E + q];
      __builtin_amdgcn_wave_barrier();
      select_token<VE>(s.logits, bal, per, k, g, lanes, lane, e, w, at);
      if (lane < k) {
        topk_idx[tj * k + at] = e;
        topk_w[tj * k + at] = w;
        atomicOr(&s.masks[e], 1ull << j);
      }
    }
  }
  __syncthreads();
}

// Each selection's row: its expert's offset, the expert's rows of earlier chunks (in `first`), earlier tokens here.
__device__ __forceinline__ void place(const int32_t* topk_idx, int t0, int n, int k, const int* first,
                                      const unsigned long long* masks, int32_t* __restrict__ perm_src,
                                      int32_t* __restrict__ perm_pos) {
  for (int i = threadIdx.x; i < n * k; i += 1024) {
    const int tl = i / k;
    const int e = topk_idx[(size_t)t0 * k + i];
    const int pos = first[e] + __popcll(masks[e] & ((1ull << tl) - 1ull));
    perm_pos[(size_t)t0 * k + i] = pos;
    perm_src[pos] = t0 + tl;
  }
}

template <int VE, int RVE>
__global__ __launch_bounds__(1024) void select_one_block(const LogitSource src, const GateArgs g, int lanes,
                                                         int row_lanes, int T, int E, int k, int32_t* topk_idx, float* __restrict__ topk_w,
                                                         int32_t* __restrict__ counts, int32_t* __restrict__ offsets,
                                                         int32_t* __restrict__ perm_src,
                                                         int32_t* __restrict__ perm_pos,
                                                         int32_t* __restrict__ counts_mirror) {
  extern __shared__ __attribute__((aligned(16))) char base[];
  __shared__ int wsum[16];
  const SelectLds s(base, E, threadIdx.x >> 6);
  if constexpr (RVE > 0)
    choose_rows<VE, RVE>(src.p, g, lanes, row_lanes, 0, T, E, k, topk_idx, topk_w, s);
  else
    choose<VE>(src, g, lanes, 0, T, E, k, topk_idx, topk_w, s);
  const int e = threadIdx.x;
  const int c = e < E ? __popcll(s.masks[e]) : 0;
  const int at = block_prefix(c, wsum);
  int* first = reinterpret_cast<int*>(base);  // over the logits, which are done with
  if (e < E) {
    counts[e] = c;
    if (counts_mirror) counts_mirror[e] = c;
    offsets[e] = at;
    first[e] = at;
  }
  if (e == 0) offsets[E] = T * k;
  __syncthreads();
  place(topk_idx, 0, T, k, first, s.masks, perm_src, perm_pos);
}

template <int VE, int RVE>
__global__ __launch_bounds__(1024) void select_chunk(const LogitSource src, const GateArgs g, int lanes, int row_lanes,
                                                     int T, int E, int k, int chunk, int32_t* __restrict__ topk_idx,
                                                     float* __restrict__ topk_w, uint8_t* __restrict__ few,
                                                     uint64_t* __restrict__ bits, int32_t* __restrict__ hist) {
  extern __shared__ __attribute__((aligned(16))) char base[];
  const SelectLds s(base, E, threadIdx.x >> 6);
  const int t0 = blockIdx.x * chunk;
  if constexpr (RVE > 0)
    choose_rows<VE, RVE>(src.p, g, lanes, row_lanes, t0, min(chunk, T - t0), E, k, topk_idx, topk_w, s);
  else
    choose<VE>(src, g, lanes, t0, min(chunk, T - t0), E, k, topk_idx, topk_w, s);
  if (few != nullptr) {
    // counts as bytes, experts padded to a multiple of 4
    const int words = (E + 3) / 4;
    for (int q = threadIdx.x; q < words; q += blockDim.x) {
      uint32_t v = 0;
      for (int b = 0; b < 4; ++b)
        if (4 * q + b < E) v |= (uint32_t)__popcll(s.masks[4 * q + b]) << (8 * b);
      reinterpret_cast<uint32_t*>(few)[(size_t)blockIdx.x * words + q] = v;
    }
  } else {
    for (int e = threadIdx.x; e < E; e += blockDim.x) {
      bits[(size_t)blockIdx.x * E + e] = s.masks[e];
      hist[(size_t)e * gridDim.x + blockIdx.x] = __popcll(s.masks[e]);
    }
  }
}

// The second launch for up to kFewTokens tokens: a block of 64 tokens adds up every chunk's counts (its 16 waves a part
// of the chunks each), all of them for the offsets and those before its first chunk c for its own rows.
__global__ __launch_bounds__(1024) void place_chunk(const int32_t* topk_idx, int T, int E, int k, int chunk,
                                                    int chunks, const uint8_t* __restrict__ few, int32_t* __restrict__ counts,
                                                    int32_t* __restrict__ offsets, int32_t* __restrict__ perm_src,
                                                    int32_t* __restrict__ perm_pos,
                                                    int32_t* __restrict__ counts_mirror) {
  extern __shared__ __attribute__((aligned(16))) char base[];
  __shared__ int wsum[16];
  const int words = (E + 3) / 4;
  unsigned long long* masks = reinterpret_cast<unsigned long long*>(base);  // [E]
  int* first = reinterpret_cast<int*>(base + (size_t)E * 8);                // [4 words]: rows of earlier chunks
  int* total = first + 4 * words;                                           // [4 words]
  const int t0 = blockIdx.x * kMaxTokensPerBlock, n = min(kMaxTokensPerBlock, T - t0), c = t0 / chunk;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  for (int e = threadIdx.x; e < E; e += 1024) masks[e] = 0ull;
  for (int e = threadIdx.x; e < 8 * words; e += 1024) first[e] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < n * k; i += 1024)
    atomicOr(&masks[topk_idx[(size_t)t0 * k + i]], 1ull << (i / k));
  for (int q = lane; q < words; q += 64) {
    // sums of at most 16384 in 16-bit halves: bytes 0 and 2, bytes 1 and 3
    uint32_t all0 = 0, all1 = 0, pre0 = 0, pre1 = 0;
#pragma unroll 8
    for (int i = wave; i < chunks; i += 16) {
      const uint32_t v = reinterpret_cast<const uint32_t*>(few)[(size_t)i * words + q];
      const uint32_t a = v & 0x00FF00FFu, b = (v >> 8) & 0x00FF00FFu;
      all0 += a;
      all1 += b;
      pre0 += i < c ? a : 0u;
      pre1 += i < c ? b : 0u;
    }
    atomicAdd(&total[4 * q], (int)(all0 & 0xFFFFu));
    atomicAdd(&total[4 * q + 1], (int)(all1 & 0xFFFFu));
    atomicAdd(&total[4 * q + 2], (int)(all0 >> 16));
    atomicAdd(&total[4 * q + 3], (int)(all1 >> 16));
    atomicAdd(&first[4 * q], (int)(pre0 & 0xFFFFu));
    atomicAdd(&first[4 * q + 1], (int)(pre1 & 0xFFFFu));
    atomicAdd(&first[4 * q + 2], (int)(pre0 >> 16));
    atomicAdd(&first[4 * q + 3], (int)(pre1 >> 16));
  }
  __syncthreads();
  const int e = threadIdx.x;
  const int cnt = e < E ? total[e] : 0;
  const int at = block_prefix(cnt, wsum);
  if (e < E) {
    first[e] += at;
    if (blockIdx.x == 0) {
      counts[e] = cnt;
      if (counts_mirror) counts_mirror[e] = cnt;
      offsets[e] = at;
    }
  }
  if (blockIdx.x == 0 && e == 0) offsets[E] = T * k;
  __syncthreads();
  place(topk_idx, t0, n, k, first, masks, perm_src, perm_pos);
}

struct SelectWs {
  size_t hist, bits, bytes;
};
SelectWs select_ws(int T, int E) {
  // Counts and masks of 64-token chunks, as moe_route's scratch has them. The byte counts of up to kFewTokens lie over
  // both, four experts to a word: of n 64-token chunks' worth at most 4 n (E + 3) bytes (16-token chunks, n <= 64) or
  // 2 n (E + 3) (32-token ones), within the 12 n E + 256 for every E >= 1.
  const size_t n = (size_t)((T + 63) / 64) * E;
  SelectWs w{};
  w.hist = 0;
  w.bits = align_up(n * 4, 256);
  w.bytes = align_up(w.bits + n * 8, 256) + 256;
  return w;
}

struct SelectCall {
  LogitSource src;
  GateArgs g;
  int T, E, k, lanes, row_lanes;
  int32_t* topk_idx;
  float* topk_w;
  int32_t *counts, *offsets, *perm_src, *perm_pos, *counts_mirror;
  char* ws;
  hipStream_t s;
};

template <int VE, int RVE>
hipError_t select_kernels(const SelectCall& a) {
  const size_t lds = select_lds(a.E);
  if (a.T <= kOneBlock) {
    hipLaunchKernelGGL((select_one_block<VE, RVE>), dim3(1), dim3(1024), lds, a.s, a.src, a.g, a.lanes, a.row_lanes,
                       a.T, a.E, a.k, a.topk_idx, a.topk_w, a.counts, a.offsets, a.perm_src, a.perm_pos,
                       a.counts_mirror);
    return hipGetLastError();
  }
  const SelectWs w = select_ws(a.T, a.E);
  const bool few = a.T <= kFewTokens;
  // 16 tokens a block while that leaves at most a block for each CU; the masks hold 64 (512 tokens of 256 experts with
  // 16 / 64 a block 15.2 / 18.5 us, 8192 with 32 / 16 23.6 / 24.1)
  const int chunk = a.T <= 4096 ? 16 : RVE > 0 || !few ? kMaxTokensPerBlock : 32;
  const int chunks = (a.T + chunk - 1) / chunk, threads = RVE > 0 ? chunk * 16 : 1024;
  int32_t* hist = reinterpret_cast<int32_t*>(a.ws + w.hist);
  uint64_t* bits = reinterpret_cast<uint64_t*>(a.ws + w.bits);
  uint8_t* bytes = few ? reinterpret_cast<uint8_t*>(a.ws) : nullptr;
  hipLaunchKernelGGL((select_chunk<VE, RVE>), dim3(chunks), dim3(threads), lds, a.s, a.src, a.g, a.lanes, a.row_lanes,
                     a.T, a.E, a.k, chunk, a.topk_idx, a.topk_w, bytes, bits, hist);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (!few)
    return launch_group_rows(a.topk_idx, a.T, a.E, a.k, bits, hist, a.counts, a.offsets, a.perm_src, a.perm_pos,
                             a.counts_mirror, a.s);
  hipLaunchKernelGGL(place_chunk, dim3((a.T + kMaxTokensPerBlock - 1) / kMaxTokensPerBlock), dim3(1024),
                     (size_t)a.E * 8 + (size_t)(a.E + 3) / 4 * 32, a.s, a.topk_idx, a.T, a.E, a.k, chunk, chunks, bytes,
                     a.counts, a.offsets, a.perm_src, a.perm_pos, a.counts_mirror);
  return hipGetLastError();
}

// A row a token (RVE experts a lane) or a wave a token. Up to 16 tokens each wave of the block has one anyway. In a
// block of its own a wave with 16 tokens' work to share takes four turns of a row's; from two launches on, a wave a token
// has the shorter chain, and a row the fewer instructions once the chip is full, which is later the more experts a
// lane of the row holds. Captured calls in us, row / wave: 64 tokens x 256 experts of 8 groups 13.7 / 26.9, 512 15.2 /
// 13.8, 2048 20.7 / 14.0, 8192 27.0 / 23.6, 16384 30.3 / 39.8; 128 experts of 4 groups, 512 14.2 / 13.1, 2048 14.4 /
// 13.4, 4096 15.1 / 17.5; 64 experts, 512 10.6 / 11.0. Without a balance most experts need no score: 256 experts by
// softmax, 4096 tokens 14.6 / 13.7, 8192 16.9 / 19.6.
template <int VE>
hipError_t select_shapes(const SelectCall& a) {
  const SelectShape row = select_shape(a.E, a.g.n_group, 16);
  const bool given = a.src.nsplit == 1 && a.src.bias == nullptr && a.src.keep == nullptr;
  const bool wave = a.T <= 16 || (a.T > kOneBlock && a.T <= (row.ve > 8 ? (a.g.balance != nullptr ? 8192 : 4096) : row.ve > 4 ? 2048 : 0));
  if (given && !wave && row.lanes > 0) {
    SelectCall b = a;
    b.row_lanes = row.lanes;
    if (row.ve <= 4) return select_kernels<VE, 4>(b);
    if (row.ve <= 8) return select_kernels<VE, 8>(b);
    if (row.ve <= kRowMaxVe) return select_kernels<VE, kRowMaxVe>(b);
  }
  return select_kernels<VE, 0>(a);
}

}  // namespace

size_t select_workspace_bytes(int T, int E) { return select_ws(T, E).bytes; }

hipError_t launch_select(const float* logits, int nsplit, const float* bias, float* keep, const GateArgs& g, int T,
                         int E, int k, int32_t* topk_idx, float* topk_w, int32_t* counts, int32_t* offsets,
                         int32_t* perm_src, int32_t* perm_pos, void* ws, hipStream_t s, int32_t* counts_mirror) {
  const SelectShape sh = select_shape(E, g.n_group);
  const SelectCall a{LogitSource{logits, nsplit, (size_t)T * E, bias, keep}, g, T, E, k, sh.lanes, 0, topk_idx, topk_w,
                     counts, offsets, perm_src, perm_pos, counts_mirror, static_cast<char*>(ws), s};
  switch (sh.ve) {
    case 1: return select_shapes<1>(a);
    case 2: return select_shapes<2>(a);
    case 4: return select_shapes<4>(a);
    case 8: return select_shapes<8>(a);
    case 16: return select_shapes<16>(a);
    default: return select_shapes<32>(a);
  }
}

}  // namespace moe
