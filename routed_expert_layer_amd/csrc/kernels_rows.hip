// Tokens sorted by expert and back: the grouping of given choices, the copies
// of the token rows, the weighted sum of a token's rows and its gradient.
//
//   order of the rows: (expert, token, j);  pos[t, j] = rank, -1 if dropped
//   dispatch:  rows[pos[t, j]] = x[t]
//   collect:   out[t] = sum_j w[t, j] rows[pos[t, j]]          (j ascending, fp32)
//   backward:  drows[pos[t, j]] = w[t, j] dout[t],  dw[t, j] = <dout[t], rows[pos[t, j]]>
//
// All of them move bytes: a row is read once, in 16-byte loads, and written
// once; the sums stay in registers. Bytes bound them: 4096 tokens to 6 experts'
// rows of 4096 bf16 values 38 us (235 MB at 6.2 TB/s, mostly writes), their
// sums back 48 (4.9 TB/s), the gradient of 16384 tokens' sums of 6 rows 322 us
// (1.75 GB at 5.4 TB/s; a copy reaches 4.9); a pass over few rows is its launch.
#include <algorithm>
#include <type_traits>

#include "dev_common.hpp"
#include "moe_kernels.hpp"
#include "row_vec.hpp"

namespace moe {
namespace {

// ---------------------------------------------------------------------------
// Grouping.
// ---------------------------------------------------------------------------
constexpr int kGroupThreads = 1024;
constexpr int kGroupWaves = kGroupThreads / 64;
constexpr int kGroupBlocks = 64;     // most blocks of the two-launch form
constexpr int kGroupExperts = 1024;
// Forms: one block that counts what it places; several blocks that each count all the entries; or a launch that counts
// (group_count) and one that places. A block places 1024 entries a round, or 4096 where rounds are long anyway. Counting
// everything in each block saves a launch and costs a load and an LDS atomic for 1024 entries: 24576 entries of 256 experts
// 8.2 us, 11.8 with two launches, 32768 9.3 and 10.7, 40000 10.5 and 11.3, 65536 14.2 and 11.2. 6 entries take 3.0 us,
// latency of loads and of ten steps through LDS.
enum { kGroupOne, kGroupAll, kGroupTwo };
constexpr int kGroupOneMost = kGroupThreads;   // entries up to which each form is taken
constexpr int kGroupAllMost = 32768;
constexpr int group_round(int sub) { return kGroupThreads * sub; }

// Exclusive prefix sum of v over the block's threads (1024) and its total.
__device__ __forceinline__ int block_prefix(int v, int* sums, int& total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int s = v;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(s, d, 64);
    if (lane >= d) s += o;
  }
  if (lane == 63) sums[wave] = s;
  __syncthreads();
  int before = 0, all = 0;
  for (int w = 0; w < kGroupWaves; ++w) {
    before += w < wave ? sums[w] : 0;
    all += sums[w];
  }
  __syncthreads();
  total = all;
  return before + s - v;
}

// Choices per expert of each block's segment of the entries, hist[block][E].
__global__ __launch_bounds__(kGroupThreads) void group_count(const int32_t* __restrict__ idx, int n, int seg, int E,
                                                             int32_t* __restrict__ hist) {
  __shared__ int h[kGroupExperts];
  for (int e = threadIdx.x; e < E; e += kGroupThreads) h[e] = 0;
  __syncthreads();
  const int first = (int)min((int64_t)n, (int64_t)blockIdx.x * seg), end = (int)min((int64_t)n, (int64_t)first + seg);
#pragma unroll 4
  for (int i = first + (int)threadIdx.x; i < end; i += kGroupThreads) {
    const int e = idx[i];
    if ((unsigned)e < (unsigned)E) atomicAdd(&h[e], 1);  // integers: the order does not matter
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += kGroupThreads) hist[(size_t)blockIdx.x * E + e] = h[e];
}

// Places of a segment's entries. The rank of an entry among its expert's is
// the number in earlier segments and rounds (base), earlier waves and chunks of
// the round (cnt) and lower lanes of its chunk of 64: the lanes with the same
// expert are found by one ballot per bit of the expert's number. SUB chunks a
// wave per round.
template <int FORM, int SUB>
__global__ __launch_bounds__(kGroupThreads) void group_place(const int32_t* __restrict__ idx, int n, int seg, int k,
                                                             int E, int bits, const int32_t* __restrict__ hist,
                                                             int32_t* __restrict__ counts,
                                                             int32_t* __restrict__ offsets,
                                                             int32_t* __restrict__ perm_src,
                                                             int32_t* __restrict__ perm_pos) {
  __shared__ int cnt[kGroupWaves][kGroupExperts];
  __shared__ int sums[kGroupWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const uint64_t below = (1ull << lane) - 1ull;
  const int first = FORM == kGroupOne ? 0 : (int)min((int64_t)n, (int64_t)blockIdx.x * seg);
  const int end = FORM == kGroupOne ? n : (int)min((int64_t)n, (int64_t)first + seg);
  int base = 0;  // thread e: the place of the next entry of expert e
  auto publish = [&](int count) {
    int total;
    const int at = block_prefix(count, sums, total);
    if (blockIdx.x == 0) {
      if (tid < E) {
        counts[tid] = count;
        offsets[tid] = at;
      }
      if (tid == 0) offsets[E] = total;
    }
    return at;
  };
  if constexpr (FORM != kGroupOne) {
    int before = 0, all = 0;
    if constexpr (FORM == kGroupAll) {
      if (tid < E) cnt[0][tid] = cnt[1][tid] = 0;
      __syncthreads();
#pragma unroll 8
      for (int i = tid; i < n; i += kGroupThreads) {
        const int e = idx[i];
        if ((unsigned)e < (unsigned)E) atomicAdd(&cnt[i < first ? 0 : 1][e], 1);  // integers: the order does not matter
      }
      __syncthreads();
      if (tid < E) {
        before = cnt[0][tid];
        all = before + cnt[1][tid];
      }
    } else {
      if (tid < E)
#pragma unroll 8
        for (int b = 0; b < (int)gridDim.x; ++b) {
          const int c = hist[(size_t)b * E + tid];
          before += b < (int)blockIdx.x ? c : 0;
          all += c;
        }
    }
    base = publish(all) + before;  // its barriers stand before the next use of cnt too
  }
  for (int r = first; FORM == kGroupOne || r < end; r += group_round(SUB)) {
    const int here = min(group_round(SUB), end - r);
    const int waves = (here + 64 * SUB - 1) / (64 * SUB);
    for (int w = 0; w < waves; ++w)
      if (tid < E) cnt[w][tid] = 0;
    int e[SUB], rank[SUB];
#pragma unroll
    for (int c = 0; c < SUB; ++c) {
      const int i = (wave * SUB + c) * 64 + lane;
      const int v = i < here ? idx[r + i] : E;
      e[c] = (unsigned)v < (unsigned)E ? v : E;
    }
    __syncthreads();
    if (wave < waves)
#pragma unroll
      for (int c = 0; c < SUB; ++c) {
        uint64_t same = ~0ull;
        for (int b = 0; b < bits; ++b) {
          const bool on = (e[c] >> b) & 1;
          const uint64_t m = __ballot(on);
          same &= on ? m : ~m;
        }
        if (e[c] < E) {
          const int before = cnt[wave][e[c]];
          rank[c] = before + __popcll(same & below);
          if ((same & below) == 0) cnt[wave][e[c]] = before + __popcll(same);
        }
        __builtin_amdgcn_wave_barrier();  // the next chunk's reads follow this one's writes
      }
    __syncthreads();
    int run = base;
    if constexpr (FORM == kGroupOne) {
      int count = 0;
      if (tid < E)
        for (int w = 0; w < waves; ++w) count += cnt[w][tid];
      run = publish(count);
    }
    if (tid < E)
      for (int w = 0; w < waves; ++w) {
        const int c = cnt[w][tid];
        cnt[w][tid] = run;
        run += c;
      }
    base = run;
    __syncthreads();
#pragma unroll
    for (int c = 0; c < SUB; ++c) {
      const int i = (wave * SUB + c) * 64 + lane;
      if (i >= here) continue;
      const bool kept = e[c] < E;
      const int p = kept ? cnt[wave][e[c]] + rank[c] : -1;
      perm_pos[r + i] = p;
      if (kept) perm_src[p] = (int)((unsigned)(r + i) / (unsigned)k);
    }
    if constexpr (FORM == kGroupOne) break;
    __syncthreads();
  }
}

// Blocks and entries to a block of the two-launch form.
int group_blocks(int n) { return std::min(kGroupBlocks, (n + group_round(4) - 1) / group_round(4)); }

// ---------------------------------------------------------------------------
// Rows. A block takes 256 >> ls tokens, 1 << ls threads each; a thread takes
// kVecElems elements of its token's row.
// ---------------------------------------------------------------------------
struct RowShape {
  int T, k, H, rows, ls;
};

template <bool BF16, bool STREAM>
__global__ __launch_bounds__(256) void dispatch_kernel(const void* __restrict__ x, const int32_t* __restrict__ pos,
                                                       const RowShape s, void* __restrict__ out) {
  constexpr int N = kVecElems<BF16>;
  const int t = blockIdx.x * (256 >> s.ls) + ((int)threadIdx.x >> s.ls);
  const int c = (blockIdx.y * (1 << s.ls) + ((int)threadIdx.x & ((1 << s.ls) - 1))) * N;
  if (t >= s.T || c >= s.H) return;
  RowVec<BF16, N> v;
  v.load(x, (size_t)t * s.H + c, s.H - c);
  for (int j = 0; j < s.k; ++j) {
    const int p = pos[(size_t)t * s.k + j];
    if ((unsigned)p < (unsigned)s.rows) v.template store<STREAM>(out, (size_t)p * s.H + c, s.H - c);
  }
}

constexpr int kRowsAtOnce = 8;  // rows of a token whose loads are in flight together

template <bool BF16, bool OUT_BF16>
__global__ __launch_bounds__(256) void collect_kernel(const void* __restrict__ rows, const int32_t* __restrict__ pos,
                                                      const float* __restrict__ w, const RowShape s,
                                                      void* __restrict__ out) {
  constexpr int N = kVecElems<BF16>;
  const int t = blockIdx.x * (256 >> s.ls) + ((int)threadIdx.x >> s.ls);
  int c = (blockIdx.y * (1 << s.ls) + ((int)threadIdx.x & ((1 << s.ls) - 1))) * N;
  if (t >= s.T || c >= s.H) return;
  c = piece_start<N>(c, s.H);
  float acc[N] = {};
  for (int j0 = 0; j0 < s.k; j0 += kRowsAtOnce) {
    int p[kRowsAtOnce];
    float wj[kRowsAtOnce];
    RowVec<BF16, N> v[kRowsAtOnce];
#pragma unroll
    for (int j = 0; j < kRowsAtOnce; ++j) {
      p[j] = j0 + j < s.k ? pos[(size_t)t * s.k + j0 + j] : -1;
      wj[j] = w && j0 + j < s.k ? w[(size_t)t * s.k + j0 + j] : 1.f;
    }
#pragma unroll
    for (int j = 0; j < kRowsAtOnce; ++j)
      if ((unsigned)p[j] < (unsigned)s.rows) v[j].load(rows, (size_t)p[j] * s.H + c, s.H - c);
#pragma unroll
    for (int j = 0; j < kRowsAtOnce; ++j)
      if ((unsigned)p[j] < (unsigned)s.rows) {
#pragma unroll
        for (int i = 0; i < N; ++i) acc[i] = fmaf(wj[j], v[j].get(i), acc[i]);
      }
  }
  RowVec<OUT_BF16, N> o;
  o.set(acc);
  o.store(out, (size_t)t * s.H + c, s.H - c);
}

// dout's row is read once, each of the token's rows once. 1 << ls threads to a token, all 256 or a part of a wave.
template <bool BF16, bool OUT_BF16, bool DROWS, bool DW, bool STREAM>
__global__ __launch_bounds__(256) void collect_backward_kernel(const void* __restrict__ dout,
                                                               const void* __restrict__ rows,
                                                               const int32_t* __restrict__ pos,
                                                               const float* __restrict__ w, const RowShape s,
                                                               void* __restrict__ drows, float* __restrict__ dw) {
  constexpr int N = kVecElems<BF16>;
  __shared__ float part[4][kRowsAtOnce];
  const int t = blockIdx.x * (256 >> s.ls) + ((int)threadIdx.x >> s.ls);
  const int team = 1 << s.ls, rank = (int)threadIdx.x & (team - 1);
  const bool on = t < s.T;  // the others stay for the barriers
  for (int j0 = 0; j0 < s.k; j0 += kRowsAtOnce) {
    int p[kRowsAtOnce];
    float wj[kRowsAtOnce], dot[kRowsAtOnce] = {};
#pragma unroll
    for (int j = 0; j < kRowsAtOnce; ++j) {
      p[j] = on && j0 + j < s.k ? pos[(size_t)t * s.k + j0 + j] : -1;
      wj[j] = on && w && j0 + j < s.k ? w[(size_t)t * s.k + j0 + j] : 1.f;
    }
    for (int c0 = rank * N; on && c0 < s.H; c0 += team * N) {
      const int c = piece_start<N>(c0, s.H), before = c0 - c;  // elements of the piece before, not to be summed again
      RowVec<OUT_BF16, N> d;
      d.load(dout, (size_t)t * s.H + c, s.H - c);
      RowVec<BF16, N> v[kRowsAtOnce];
      if constexpr (DW) {
#pragma unroll
        for (int j = 0; j < kRowsAtOnce; ++j)
          if ((unsigned)p[j] < (unsigned)s.rows) v[j].template load<true>(rows, (size_t)p[j] * s.H + c, s.H - c);
      }
#pragma unroll
      for (int j = 0; j < kRowsAtOnce; ++j)
        if ((unsigned)p[j] < (unsigned)s.rows) {
          if constexpr (DW) {
            if (before == 0) {
#pragma unroll
              for (int i = 0; i < N; ++i) dot[j] = fmaf(d.get(i), v[j].get(i), dot[j]);
            } else {
#pragma unroll
              for (int i = 1; i < N; ++i) dot[j] = i >= before ? fmaf(d.get(i), v[j].get(i), dot[j]) : dot[j];
            }
          }
          if constexpr (DROWS) {
            float g[N];
#pragma unroll
            for (int i = 0; i < N; ++i) g[i] = wj[j] * d.get(i);
            RowVec<BF16, N> o;
            o.set(g);
            o.template store<STREAM>(drows, (size_t)p[j] * s.H + c, s.H - c);
          }
        }
    }
    if constexpr (DW) {
      for (int m = min(team, 64) / 2; m > 0; m >>= 1)
#pragma unroll
        for (int j = 0; j < kRowsAtOnce; ++j) dot[j] += __shfl_xor(dot[j], m, 64);
      if (team > 64) {
        if ((threadIdx.x & 63) == 0)
#pragma unroll
          for (int j = 0; j < kRowsAtOnce; ++j) part[threadIdx.x >> 6][j] = dot[j];
        __syncthreads();
        const int j = threadIdx.x;
        if (j < kRowsAtOnce && j0 + j < s.k)
          dw[(size_t)t * s.k + j0 + j] = (part[0][j] + part[1][j]) + (part[2][j] + part[3][j]);
        __syncthreads();
      } else if (on && rank == 0) {
#pragma unroll
        for (int j = 0; j < kRowsAtOnce; ++j)
          if (j0 + j < s.k) dw[(size_t)t * s.k + j0 + j] = dot[j];
      }
    }
  }
}

// Threads a token's row of n vectors gets, as a power of two of at most 256.
int lane_bits(int n) {
  int ls = 0;
  while (ls < 8 && (1 << ls) < n) ++ls;
  return ls;
}

// Whether rows that other kernels read next are stored past the caches. Rows whose pieces lie across cache lines, two of
// which then make a line together, are not where the memory-side cache holds them all. Past the caches and through them, us
// (buffers in turn): 30000 x 6 rows of 219 bf16 values out 22.9 and 18.5, their gradient 52.9 and 44.2; 4096 x 6 of 4095
// 55.2 and 52.5, 93 and 95; more than it holds: 16384 x 6 of 4095 207 and 244, 359 and 387; 16384 x 6 of 1001 fp32 values
// 100 and 104, 168 and 184; 8192 x 2 of 4097 68 and 93, 137 and 155. Near its size it goes either way: 4096 x 6 of 2047
// fp32 values (201 MB) out 57 and 51, 30000 x 6 of 219 (158 MB) 40 and 51.
constexpr int64_t kCacheBytes = 1 << 28;
bool past_caches(bool bf16, int H, int64_t rows) {
  return H % (bf16 ? kVecElems<true> : kVecElems<false>) == 0 || rows * H * (bf16 ? 2 : 4) > kCacheBytes;
}

template <typename F>
void with_flag(bool b, const F& f) {
  if (b) f(std::true_type{});
  else f(std::false_type{});
}

}  // namespace

size_t group_workspace_bytes(int T, int k, int E) {
  const int n = T * k;
  return n <= kGroupAllMost ? 0 : (size_t)group_blocks(n) * E * sizeof(int32_t);
}

hipError_t launch_group(const int32_t* idx, int T, int k, int E, int32_t* counts, int32_t* offsets, int32_t* perm_src,
                        int32_t* perm_pos, void* ws, hipStream_t s) {
  const int n = T * k;
  int bits = 0;
  while ((1 << bits) < E + 1) ++bits;
  const dim3 threads(kGroupThreads);
  if (n <= kGroupOneMost) {
    hipLaunchKernelGGL((group_place<kGroupOne, 1>), dim3(1), threads, 0, s, idx, n, 0, k, E, bits, nullptr, counts,
                       offsets, perm_src, perm_pos);
  } else if (n <= kGroupAllMost) {
    const int seg = group_round(1);
    hipLaunchKernelGGL((group_place<kGroupAll, 1>), dim3((n + seg - 1) / seg), threads, 0, s, idx, n, seg, k, E, bits,
                       nullptr, counts, offsets, perm_src, perm_pos);
  } else {
    const int blocks = group_blocks(n), round = group_round(4);
    const int seg = ((n + blocks - 1) / blocks + round - 1) / round * round;
    int32_t* hist = static_cast<int32_t*>(ws);
    hipLaunchKernelGGL(group_count, dim3(blocks), threads, 0, s, idx, n, seg, E, hist);
    hipLaunchKernelGGL((group_place<kGroupTwo, 4>), dim3(blocks), threads, 0, s, idx, n, seg, k, E, bits, hist, counts,
                       offsets, perm_src, perm_pos);
  }
  return hipGetLastError();
}

hipError_t launch_dispatch(const void* x, bool bf16, const int32_t* pos, int T, int k, int H, int rows, void* out,
                           hipStream_t s) {
  const int n = bf16 ? 8 : 4, nv = (H + n - 1) / n, ls = lane_bits(nv);
  const RowShape sh{T, k, H, rows, ls};
  const dim3 grid((T + (256 >> ls) - 1) / (256 >> ls), (nv + (1 << ls) - 1) >> ls);
  with_flag(bf16, [&](auto b) {
    with_flag(past_caches(bf16, H, std::min((int64_t)T * k, (int64_t)rows)), [&](auto p) {
      hipLaunchKernelGGL((dispatch_kernel<decltype(b)::value, decltype(p)::value>), grid, dim3(256), 0, s, x, pos, sh, out);
    });
  });
  return hipGetLastError();
}

hipError_t launch_collect(const void* rows, bool bf16, const int32_t* pos, const float* w, int T, int k, int H,
                          int n_rows, void* out, bool out_bf16, hipStream_t s) {
  const int n = bf16 ? 8 : 4, nv = (H + n - 1) / n, ls = lane_bits(nv);
  const RowShape sh{T, k, H, n_rows, ls};
  const dim3 grid((T + (256 >> ls) - 1) / (256 >> ls), (nv + (1 << ls) - 1) >> ls);
  with_flag(bf16, [&](auto b) {
    with_flag(out_bf16, [&](auto ob) {
      hipLaunchKernelGGL((collect_kernel<decltype(b)::value, decltype(ob)::value>), grid, dim3(256), 0, s, rows, pos, w,
                         sh, out);
    });
  });
  return hipGetLastError();
}

hipError_t launch_collect_backward(const void* dout, bool out_bf16, const void* rows, bool bf16, const int32_t* pos,
                                   const float* w, int T, int k, int H, int n_rows, void* drows, float* dw,
                                   hipStream_t s) {
  const int n = bf16 ? 8 : 4, nv = (H + n - 1) / n;
  // 256 threads to a token, so that few tokens fill the chip too; a wave or less where there are tokens enough and one or
  // two rows of each, whose sums would take as long as the rows (5000 tokens x 1 row of 720 values 18.5 us, 11.6 so; 4096 x
  // 6 of 4096 83 and 93), or where the row is short.
  const int most = T >= 2048 && k <= 2 ? 6 : 8;
  const int ls = lane_bits(nv) <= 6 ? lane_bits(nv) : most;
  const RowShape sh{T, k, H, n_rows, ls};
  const dim3 grid((T + (256 >> ls) - 1) / (256 >> ls));
  with_flag(bf16, [&](auto b) {
    with_flag(out_bf16, [&](auto ob) {
      with_flag(drows != nullptr, [&](auto dr) {
        with_flag(dw != nullptr, [&](auto dd) {
          with_flag(drows && past_caches(bf16, H, std::min((int64_t)T * k, (int64_t)n_rows)), [&](auto pc) {
            constexpr bool DR = decltype(dr)::value, DD = decltype(dd)::value, P = decltype(pc)::value;
            if constexpr (DR || (DD && !P))
              hipLaunchKernelGGL((collect_backward_kernel<decltype(b)::value, decltype(ob)::value, DR, DD, P>), grid,
                                 dim3(256), 0, s, dout, rows, pos, w, sh, drows, dw);
          });
        });
      });
    });
  });
  return hipGetLastError();
}

}  // namespace moe
