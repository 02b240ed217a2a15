// Selection of experts from given logits (or from the router products'
// partial sums) under a gate, and the grouping of the rows by expert.
#include "dev_common.hpp"
#include "dev_select.hpp"
#include "moe_kernels.hpp"

namespace moe {
namespace {

// Where a token's logits come from: nsplit slabs of partial sums, `slab`
// floats apart, added in order, plus a bias; nsplit 1 and no bias for logits
// as given. The sums go to `keep` when it is set.
struct LogitSource {
  const float* p;
  int nsplit;
  size_t slab;
  const float* bias;
  float* keep;
  template <int VE>
  __device__ __forceinline__ void load(int t, int E, int lane, float (&l)[VE]) const {
#pragma unroll
    for (int v = 0; v < VE; ++v) {
      const int e = lane * VE + v;
      l[v] = -INFINITY;
      if (e < E) {
        const size_t at = (size_t)t * E + e;
        float x = p[at];
        for (int z = 1; z < nsplit; ++z) x += p[(size_t)z * slab + at];
        if (bias) x += bias[e];
        if (keep) keep[at] = x;
        l[v] = x;
      }
    }
  }
};

// A block takes 64 tokens, a wave one token at a time: their choice, and the
// block's masks (which of its tokens chose an expert) and counts for the
// grouping kernels.
template <int VE>
__global__ __launch_bounds__(1024) void select_chunk(const LogitSource src, const GateArgs g, int T, int E, int k,
                                                     int nchunks, int32_t* __restrict__ topk_idx,
                                                     float* __restrict__ topk_w, uint64_t* __restrict__ bits,
                                                     int32_t* __restrict__ hist) {
  __shared__ unsigned long long bm[64 * VE];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  for (int e = threadIdx.x; e < E; e += 1024) bm[e] = 0ull;
  __syncthreads();
  for (int i = wave; i < 64; i += 16) {
    const int t = blockIdx.x * 64 + i;
    if (t >= T) break;
    float l[VE];
    src.load(t, E, lane, l);
    int e;
    float w;
    select_token(l, E, k, g, lane, e, w);
    if (lane < k) {
      topk_idx[(size_t)t * k + lane] = e;
      topk_w[(size_t)t * k + lane] = w;
      atomicOr(&bm[e], 1ull << i);
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += 1024) {
    const uint64_t b = bm[e];
    bits[(size_t)blockIdx.x * E + e] = b;
    hist[(size_t)e * nchunks + blockIdx.x] = __popcll(b);
  }
}

template <int VE>
hipError_t launch_chunks(const LogitSource& src, const GateArgs& g, int T, int E, int k, int32_t* topk_idx,
                         float* topk_w, uint64_t* bits, int32_t* hist, hipStream_t s) {
  const int nchunks = (T + 63) / 64;
  hipLaunchKernelGGL(select_chunk<VE>, dim3(nchunks), dim3(1024), 0, s, src, g, T, E, k, nchunks, topk_idx, topk_w,
                     bits, hist);
  return hipGetLastError();
}

struct SelectWs {
  size_t hist, bits, bytes;
};
SelectWs select_ws(int T, int E) {
  const size_t n = (size_t)((T + 63) / 64) * E;
  SelectWs w{};
  w.hist = 0;
  w.bits = align_up(n * 4, 256);
  w.bytes = align_up(w.bits + n * 8, 256) + 256;
  return w;
}

}  // namespace

size_t select_workspace_bytes(int T, int E) { return select_ws(T, E).bytes; }

hipError_t launch_select(const float* logits, int nsplit, const float* bias, float* keep, const GateArgs& g, int T,
                         int E, int k, int32_t* topk_idx, float* topk_w, int32_t* counts, int32_t* offsets,
                         int32_t* perm_src, int32_t* perm_pos, void* ws, hipStream_t s, int32_t* counts_mirror) {
  const SelectWs w = select_ws(T, E);
  int32_t* hist = reinterpret_cast<int32_t*>(static_cast<char*>(ws) + w.hist);
  uint64_t* bits = reinterpret_cast<uint64_t*>(static_cast<char*>(ws) + w.bits);
  const LogitSource src{logits, nsplit, (size_t)T * E, bias, keep};
  hipError_t e = hipSuccess;
  if (T > 0) {
    if (E <= 64) e = launch_chunks<1>(src, g, T, E, k, topk_idx, topk_w, bits, hist, s);
    else if (E <= 128) e = launch_chunks<2>(src, g, T, E, k, topk_idx, topk_w, bits, hist, s);
    else if (E <= 256) e = launch_chunks<4>(src, g, T, E, k, topk_idx, topk_w, bits, hist, s);
    else if (E <= 512) e = launch_chunks<8>(src, g, T, E, k, topk_idx, topk_w, bits, hist, s);
    else e = launch_chunks<16>(src, g, T, E, k, topk_idx, topk_w, bits, hist, s);
  }
  if (e != hipSuccess) return e;
  return launch_group_rows(topk_idx, T, E, k, bits, hist, counts, offsets, perm_src, perm_pos, counts_mirror, s);
}

}  // namespace moe
