// Choice of a token's experts from scores of its logits, by one wave.
#pragma once
#include "dev_common.hpp"
#include "moe_kernels.hpp"

namespace moe {
namespace {

// Order-preserving map of a double (not a NaN) to a nonzero 64-bit key (-0 folded into +0).
__device__ __forceinline__ uint64_t double_key(double d) {
  const uint64_t u = (uint64_t)__double_as_longlong(d + 0.0);
  return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}

__device__ __forceinline__ uint64_t shfl_max_u64(uint64_t v) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) {
    const uint64_t o = (uint64_t)__shfl_xor((unsigned long long)v, d, 64);
    v = o > v ? o : v;
  }
  return v;
}

// One token's k experts (largest first) and their weights, lane j holding the
// j-th. Lane l holds the logits of experts VE l .. VE l + VE - 1 (E <= 64 VE).
//   s = softmax or sigmoid of the logits, c = s + balance
//   a group's rank: the sum of its group_top largest c; the topk_group best groups stay (ties to the lower group)
//   the k largest c in them (ties to the lower expert), w = s [/ their sum] * scale
// Scores are formed in 64 bits: the choice is whole numbers, and two biased
// scores are often closer than 32 bits tell apart over a long batch.
template <int VE>
__device__ __forceinline__ void select_token(const float (&l)[VE], int E, int k, const GateArgs& g, int lane,
                                             int& my_e, float& my_w) {
  double s[VE], c[VE];
  const int e0 = lane * VE;
  if (g.score == 0) {
    float m = -INFINITY;
#pragma unroll
    for (int v = 0; v < VE; ++v)
      if (e0 + v < E) m = fmaxf(m, l[v]);  // a NaN is never the larger
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor(m, d, 64));
    double z = 0.0;
#pragma unroll
    for (int v = 0; v < VE; ++v) {
      const float x = isnan(l[v]) ? -INFINITY : l[v];
      s[v] = e0 + v < E ? (x == m ? 1.0 : exp((double)x - (double)m)) : 0.0;
      z += s[v];
    }
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) z += __shfl_xor(z, d, 64);
#pragma unroll
    for (int v = 0; v < VE; ++v) s[v] /= z;
  } else {
#pragma unroll
    for (int v = 0; v < VE; ++v) s[v] = isnan(l[v]) ? 0.0 : 1.0 / (1.0 + exp(-(double)l[v]));
  }
#pragma unroll
  for (int v = 0; v < VE; ++v) {
    c[v] = s[v];
    if (g.balance != nullptr && e0 + v < E) c[v] += (double)g.balance[e0 + v];
    if (isnan(c[v])) c[v] = -INFINITY;
  }
  uint64_t key[VE];
#pragma unroll
  for (int v = 0; v < VE; ++v) key[v] = e0 + v < E ? double_key(c[v]) : 0ull;
  if (g.n_group > 1) {
    const int per = E / g.n_group;
    double rank = -INFINITY;  // lane i: group i's
    for (int i = 0; i < g.n_group; ++i) {
      double a = -INFINITY, b = -INFINITY;  // the two largest
#pragma unroll
      for (int v = 0; v < VE; ++v)
        if (e0 + v >= i * per && e0 + v < (i + 1) * per) {
          if (c[v] > a) {
            b = a;
            a = c[v];
          } else if (c[v] > b) {
            b = c[v];
          }
        }
#pragma unroll
      for (int d = 32; d > 0; d >>= 1) {
        const double oa = __shfl_xor(a, d, 64), ob = __shfl_xor(b, d, 64);
        b = fmax(fmin(a, oa), fmax(b, ob));
        a = fmax(a, oa);
      }
      if (lane == i) rank = (g.group_top == 2 && per > 1) ? a + b : a;
    }
    if (isnan(rank)) rank = -INFINITY;  // of an infinite balance of either sign
    uint64_t gk = lane < g.n_group ? double_key(rank) : 0ull, kept = 0;
    for (int i = 0; i < g.topk_group; ++i) {
      const uint64_t best = shfl_max_u64(gk);
      const int win = __ffsll((unsigned long long)__ballot(gk == best)) - 1;
      kept |= 1ull << win;
      if (lane == win) gk = 0;
    }
#pragma unroll
    for (int v = 0; v < VE; ++v)
      if (e0 + v < E && !(kept >> ((e0 + v) / per) & 1)) key[v] = 0;
  }
  double my_s = 0.0, sum = 0.0;
  my_e = 0;
  for (int j = 0; j < k; ++j) {
    uint64_t local = 0;
    int at = 0;
    double sv = 0.0;
#pragma unroll
    for (int v = 0; v < VE; ++v)
      if (key[v] > local) {
        local = key[v];
        at = v;
        sv = s[v];
      }
    const uint64_t best = shfl_max_u64(local);
    const int win = __ffsll((unsigned long long)__ballot(local == best)) - 1;
    const int e = __shfl(e0 + at, win, 64);
    const double ws = __shfl(sv, win, 64);
    if (lane == win) {
#pragma unroll
      for (int v = 0; v < VE; ++v)
        if (v == at) key[v] = 0;
    }
    sum += ws;
    if (lane == j) {
      my_e = e;
      my_s = ws;
    }
  }
  if (g.renorm) my_s = sum > 0.0 ? my_s / sum : 0.0;
  my_w = (float)(my_s * (double)g.scale);
}

}  // namespace
}  // namespace moe
