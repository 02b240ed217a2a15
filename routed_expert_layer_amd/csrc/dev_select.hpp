// Choice of a token's experts from scores of its logits, by one wave.
//
//   s = softmax or sigmoid of the logits, c = s + balance
//   a group's rank: its largest c, or the sum of its two largest; the
//   topk_group best groups stay (ties to the lower group)
//   the k largest c in them (ties to the lower expert)
//   w = s [/ their sum] * scale
//
// The choice is whole numbers and is that of 64-bit scores. Two biased scores
// of a long batch are now and then closer than 32 bits tell apart, but seldom:
// so the wave looks for a threshold that k experts' 32-bit scores reach (or
// their logits, which are in the same order, where there is no balance), forms
// the 64-bit scores of those alone, one a lane, orders them, and keeps the
// choice if all are above the threshold by more than the 32-bit scores' error.
// Otherwise it chooses again from 64-bit scores of every expert (one token in
// 1600 of 256 experts with a balance, in 3600 with groups too, of which the row
// form below hands on one in 1400; none of 82000 without a balance).
// Long batches are instructions and the latency of their steps, not bytes
// (16384 tokens of 256 experts in 8 groups: 25 us, 0.7 TB/s of logits, 61% of
// the VALU's issue slots at four waves a SIMD; a first kernel that formed 64-bit
// scores of every expert took 86 us a call): more than half of a token's
// instructions do not depend on how many experts a lane holds, so a token has
// a row of 16 lanes there (select_row), four tokens to a wave. In
// short ones latency counts and a token has a wave (select_token; 6.8 us in the
// kernel for one token of 256).
#pragma once
#include "dev_common.hpp"
#include "moe_kernels.hpp"

namespace moe {
namespace {

// How the E experts lie on a wave, or on a row of 16 lanes: each group has
// `lanes` lanes (a power of two), lane i of a group VE consecutive experts of
// it. lanes 0: more groups than lanes.
struct SelectShape {
  int lanes, ve;
};
inline SelectShape select_shape(int E, int n_group, int width = 64) {
  SelectShape s{width, 1};
  while (s.lanes * n_group > width) s.lanes /= 2;
  while (s.lanes > 0 && s.ve * s.lanes * n_group < E) s.ve *= 2;
  return s;
}
constexpr int kRowMaxVe = 16;  // experts a lane of a row

// Order-preserving map of a float / double (not a NaN) to a nonzero key (-0 folded into +0).
__device__ __forceinline__ uint32_t order_key(float f) {
  const uint32_t u = __float_as_uint(f + 0.0f);
  return (u >> 31) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float order_value(uint32_t k) {
  return __uint_as_float((k >> 31) ? (k & 0x7FFFFFFFu) : ~k);
}
__device__ __forceinline__ uint64_t order_key(double d) {
  const uint64_t u = (uint64_t)__double_as_longlong(d + 0.0);
  return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}

template <int CTRL, int ROWS = 0xF>
__device__ __forceinline__ uint32_t dpp_u32(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, CTRL, ROWS, 0xF, false);
}
// Max over the wave, wave-uniform: within rows of 16 lanes by quad permutes and rotations, then down the rows
// (row_bcast:15 into rows 1 and 3, row_bcast:31 into rows 2 and 3), so that lane 63 has it.
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  v = max(v, dpp_u32<0xB1>(v));
  v = max(v, dpp_u32<0x4E>(v));
  v = max(v, dpp_u32<0x124>(v));
  v = max(v, dpp_u32<0x128>(v));
  v = max(v, dpp_u32<0x142, 0xA>(v));
  v = max(v, dpp_u32<0x143, 0xC>(v));
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}
__device__ __forceinline__ float wave_max(float f) { return order_value(wave_max(order_key(f))); }
__device__ __forceinline__ float wave_min(float f) { return order_value(~wave_max(~order_key(f))); }
__device__ __forceinline__ uint64_t wave_max(uint64_t v) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) {
    const uint64_t o = (uint64_t)__shfl_xor((unsigned long long)v, d, 64);
    v = o > v ? o : v;
  }
  return v;
}
template <typename F>
__device__ __forceinline__ F wave_sum(F v) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d, 64);
  return v;
}

__device__ __forceinline__ double sigmoid64(float l) { return 1.0 / (1.0 + exp(-(double)l)); }
// exp(l - m) for m the row's largest logit: 1 where they are equal (an infinite m among them)
__device__ __forceinline__ double share64(float l, float m) { return l == m ? 1.0 : exp((double)l - (double)m); }

// 32-bit scores s, within kErr. Sigmoid: e = exp(-l) is off by 6e-8 |l| (the rounded argument) and a step, which moves s
// by s (1 - s) of that, below 5e-8; the sum's and the reciprocal's roundings by 1.8e-7 s. Softmax: the argument
// x = m - l counts 1.2e-7 x and the roundings 2.4e-7, of s <= exp(-x): below 2.4e-7. Both are under half of kErr.
constexpr float kErr = 0x1p-21f;
__device__ __forceinline__ float score32(float l, float m, float iz, int score) {
  return score == 0 ? (l == m ? 1.f : __expf(l - m)) * iz : __builtin_amdgcn_rcpf(1.f + __expf(-l));
}
// Bounds between which another group's rank may come before one of `rank` or not. Logits 1e-6 apart have different
// 64-bit scores up to 20 (a sigmoid's distance from 1) and down to -600 (of the largest, for a softmax).
// By c, a rank r of one c or of two, a + b, of magnitudes up to M: each c is off by kErr / 2 and its rounding 2^-24 |c|,
// their sum by 2^-24 |r|, so r by kErr + 2^-22 M at most. Where M <= 1 + 2 |r| (else it cancels, and its token is undecided) that is below
// 1.5 kErr + 2^-21 |r|. Two ranks r, o then differ truly if |r - o| > 3 kErr + 2^-21 (|r| + |o|): d covers it for
// |o| <= 2 |r|, and a larger |o| is itself twice that far from r.
__device__ __forceinline__ void rank_bounds(float rank, bool by_c, int score, float m, float& above, float& below) {
  const float d = by_c ? 8.f * kErr + 0x1p-19f * fabsf(rank) : 1e-6f;
  above = by_c ? rank + d : fmaxf(rank + d, score == 0 ? m - 600.f : -600.f);
  below = rank - d;
}

// A first threshold: somewhat below the least of values whose largest is hi, so that it is none of them.
__device__ __forceinline__ float below_all(float least, float hi) {
  return least - (0.0625f * (hi - least) + 1e-6f * fabsf(least) + 1e-30f);
}

// The two largest of a set, merged with another lane's.
template <typename F>
struct Top2 {
  F a, b;
  __device__ __forceinline__ void put(F v) {
    if constexpr (sizeof(F) == 4) {
      b = __builtin_amdgcn_fmed3f(a, b, v);
      a = fmaxf(a, v);
    } else {
      b = v > a ? a : (v > b ? v : b);
      a = v > a ? v : a;
    }
  }
  __device__ __forceinline__ void merge(F oa, F ob) {
    const F lo = oa > a ? a : oa, hb = ob > b ? ob : b;
    a = oa > a ? oa : a;
    b = lo > hb ? lo : hb;
  }
};
// Lane i ^ D's value, for a value that already agrees over groups of D lanes (mirrors then do for exchanges).
template <int D, typename F>
__device__ __forceinline__ F across(F v) {
  static_assert(sizeof(F) == 4 || sizeof(F) == 8, "whole registers");
  if constexpr (D >= 16) {
    return __shfl_xor(v, D, 64);
  } else {
    constexpr int ctrl = D == 1 ? 0xB1 : D == 2 ? 0x4E : D == 4 ? 0x141 : 0x140;
    if constexpr (sizeof(F) == 4) {
      return __builtin_bit_cast(F, dpp_u32<ctrl>(__builtin_bit_cast(uint32_t, v)));
    } else {
      const uint64_t u = __builtin_bit_cast(uint64_t, v);
      const uint64_t lo = dpp_u32<ctrl>((uint32_t)u), hi = dpp_u32<ctrl>((uint32_t)(u >> 32));
      return __builtin_bit_cast(F, (hi << 32) | lo);
    }
  }
}
template <int D, typename F>
__device__ __forceinline__ void top2_step(Top2<F>& t, int lanes, bool two) {
  if (lanes > D) t.merge(across<D>(t.a), two ? across<D>(t.b) : t.b);
}
// A group's rank, on each of its lanes, from the lanes' values (`ok` of them first). cancels: its two c are of opposite
// signs (balances that pin one expert and mask another) and their sum says nothing of the error that it carries.
template <int WIDTH, int VE, typename F>
__device__ __forceinline__ F group_rank(const F (&c)[VE], int ok, int lanes, bool two, bool& cancels) {
  Top2<F> t{-INFINITY, -INFINITY};
#pragma unroll
  for (int v = 0; v < VE; ++v)
    if (v < ok) t.put(c[v]);
  top2_step<1>(t, lanes, two);
  top2_step<2>(t, lanes, two);
  top2_step<4>(t, lanes, two);
  top2_step<8>(t, lanes, two);
  if constexpr (WIDTH > 16) {
    top2_step<16>(t, lanes, two);
    top2_step<32>(t, lanes, two);
  }
  const F r = two ? t.a + t.b : t.a;
  cancels = two && fmax(fabs(t.a), fabs(t.b)) > 1 + 2 * fabs(r);
  return isnan(r) ? (F)-INFINITY : r;  // of infinite balances of either sign
}
// How many groups come before this lane's: larger ranks, and equal ones of lower groups.
__device__ __forceinline__ int groups_before(double rank, int group, int lanes, int n_group) {
  int n = 0;
  for (int i = 0; i < n_group; ++i) {
    const double o = __shfl(rank, i * lanes, 64);
    n += (o > rank || (o == rank && i < group)) ? 1 : 0;
  }
  return n;
}

// The choice from 64-bit scores of every expert.
template <int VE>
__device__ __forceinline__ void select_exact(const float (&l)[VE], int ok, int base, int group, int lanes, int per,
                                             int k, const GateArgs& g, const float* bal, int lane, float m, double z,
                                             int& my_e, double& my_s) {
  double c[VE];
  uint64_t key[VE];
#pragma unroll
  for (int v = 0; v < VE; ++v) {
    c[v] = -INFINITY;
    if (v < ok) {
      c[v] = g.score == 0 ? share64(l[v], m) / z : sigmoid64(l[v]);
      if (bal != nullptr) c[v] += (double)bal[base + v];
      if (isnan(c[v])) c[v] = -INFINITY;
    }
  }
  bool kept = true;
  if (g.topk_group < g.n_group) {
    bool cancels;  // not of interest in 64 bits
    const double rank = group_rank<64>(c, ok, lanes, g.group_top == 2 && per > 1, cancels);
    kept = groups_before(rank, group, lanes, g.n_group) < g.topk_group;
  }
#pragma unroll
  for (int v = 0; v < VE; ++v) key[v] = v < ok && kept ? order_key(c[v]) : 0ull;
  for (int j = 0; j < k; ++j) {
    uint64_t local = 0;
    int at = 0;
#pragma unroll
    for (int v = 0; v < VE; ++v)
      if (key[v] > local) {
        local = key[v];
        at = v;
      }
    const uint64_t best = wave_max(local);
    const int win = __ffsll((unsigned long long)__ballot(local == best)) - 1;
    float lv = 0.f;
#pragma unroll
    for (int v = 0; v < VE; ++v) {
      if (v == at) lv = l[v];
      if (v == at && lane == win) key[v] = 0;
    }
    const int e = __shfl(base + at, win, 64);
    const float lw = __shfl(lv, win, 64);
    if (lane == j) {
      my_e = e;
      my_s = g.score == 0 ? share64(lw, m) / z : sigmoid64(lw);
    }
  }
}

// One token's k experts and their weights: lane j < k holds one, my_at its
// place (0 the largest). logits: the token's E logits in LDS; bal: the
// balance, LDS or global; per = E / n_group.
template <int VE>
__device__ __forceinline__ void select_token(const float* logits, const float* bal, int per, int k, const GateArgs& g,
                                             int lanes, int lane, int& my_e, float& my_w, int& my_at) {
  const int group = lane / lanes, sub = lane & (lanes - 1);
  const int base = group * per + sub * VE;
  const int ok = group < g.n_group ? min(max(per - sub * VE, 0), VE) : 0;  // experts of this lane
  float l[VE];
#pragma unroll
  for (int v = 0; v < VE; ++v) {
    l[v] = -INFINITY;
    if (v < ok) l[v] = logits[base + v];
    if (isnan(l[v])) l[v] = -INFINITY;
  }
  const bool drops = g.topk_group < g.n_group, two = g.group_top == 2 && per > 1;
  float m = 0.f;
  double z = 1.0;  // the softmax's denominator, where more than its order and ratios are asked for
  if (g.score == 0) {
    m = l[0];
#pragma unroll
    for (int v = 1; v < VE; ++v) m = fmaxf(m, l[v]);
    m = wave_max(m);
    if (bal != nullptr || !g.renorm || (two && drops)) {
      z = 0.0;
#pragma unroll
      for (int v = 0; v < VE; ++v) z += v < ok ? share64(l[v], m) : 0.0;
      z = wave_sum(z);
    }
  }
  float c[VE];
  if (bal != nullptr || (two && drops)) {
    const float iz = (float)(1.0 / z);
#pragma unroll
    for (int v = 0; v < VE; ++v) {
      const float s = score32(l[v], m, iz, g.score);
      c[v] = bal != nullptr && v < ok ? s + bal[base + v] : s;
      if (isnan(c[v])) c[v] = -INFINITY;
    }
  }
  bool unsure = false, kept = true;
  if (drops) {
    const bool by_c = bal != nullptr || two;
    bool cancels;
    const float rank = by_c ? group_rank<64>(c, ok, lanes, two, cancels) : group_rank<64>(l, ok, lanes, false, cancels);
    float above, below;  // groups surely before this one, and groups that may be
    rank_bounds(rank, by_c, g.score, m, above, below);
    int sure = 0, may = -1;  // its own rank is one of the latter
    for (int i = 0; i < g.n_group; ++i) {
      const float o = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(rank), i * lanes));
      sure += o > above ? 1 : 0;
      may += o >= below ? 1 : 0;
    }
    kept = may < g.topk_group;
    unsure = cancels || (!kept && sure < g.topk_group);
    unsure = unsure || (kept && !(by_c || g.score == 0 ? rank < INFINITY : rank < 20.f));
    unsure = unsure && group < g.n_group;
  }
  // the values that decide, -inf where an expert cannot be chosen; a threshold T that k of them reach
  float x[VE];
  float top = -INFINITY;
#pragma unroll
  for (int v = 0; v < VE; ++v) {
    x[v] = v < ok && kept ? (bal != nullptr ? c[v] : l[v]) : -INFINITY;
    top = fmaxf(top, x[v]);
  }
  float hi = wave_max(top);
  float lo = below_all(wave_min(top > -INFINITY ? top : INFINITY), hi);  // each lane's largest above -inf reaches it
  const auto reach = [&](float T) {
    int n = 0;
#pragma unroll
    for (int v = 0; v < VE; ++v) n += __popcll(__ballot(x[v] >= T));
    return n;
  };
  bool found = __ballot(unsure) == 0 && hi < INFINITY;
  float T = lo;
  if (found) {
    int n = reach(T);
    if (n < k) {  // fewer lanes than choices: from the least value
      float least = INFINITY;
#pragma unroll
      for (int v = 0; v < VE; ++v)
        if (x[v] > -INFINITY) least = fminf(least, x[v]);
      T = lo = below_all(wave_min(least), hi);
      n = reach(T);
      found = n >= k;
    }
    // halving: four or five steps, since the values above lo are few; equal ones at the k-th never end it
    for (int i = 0; n != k && found; ++i) {
      T = 0.5f * (lo + hi);
      n = reach(T);
      if (n > k) lo = T; else hi = T;
      found = i < 24;
    }
  }
  // the chosen to lanes 0 .. k - 1 (the others to lane 63, which is not read)
  my_e = 0;
  if (found) {
    int before = 0;
#pragma unroll
    for (int v = 0; v < VE; ++v) {
      const bool take = x[v] >= T;
      const uint64_t mask = __ballot(take);
      const int at = before + (int)__builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32),
                                                             __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0));
      my_e |= __builtin_amdgcn_ds_permute((take ? at : 63) * 4, take ? base + v : 0);
      before += __popcll(mask);
    }
  }
  // their 64-bit scores, in order, if those are above all that the others can have (below T by the 32-bit scores)
  double s = 0.0, cs = 0.0;
  bool wrong = false;
  if (found && lane < k) {
    const float le = fmaxf(logits[my_e], -INFINITY);  // a NaN is -inf: with a balance it can be chosen
    s = g.score == 0 ? share64(le, m) / z : sigmoid64(le);
    cs = s;
    double most;
    if (bal != nullptr) {
      cs += (double)bal[my_e];
      most = (double)T + (double)(kErr + 0x1p-22f * fabsf(T));
    } else {
      most = g.score == 0 ? share64(T, m) / z : sigmoid64(T);
    }
    wrong = !(cs > most) && g.topk_group * per > k;
  }
  my_at = lane;
  if (__builtin_expect(!found || __ballot(wrong) != 0, 0)) {
    if (g.score == 0 && bal == nullptr) {
      // the scores' ratios and order need no denominator, but equal 64-bit scores have to be those of the quotients
      z = 0.0;
#pragma unroll
      for (int v = 0; v < VE; ++v) z += v < ok ? share64(l[v], m) : 0.0;
      z = wave_sum(z);
    }
    select_exact(l, ok, base, group, lanes, per, k, g, bal, lane, m, z, my_e, s);
  } else {
    const uint64_t bits = (uint64_t)__double_as_longlong(cs);
    int n = 0;
    for (int i = 0; i < k; ++i) {
      const uint64_t o = ((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(bits >> 32), i) << 32) |
                         (uint32_t)__builtin_amdgcn_readlane((int)bits, i);
      const double oc = __longlong_as_double((long long)o);
      const int oe = __builtin_amdgcn_readlane(my_e, i);
      n += (oc > cs || (oc == cs && oe < my_e)) ? 1 : 0;
    }
    my_at = n;
  }
  if (lane >= k) s = 0.0;
  if (g.renorm) {  // the first 16 lanes hold all of them
    double sum = s;
    sum += across<1>(sum);
    sum += across<2>(sum);
    sum += across<4>(sum);
    sum += across<8>(sum);
    s = sum > 0.0 ? s / sum : 0.0;
  }
  my_w = (float)(s * (double)g.scale);
}

// The logits of a row's lanes (-inf past the experts); vec: whole pieces of four, 16-byte aligned.
template <int VE>
__device__ __forceinline__ void load_row(const float* __restrict__ logits, bool vec, int per, int n_group, int lanes,
                                         int lane, float (&l)[VE]) {
  const int r = lane & 15, group = r / lanes, sub = r & (lanes - 1);
  const int base = group * per + sub * VE;
  const int ok = group < n_group ? min(max(per - sub * VE, 0), VE) : 0;
  if (VE % 4 == 0 && vec) {
#pragma unroll
    for (int v = 0; v < VE; v += 4) {
      f32x4_t q = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
      if (v < ok) q = *reinterpret_cast<const f32x4_t*>(logits + base + v);
#pragma unroll
      for (int u = 0; u < 4; ++u) l[v + u] = q[u];
    }
  } else {
#pragma unroll
    for (int v = 0; v < VE; ++v) {
      l[v] = -INFINITY;
      if (v < ok) l[v] = logits[base + v];
    }
  }
}

// A row of 16 lanes a token, four tokens to a wave. l: load_row's; logits: the lane's token's, in memory; pick, score: LDS of the wave
// (64 each); bal: the balance in LDS, without NaN. Lane r < k of a row holds one choice, my_at its place. False: the
// row's token is one that 32-bit scores do not decide (select_token then does).
template <int VE>
__device__ __forceinline__ bool select_row(float (&l)[VE], const float* __restrict__ logits, const float* bal, int per,
                                           int k, const GateArgs& g, int lanes, int lane, int* pick, double* score, int& my_e,
                                           float& my_w, int& my_at) {
  const int r = lane & 15, row = lane & 48;
  const int group = r / lanes, sub = r & (lanes - 1);
  const int base = group * per + sub * VE;
  const int ok = group < g.n_group ? min(max(per - sub * VE, 0), VE) : 0;
  float most = -INFINITY;
#pragma unroll
  for (int v = 0; v < VE; ++v) {
    l[v] = fmaxf(l[v], -INFINITY);  // a NaN is -inf
    most = fmaxf(most, l[v]);
  }
  const auto row_max = [](float f) {
    f = fmaxf(f, across<1>(f));
    f = fmaxf(f, across<2>(f));
    f = fmaxf(f, across<4>(f));
    return fmaxf(f, across<8>(f));
  };
  const auto row_sum = [](auto f) {
    f += across<1>(f);
    f += across<2>(f);
    f += across<4>(f);
    return f + across<8>(f);
  };
  const bool drops = g.topk_group < g.n_group, two = g.group_top == 2 && per > 1;
  float m = 0.f;
  double z = 1.0;
  if (g.score == 0) {
    m = row_max(most);
    if (bal != nullptr || !g.renorm || (two && drops)) {
      z = 0.0;
#pragma unroll
      for (int v = 0; v < VE; ++v) z += v < ok ? share64(l[v], m) : 0.0;
      z = row_sum(z);
    }
  }
  // x: the values that decide
  float x[VE];
  bool kept = true, unsure = false, cancels = false;
  if (bal != nullptr || (two && drops)) {
    const float iz = (float)(1.0 / z);
    float c[VE];
#pragma unroll
    for (int v = 0; v < VE; ++v) {
      const float s = score32(l[v], m, iz, g.score);
      c[v] = s;
      if (bal != nullptr) c[v] = v < ok ? s + bal[base + v] : -INFINITY;
    }
    float rank = 0.f;
    if (drops) rank = group_rank<16>(c, ok, lanes, two, cancels);
#pragma unroll
    for (int v = 0; v < VE; ++v) x[v] = bal != nullptr ? c[v] : l[v];
    most = rank;
  } else {
    if (drops) most = group_rank<16>(l, ok, lanes, false, cancels);
#pragma unroll
    for (int v = 0; v < VE; ++v) x[v] = l[v];
  }
  if (drops) {
    const float rank = most;
    const bool by_c = bal != nullptr || two;
    float above, below;
    rank_bounds(rank, by_c, g.score, m, above, below);
    int sure = 0, may = -1;
    // four at a time, so that their exchanges are in flight together
    for (int i = 0; i < g.n_group; i += 4) {
      float o[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) o[u] = __shfl(rank, row + min(i + u, g.n_group - 1) * lanes, 64);
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (i + u < g.n_group) {
          sure += o[u] > above ? 1 : 0;
          may += o[u] >= below ? 1 : 0;
        }
    }
    kept = may < g.topk_group;
    unsure = cancels || (!kept && sure < g.topk_group);
    unsure = unsure || (kept && !(by_c || g.score == 0 ? rank < INFINITY : rank < 20.f));
    unsure = unsure && group < g.n_group;
  }
  float top = x[0];
#pragma unroll
  for (int v = 1; v < VE; ++v) top = fmaxf(top, x[v]);
  top = kept && ok > 0 ? top : -INFINITY;
  const auto reach = [&](float T) {  // counts what is picked below, no more: a dropped group's logit may be infinite
    int n = 0;
#pragma unroll
    for (int v = 0; v < VE; ++v) n += x[v] >= T ? 1 : 0;
    return kept && ok > 0 ? n : 0;
  };
  float hi = row_max(top), lo = below_all(-row_max(top > -INFINITY ? -top : -INFINITY), hi);
  const int doubts = row_sum(unsure ? 1 : 0);
  bool open = hi < INFINITY && doubts == 0;  // still looking for the token's threshold
  float T = lo;
  int mine = reach(T), n = row_sum(mine);
  if (__ballot(open && n < k) != 0) {
    float least = INFINITY;
#pragma unroll
    for (int v = 0; v < VE; ++v)
      if (x[v] > -INFINITY && kept && ok > 0) least = fminf(least, x[v]);
    least = -row_max(-least);
    if (n < k) T = lo = below_all(least, hi);
    mine = reach(T);
    n = row_sum(mine);
    if (n < k) open = false;
  }
  bool found = open && n == k;
  open = open && n != k;
  for (int i = 0; i < 24 && __ballot(open) != 0; ++i) {
    const float mid = 0.5f * (lo + hi);
    const int c = reach(mid), all = row_sum(c);
    if (open) {
      T = mid;
      mine = c;
      if (all > k) lo = mid; else hi = mid;
      found = all == k;
      open = all != k;
    }
  }
  // the chosen to lanes 0 .. k - 1 of the row
  int at = mine;
  // prefix over the row, by shifts of 1, 2, 4 and 8 lanes, each taken by every lane before it is used by some (inside a
  // conditional expression the lanes that are read could be inactive)
  const auto shifted_add = [&](int o, int d) { at += r >= d ? o : 0; };
  const int o1 = (int)dpp_u32<0x111>((uint32_t)at);
  shifted_add(o1, 1);
  const int o2 = (int)dpp_u32<0x112>((uint32_t)at);
  shifted_add(o2, 2);
  const int o4 = (int)dpp_u32<0x114>((uint32_t)at);
  shifted_add(o4, 4);
  const int o8 = (int)dpp_u32<0x118>((uint32_t)at);
  shifted_add(o8, 8);
  at += row - mine;
  if (found) {
#pragma unroll
    for (int v = 0; v < VE; ++v)
      if (x[v] >= T && kept && ok > 0) pick[at++] = base + v;
  }
  __builtin_amdgcn_wave_barrier();
  double s = 0.0, cs = 0.0;
  bool wrong = !found;
  my_e = 0;
  if (found && r < k) {
    my_e = pick[lane];
    const float le = fmaxf(logits[my_e], -INFINITY);  // a NaN is -inf
    s = g.score == 0 ? share64(le, m) / z : sigmoid64(le);
    cs = s;
    double bound;
    if (bal != nullptr) {
      cs += (double)bal[my_e];
      bound = (double)T + (double)(kErr + 0x1p-22f * fabsf(T));
    } else {
      bound = g.score == 0 ? share64(T, m) / z : sigmoid64(T);
    }
    wrong = !(cs > bound) && g.topk_group * per > k;
  }
  score[lane] = cs;
  __builtin_amdgcn_wave_barrier();
  my_at = 0;
  for (int i = 0; i < k; i += 4) {
    double oc[4];
    int oe[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      oc[u] = score[row + min(i + u, k - 1)];
      oe[u] = pick[row + min(i + u, k - 1)];
    }
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (i + u < k) my_at += (oc[u] > cs || (oc[u] == cs && oe[u] < my_e)) ? 1 : 0;
  }
  __builtin_amdgcn_wave_barrier();
  if (g.renorm) {
    const double sum = row_sum(s);
    s = sum > 0.0 ? s / sum : 0.0;
  }
  my_w = (float)(s * (double)g.scale);
  return row_sum(wrong ? 1 : 0) == 0;
}

}  // namespace
}  // namespace moe
