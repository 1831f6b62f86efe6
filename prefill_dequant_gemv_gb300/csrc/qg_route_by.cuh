// Choice of a token's experts by a rule (scores, bias, groups): one warp a token.
//
// The choice has to be the one that 64-bit scores give, and 64-bit arithmetic runs at a
// hundredth of the fp32 rate here.  Where the choice values c are ordered as the logits are
// (no bias, and group values that are single scores) the logits decide.  Otherwise c is
// computed in fp32; the token is decided there if every two values whose order matters lie
// further apart than twice the error of c, and redone in 64 bits if not (one token in some
// thousand): first only the experts that can be among the topk, one a lane; or all of them
// where the groups are in doubt, or more than 32 experts are.
//
// Error of c in fp32 (u = 2^-24): __expf(x) is within 2 + 1.173 |x| ulps, an ulp being 2 u at most, the approximate
// reciprocal within one.  Sigmoid: e^-l enters s with the weight s (1 - s), which leaves less than 0.65 ulps of it; 1 + e and the
// reciprocal add 3 u: s is off by less than 5 u.  Softmax: with d = max - l, the terms e^-d are off by 2 u (2 + 1.173 d) e^-d and
// their argument's rounding by u d e^-d, together below 6 u of the largest; in the sum S >= 1 the mean of d over e^-d / S is
// at most log 512, so S is off by 2 (2 + 1.173 * 6.3) + 6.3 u, its 21 additions by 21 u, its reciprocal by 2 u: s
// is off by less than 56 u / S.  The sum with the bias adds u |c|.  Two values may be off by twice that: the tolerance is 2^-20
// (sigmoid; 16 u) or 2^-17 / S (softmax; 128 u), and 2^-22 |c| (4 u).  A sum of two c is off by the errors of both, u times
// each one's magnitude among them, and by its own rounding; the magnitudes may be far larger than the sum, so that the tolerance of two such
// sums is twice the first part and 2^-21 of the largest |c| + |c'| (8 u, of which 4 u are needed).
//
// What bounds many tokens is a warp's instructions, one after the other (issue 54%; a token of 512 experts by sigmoid and bias
// 1062).  So the winners are not taken one by one from all experts, in rounds that a warp's reductions make long (1539
// instructions, 27.6 us for 8192 tokens under ncu against 20.9): the k-th largest of the lanes' largest values is below the winners, the few experts
// above it go to one lane each, and each counts those that come before it.
//
// Measured in a graph, call after call, tables included (us): one token of 256 experts in groups 4.8, 64 of 512 by softmax and bias 6.6,
// 8192 by sigmoid and bias 26 (their logits at the copy rate: 2.5), 8192 of 256 in groups 27, 5001 of 160 in groups by softmax 16.7, without
// renormalising 17.2.  A near tie of sigmoids adds 2 us to a call, of softmax 3, or 16 where the softmax's sum is redone.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "qg_route.h"
#include "qg_route_dev.cuh"

namespace qg {

// Score of a logit in 64 bits: sigmoid, or softmax with the largest logit m and 1 / S.
__device__ __forceinline__ double score_of(const RouteRule& r, double l, double m, double inv) {
  return r.sigmoid ? 1.0 / (1.0 + exp(-l)) : exp(l - m) * inv;
}
// The same in fp32, with the error above.
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float quick_score(const RouteRule& r, float l, float m, float inv) {
  return r.sigmoid ? rcp_approx(1.0f + __expf(-l)) : __expf(l - m) * inv;
}

// A lane's share of a softmax's sum as the weights need it: expf, added in pairs (S: a power of two), so that a large term
// meets log2 S roundings and not S.
template <int S>
__device__ __forceinline__ float exp_sum(const float (&c)[S], float m) {
  float part[6];  // part[b]: of the 2^b terms before, where they are complete
  int b = 0;
#pragma unroll
  for (int i = 0; i < S; ++i) {
    float v = c[i] == c[i] ? expf(c[i] - m) : 0.0f;  // NaN: no expert, or one left out
#pragma unroll
    for (b = 0; i >> b & 1; ++b) v = part[b] + v;
    part[b] = v;
  }
  return part[b];
}

// The two largest of a and b's (a0 >= a1, b0 >= b1).
template <class F>
__device__ __forceinline__ void merge2(F& a0, F& a1, F b0, F b1) {
  const F x = a0 < b0 ? a0 : b0;
  a0 = a0 < b0 ? b0 : a0;
  a1 = a1 < b1 ? b1 : a1;
  a1 = a1 < x ? x : a1;
}

// Bit g set: group g is among the `kept` of largest value (lane g holds group g's; ties to the lower).
// `gap`: the smallest kept value less the largest other one (NaN counts as -infinity).
template <class F>
__device__ __forceinline__ uint32_t keep_groups(F value, int n, int kept, F* gap) {
  const int lane = threadIdx.x & 31;
  if (!(value == value)) value = -F(INFINITY);
  int rank = 0;
  for (int i = 0; i < n; ++i) {
    const F o = __shfl_sync(0xFFFFFFFFu, value, i);
    rank += o > value || (o == value && i < lane);
  }
  const bool in = lane < n && rank < kept;
  F low = in ? value : F(INFINITY), top = lane < n && !in ? value : -F(INFINITY);
#pragma unroll
  for (int off = 16; off; off >>= 1) {
    const F a = __shfl_xor_sync(0xFFFFFFFFu, low, off), b = __shfl_xor_sync(0xFFFFFFFFu, top, off);
    low = a < low ? a : low;
    top = b > top ? b : top;
  }
  *gap = low - top;
  return __ballot_sync(0xFFFFFFFFu, in);
}

__device__ __forceinline__ int group_of(const RouteRule& r, int e) { return (int)(((uint32_t)e * r.group_mul) >> 20); }

// Everything in 64 bits: the slot (0 .. k-1) of this lane's winner goes to *slot (-1: none), its
// expert to *id.  Rare; kept out of line so that it costs the other tokens no registers.
__device__ __noinline__ void route_exact(const RouteRule& r, const float* lg, int E, int k, int* slot, int* id) {
  const int lane = threadIdx.x & 31;
  double m = -INFINITY, s = 0.0;
  if (!r.sigmoid) {
    for (int e = lane; e < E; e += 32) m = fmax(m, (double)lg[e]);  // a NaN is passed over
#pragma unroll
    for (int off = 16; off; off >>= 1) m = fmax(m, __shfl_xor_sync(0xFFFFFFFFu, m, off));
    for (int e = lane; e < E; e += 32) s += lg[e] == lg[e] ? exp((double)lg[e] - m) : 0.0;
#pragma unroll
    for (int off = 16; off; off >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, off);
  }
  const double inv = 1.0 / s;
  double c[16];
#pragma unroll 1
  for (int i = 0; i < 16; ++i) {
    const int e = lane + 32 * i;
    if (e < E) c[i] = score_of(r, lg[e], m, inv) + (r.bias ? (double)r.bias[e] : 0.0);
  }
  uint32_t groups = 0xFFFFFFFFu;
  if (r.n_groups > 1) {
    double value = -INFINITY;
    for (int g = 0; g < r.n_groups; ++g) {
      double a0 = -INFINITY, a1 = -INFINITY;
      for (int i = 0; i < 16; ++i) {
        const int e = lane + 32 * i;
        if (e < E && group_of(r, e) == g && c[i] == c[i]) merge2(a0, a1, c[i], -(double)INFINITY);
      }
      for (int off = 16; off; off >>= 1)
        merge2(a0, a1, __shfl_xor_sync(0xFFFFFFFFu, a0, off), __shfl_xor_sync(0xFFFFFFFFu, a1, off));
      if (lane == g) value = r.group_best == 2 ? a0 + a1 : a0;
    }
    double gap;
    groups = keep_groups(value, r.n_groups, r.topk_groups, &gap);
  }
  uint32_t open = 0;  // this lane's experts that may still be taken
  for (int i = 0; i < 16; ++i) {
    const int e = lane + 32 * i;
    if (e < E && (r.n_groups == 1 || (groups >> group_of(r, e) & 1))) open |= 1u << i;
  }
  *slot = -1;
  *id = 0;
  for (int j = 0; j < k; ++j) {
    double best = 0.0;
    int who = 1 << 20;  // no expert; a NaN comes after every number, -infinity among them
    for (int i = 0; i < 16; ++i)
      if (open >> i & 1) {
        const bool num = c[i] == c[i];
        const bool better = who == 1 << 20 || (num && !(best == best)) || c[i] > best;
        if (better) {
          best = c[i];
          who = lane + 32 * i;
        }
      }
#pragma unroll
    for (int off = 16; off; off >>= 1) {
      const double ob = __shfl_xor_sync(0xFFFFFFFFu, best, off);
      const int ow = __shfl_xor_sync(0xFFFFFFFFu, who, off);
      const bool on = ob == ob, mn = best == best;
      const bool equal = on == mn && (!on || ob == best);
      const bool take = ow != 1 << 20 && (who == 1 << 20 || (on && !mn) || (on && mn && ob > best) || (equal && ow < who));
      best = take ? ob : best;
      who = take ? ow : who;
    }
    if ((who & 31) == lane) open &= ~(1u << (who >> 5));
    if (lane == j) {
      *slot = j;
      *id = who;
    }
  }
}

// One over the sum of a softmax in 64 bits; m its largest logit.
__device__ __forceinline__ double exact_inverse(const RouteRule& r, const float* lg, int E, float m) {
  if (r.sigmoid) return 1.0;
  double s = 0.0;
#pragma unroll 4
  for (int e = threadIdx.x & 31; e < E; e += 32) s += lg[e] == lg[e] ? exp((double)lg[e] - m) : 0.0;
#pragma unroll
  for (int off = 16; off; off >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, off);
  return 1.0 / s;
}

// The topk of `count` (k to 32) experts in `list` by their values in 64 bits, one a lane: as route_exact.  The sum of a softmax is
// the dear part: first `near_inv`, its inverse in fp32, is taken for it, whose error is one factor of all s and so moves c_i
// against c_j by less than 2^-18 |s_i - s_j|; the sum is redone in 64 bits if two values are not further apart than that
// (and equal logits and biases are not the reason).
__device__ __noinline__ void route_listed(const RouteRule& r, const float* lg, int E, int k, float m, float near_inv, const int* list,
                                          int count, int* slot, int* id) {
  const int lane = threadIdx.x & 31, e = lane < count ? list[lane] : 1 << 20;
  const float l = lane < count ? lg[e] : 0.0f, b = lane < count && r.bias ? r.bias[e] : 0.0f;
  const double s1 = score_of(r, l, m, 1.0);
  double s = r.sigmoid ? s1 : s1 * (double)near_inv;
  int rank;
  for (int turn = 0; turn < 2; ++turn) {
    const double d = lane < count ? s + (double)b : -(double)INFINITY;
    bool doubt = false;
    rank = 0;
    for (int i = 0; i < count; ++i) {
      const double o = __shfl_sync(0xFFFFFFFFu, d, i);
      const int oe = __shfl_sync(0xFFFFFFFFu, e, i);
      rank += o > d || (o == d && oe < e);
      if (!r.sigmoid && !turn) {
        const double os = __shfl_sync(0xFFFFFFFFu, s, i);
        const float ol = __shfl_sync(0xFFFFFFFFu, l, i), ob = __shfl_sync(0xFFFFFFFFu, b, i);
        doubt |= !(fabs(o - d) > 0x1p-18 * fabs(os - s) + 0x1p-48 * fabs(d)) && !(ol == l && ob == b);
      }
    }
    if (r.sigmoid || turn || !__any_sync(0xFFFFFFFFu, doubt && lane < count)) break;
    s = s1 * exact_inverse(r, lg, E, m);
  }
  *slot = lane < count && rank < k ? rank : -1;
  *id = e;
}

// The kept groups by values in 64 bits; `list` has the experts that can be among the best of their groups (up to 32).
__device__ __noinline__ uint32_t groups_listed(const RouteRule& r, const float* lg, int E, float m, const int* list, int count) {
  const int lane = threadIdx.x & 31, e = lane < count ? list[lane] : 0, g = group_of(r, e);
  const double inv = exact_inverse(r, lg, E, m);
  const double d = lane < count ? score_of(r, lg[e], m, inv) + (r.bias ? (double)r.bias[e] : 0.0) : 0.0;
  double a0 = -INFINITY, a1 = -INFINITY, gap;
  for (int i = 0; i < count; ++i) {
    const double o = __shfl_sync(0xFFFFFFFFu, d, i);
    if (__shfl_sync(0xFFFFFFFFu, g, i) == lane) merge2(a0, a1, o, -(double)INFINITY);
  }
  return keep_groups(r.group_best == 2 ? a0 + a1 : a0, r.n_groups, r.topk_groups, &gap);
}

// The experts l + 32 i for the bits i of lane l's mask, in `list`; how many (past 32: none is written).
__device__ __forceinline__ int list_experts(uint32_t mask, int* list) {
  const int lane = threadIdx.x & 31, count = __reduce_add_sync(0xFFFFFFFFu, __popc(mask));
  if (count > 32) return count;
  int at = __popc(mask);
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int o = __shfl_up_sync(0xFFFFFFFFu, at, off);
    if (lane >= off) at += o;
  }
  at -= __popc(mask);
  __syncwarp();
  for (; mask; mask &= mask - 1) list[at++] = lane + 32 * (__ffs(mask) - 1);
  __syncwarp();
  return count;
}

// A warp's choice for one token of up to 32 S experts: ids and weights, and a copy of the ids and a count of them in hist
// where they are given.  `cs`: 32 S + 32 floats of shared memory, the warp's own.  Of the logits and biases only the choice values
// stay in registers (three blocks of warps an SM instead of two); what is rare reads them again.
template <int S>
__device__ __forceinline__ void warp_route(const RouteRule& r, const float* lg, int E, int k, float* cs, int32_t* ids, float* wts,
                                           int* ids_copy, int* hist) {
  const int lane = threadIdx.x & 31;
  float c[S];  // the logits first: lane l has expert l + 32 i's in c[i], NaN where there is none
#pragma unroll
  for (int i = 0; i < S; ++i) c[i] = lane + 32 * i < E ? lg[lane + 32 * i] : __int_as_float(0x7FC00000);
  float m = -INFINITY, inv = 1.0f;
  if (!r.sigmoid && (r.values || !r.renormalise)) {
#pragma unroll
    for (int i = 0; i < S; ++i) m = fmaxf(m, c[i]);  // a NaN is passed over
#pragma unroll
    for (int off = 16; off; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, off));
    float s = 0.0f;
    if (r.renormalise) {  // the sum enters the choice alone
#pragma unroll
      for (int i = 0; i < S; ++i) s += c[i] == c[i] ? __expf(c[i] - m) : 0.0f;
    } else {
      s = exp_sum(c, m);
    }
#pragma unroll
    for (int off = 16; off; off >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, off);
    inv = r.renormalise ? rcp_approx(s) : __frcp_rn(s);
  }
  float near = 0.0f;  // and 2^-22 |c|
  if (r.values) {
    near = r.sigmoid ? 0x1p-20f : 0x1p-17f * inv;
    float bias[S];
#pragma unroll
    for (int i = 0; i < S; ++i) bias[i] = r.bias && lane + 32 * i < E ? r.bias[lane + 32 * i] : 0.0f;
#pragma unroll
    for (int i = 0; i < S; ++i) c[i] = quick_score(r, c[i], m, inv) + bias[i];
  }
  uint32_t open = 0xFFFFFFFFu;  // bit i: the lane's expert i may be chosen
  bool doubt = false;
  if (r.n_groups > 1) {
#pragma unroll
    for (int i = 0; i < S; ++i) cs[lane + 32 * i] = c[i];
    __syncwarp();
    // `per` lanes (a power of two) to a group, each over every per-th of its experts
    const int per = r.group_lanes, size = E / r.n_groups, g = lane / per;
    float a0 = -INFINITY, a1 = -INFINITY;
    if (g < r.n_groups)
      for (int i = lane % per; i < size; i += per) {
        const float v = cs[g * size + i];
        if (v == v) merge2(a0, a1, v, -INFINITY);
      }
    for (int off = per >> 1; off; off >>= 1)
      merge2(a0, a1, __shfl_xor_sync(0xFFFFFFFFu, a0, off), __shfl_xor_sync(0xFFFFFFFFu, a1, off));
    a0 = __shfl_sync(0xFFFFFFFFu, a0, (lane * per) & 31);
    a1 = __shfl_sync(0xFFFFFFFFu, a1, (lane * per) & 31);
    const float value = r.group_best == 2 ? a0 + a1 : a0;
    // the summands' magnitudes (past fp32's range: no group is clearly apart); infinite ones have no error
    const float mag = r.group_best == 2 ? (fabsf(a1) < INFINITY ? fabsf(a0) + fabsf(a1) : 0.0f) : fabsf(a0);
    float gap, size_of = lane < r.n_groups && fabsf(a0) < INFINITY ? mag : 0.0f;
    uint32_t groups = keep_groups(value, r.n_groups, r.topk_groups, &gap);
    if (r.values && r.topk_groups < r.n_groups) {
      size_of = __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(size_of)));
      if (!(gap > 2.0f * near + 0x1p-21f * size_of)) {
        // the groups' order hangs on values that are near each other: their best experts, and those near them, in 64 bits
        __syncwarp();
        const float last = r.group_best == 2 ? a1 : a0;
        if (lane < r.n_groups) cs[lane] = last == INFINITY ? last : last - (near + 0x1p-22f * fabsf(last));
        __syncwarp();
        uint32_t best = 0;
#pragma unroll
        for (int i = 0; i < S; ++i)
          if (lane + 32 * i < E && c[i] >= cs[group_of(r, lane + 32 * i)]) best |= 1u << i;
        int* list = reinterpret_cast<int*>(cs) + 32 * S;
        const int count = list_experts(best, list);
        doubt = count > 32;
        if (!doubt) groups = groups_listed(r, lg, E, m, list, count);
        __syncwarp();
#pragma unroll
        for (int i = 0; i < S; ++i) cs[lane + 32 * i] = c[i];  // (the groups' values lay there)
      }
    }
    open = 0;
#pragma unroll
    for (int i = 0; i < S; ++i) {
      const bool in = groups >> (group_of(r, lane + 32 * i) & 31) & 1;  // past the experts: any
      open |= in ? 1u << i : 0u;
      c[i] = in ? c[i] : __int_as_float(0x7FC00000);
    }
    __syncwarp();
  }
  int slot = -1, id = 0;
  // The winners are among the candidates: the experts that come up to the k-th largest of the lanes' largest values, or within
  // the tolerance of it.  They are some k to 2 k, one a lane, and each counts those before it.
  int* list = reinterpret_cast<int*>(cs) + 32 * S;
  int count = 0;
  if (!doubt) {
    float best = -INFINITY;
#pragma unroll
    for (int i = 0; i < S; ++i) best = fmaxf(best, c[i]);  // a NaN is passed over
    uint32_t key = order_key(best), kth = 0u;
    for (int j = 0; j < k; ++j) {
      kth = __reduce_max_sync(0xFFFFFFFFu, key);
      key = key == kth ? 0u : key;
    }
    const float top = key_value(kth), least = top - (near + (r.values ? 0x1p-22f * fabsf(top) : 0.0f));
    uint32_t may = 0;
#pragma unroll
    for (int i = 0; i < S; ++i) may |= c[i] >= least ? 1u << i : 0u;
    if (r.n_groups == 1) {
#pragma unroll
      for (int i = 0; i < S; ++i) cs[lane + 32 * i] = c[i];
    }
    count = list_experts(may, list);
  }
  if (count >= k && count <= 32) {
    const int e = lane < count ? list[lane] : 1 << 20;
    const float v = lane < count ? cs[e] : -INFINITY, tol = near + 0x1p-22f * fabsf(v);
    int rank = 0, close = 0;
    for (int i = 0; i < count; ++i) {
      const float o = __shfl_sync(0xFFFFFFFFu, v, i);
      const int oe = __shfl_sync(0xFFFFFFFFu, e, i);
      rank += o > v || (o == v && oe < e);
      close += fabsf(o - v) <= tol;
    }
    slot = lane < count && rank < k ? rank : -1;
    id = e;
    if (r.values && __any_sync(0xFFFFFFFFu, slot >= 0 && close > 1)) {
      // equal values of equal logits and biases are ties indeed, and the lower index has come first
      const float l = lane < count ? lg[e] : 0.0f, b = lane < count && r.bias ? r.bias[e] : 0.0f;
      bool other = false;
      for (int i = 0; i < count; ++i) {
        const float o = __shfl_sync(0xFFFFFFFFu, v, i), ol = __shfl_sync(0xFFFFFFFFu, l, i), ob = __shfl_sync(0xFFFFFFFFu, b, i);
        other |= fabsf(o - v) <= tol && !(ol == l && ob == b);
      }
      if (__any_sync(0xFFFFFFFFu, slot >= 0 && other)) route_listed(r, lg, E, k, m, inv, list, count, &slot, &id);
    }
  } else if (!doubt) {  // many equal values, or fewer numbers than winners
    uint32_t key[S], mine, top;
#pragma unroll
    for (int i = 0; i < S; ++i) key[i] = lane + 32 * i < E && (open >> i & 1) ? order_key(c[i]) : 0u;
    warp_topk_keys(key, k, mine, id, top);
    slot = lane < k ? lane : -1;
    if (r.values) {
      // equal values of equal logits and biases are ties; any other two that are near each other, among the winners or the
      // last of them and the rest, are decided in 64 bits
      const float v = key_value(mine), vk = __shfl_sync(0xFFFFFFFFu, v, k - 1);
      const float vn = __shfl_down_sync(0xFFFFFFFFu, v, 1), least = vk - (near + 0x1p-22f * fabsf(vk));
      const float lm = lane < k ? lg[id] : 0.0f, bm = lane < k && r.bias ? r.bias[id] : 0.0f;
      const float lk = __shfl_sync(0xFFFFFFFFu, lm, k - 1), bk = __shfl_sync(0xFFFFFFFFu, bm, k - 1);
      const float ln = __shfl_down_sync(0xFFFFFFFFu, lm, 1), bn = __shfl_down_sync(0xFFFFFFFFu, bm, 1);
      const bool close = lane + 1 < k && v - vn <= near + 0x1p-22f * fabsf(v) && !(lm == ln && bm == bn);
      uint32_t other = 0;
#pragma unroll
      for (int i = 0; i < S; ++i) {
        const int e = lane + 32 * i;
        if (c[i] >= least && !(lg[e] == lk && (!r.bias || r.bias[e] == bk))) other |= 1u << i;
      }
      const int others = __reduce_add_sync(0xFFFFFFFFu, __popc(other));
      const int chosen = __popc(__ballot_sync(0xFFFFFFFFu, lane < k && v >= least && !(lm == lk && bm == bk)));
      doubt = __any_sync(0xFFFFFFFFu, close) || others != chosen;
    }
  }
  __syncwarp();
  if (doubt) route_exact(r, lg, E, k, &slot, &id);
  // weights of the winners, in fp32
  const float lw = slot >= 0 ? lg[id] : 0.0f;
  float w = 0.0f;
  if (r.renormalise) {
    // relative to the largest of them, so that a sum of small scores is no 0
    float big = slot >= 0 ? lw : -INFINITY;
#pragma unroll
    for (int off = 16; off; off >>= 1) big = fmaxf(big, __shfl_xor_sync(0xFFFFFFFFu, big, off));
    if (r.sigmoid)
      w = lw > 0.0f ? 1.0f / (1.0f + expf(-lw)) : expf(lw - fminf(big, 0.0f)) / (1.0f + expf(lw));
    else  // NaN with a logit of +infinity, also where the index has chosen (a bias, every score NaN) and left it out
      w = m < INFINITY ? expf(lw - big) : __int_as_float(0x7FC00000);
    w = slot >= 0 ? w : 0.0f;
    float s = w;
#pragma unroll
    for (int off = 16; off; off >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, off);
    w = w / s;
  } else {
    w = !r.sigmoid ? expf(lw - m) * inv : lw < 0.0f ? expf(lw) / (1.0f + expf(lw)) : 1.0f / (1.0f + expf(-lw));
  }
  if (slot >= 0) {
    ids[slot] = id;
    wts[slot] = w * r.scale;
    if (ids_copy) ids_copy[slot] = id;
    if (hist) atomicAdd(&hist[id], 1);  // integer counts: order-free
  }
}

}  // namespace qg
