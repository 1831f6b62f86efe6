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
// Error of c in fp32 (u = 2^-24): expf is within 2 u (relative), as is the reciprocal.  Sigmoid:
// 1 + e and its reciprocal add 3 u: s is off by less than 6 u s <= 6 u.  Softmax: the
// argument l - max is rounded (u |l - max|, at most 0.4 u of s = exp(l - max) / S relative to the
// largest), S adds 21 sums of positive terms, its terms' errors and the arguments' rounding,
// below 40 u together: s is off by less than 48 u / S.  The sum with the bias adds u |c|.  The
// tolerance is twice that error and a margin: 2^-20 (sigmoid) or 2^-17 / S (softmax), and
// 2^-22 |c|; for sums of two c twice as much.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "qg_route.h"
#include "qg_route_dev.cuh"

namespace qg {

// Score of a logit: sigmoid, or softmax with the largest logit m and 1 / S.
template <class F>
__device__ __forceinline__ F score_of(const RouteRule& r, F l, F m, F inv) {
  if (r.sigmoid) return F(1) / (F(1) + (sizeof(F) == 4 ? F(expf(-(float)l)) : F(exp(-(double)l))));
  return (sizeof(F) == 4 ? F(expf((float)(l - m))) : F(exp((double)(l - m)))) * inv;
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
    if (e < E) c[i] = score_of<double>(r, lg[e], m, inv) + (r.bias ? (double)r.bias[e] : 0.0);
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

// A warp's choice for one token: ids and weights (and a copy of the ids).  `cs`: E floats of shared memory, the warp's own.
__device__ __forceinline__ void warp_route(const RouteRule& r, const float* lg, int E, int k, float* cs, int32_t* ids, float* wts,
                                           int* ids_copy) {
  const int lane = threadIdx.x & 31;
  float l[16];
  float m = -INFINITY, inv = 1.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int e = lane + 32 * i;
    l[i] = e < E ? lg[e] : __int_as_float(0x7FC00000);
    m = fmaxf(m, l[i]);  // a NaN is passed over
  }
  if (!r.sigmoid && (r.values || !r.renormalise)) {
#pragma unroll
    for (int off = 16; off; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, off));
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) s += l[i] == l[i] ? expf(l[i] - m) : 0.0f;
#pragma unroll
    for (int off = 16; off; off >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, off);
    inv = 1.0f / s;
  }
  float c[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int e = lane + 32 * i;
    c[i] = l[i];
    if (r.values && e < E) c[i] = score_of<float>(r, l[i], m, inv) + (r.bias ? r.bias[e] : 0.0f);
  }
  const float near = r.values ? (r.sigmoid ? 0x1p-20f : 0x1p-17f * inv) : 0.0f;  // and 2^-22 |c|
  bool doubt = false;
  uint32_t groups = 0xFFFFFFFFu;
  if (r.n_groups > 1) {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (lane + 32 * i < E) cs[lane + 32 * i] = c[i];
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
    float value = r.group_best == 2 ? a0 + a1 : a0;
    value = __shfl_sync(0xFFFFFFFFu, value, (lane * per) & 31);
    float gap;
    groups = keep_groups(value, r.n_groups, r.topk_groups, &gap);
    float size_of = lane < r.n_groups && fabsf(value) < INFINITY ? fabsf(value) : 0.0f;
#pragma unroll
    for (int off = 16; off; off >>= 1) size_of = fmaxf(size_of, __shfl_xor_sync(0xFFFFFFFFu, size_of, off));
    doubt = r.values && r.topk_groups < r.n_groups && !(gap > 2.0f * near + 0x1p-21f * size_of);
    __syncwarp();
  }
  int slot = -1, id = 0;
  if (!doubt) {
    uint32_t key[16], open = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int e = lane + 32 * i;
      const bool in = e < E && (r.n_groups == 1 || (groups >> group_of(r, e) & 1));
      key[i] = in ? order_key(c[i]) : 0u;
      open |= in ? 1u << i : 0u;
    }
    uint32_t mine, top;
    warp_topk_keys(key, k, mine, id, top);
    slot = lane < k ? lane : -1;
    if (r.values) {
      const float v = key_value(mine), vk = __shfl_sync(0xFFFFFFFFu, v, k - 1);
      const float lm = lane < k ? lg[id] : 0.0f, bm = lane < k && r.bias ? r.bias[id] : 0.0f;
      const float lk = __shfl_sync(0xFFFFFFFFu, lm, k - 1), bk = __shfl_sync(0xFFFFFFFFu, bm, k - 1);
      // two winners in a row: near, and not the same logit and bias (then it is a tie indeed)
      const float vn = __shfl_down_sync(0xFFFFFFFFu, v, 1), ln = __shfl_down_sync(0xFFFFFFFFu, lm, 1),
                  bn = __shfl_down_sync(0xFFFFFFFFu, bm, 1);
      const bool close = lane + 1 < k && v - vn <= near + 0x1p-22f * fabsf(v) && !(lm == ln && bm == bn);
      // experts that may belong to the topk: at the last winner's value or less than the tolerance below it
      const float least = vk - (near + 0x1p-22f * fabsf(vk));
      uint32_t may = 0, other = 0;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int e = lane + 32 * i;
        if ((open >> i & 1) && c[i] >= least) {
          may |= 1u << i;
          if (!(l[i] == lk && (!r.bias || r.bias[e] == bk))) other |= 1u << i;
        }
      }
      const int others = __reduce_add_sync(0xFFFFFFFFu, __popc(other));
      const int chosen = __popc(__ballot_sync(0xFFFFFFFFu, lane < k && v >= least && !(lm == lk && bm == bk)));
      if (__any_sync(0xFFFFFFFFu, close) || others != chosen) {
        const int count = __reduce_add_sync(0xFFFFFFFFu, __popc(may));
        if (count > 32 || count < k) {
          doubt = true;
        } else {  // one of them a lane, in 64 bits
          int at = __popc(may);
#pragma unroll
          for (int off = 1; off < 32; off <<= 1) {
            const int o = __shfl_up_sync(0xFFFFFFFFu, at, off);
            if (lane >= off) at += o;
          }
          at -= __popc(may);
          int* list = reinterpret_cast<int*>(cs);
          for (int i = 0; i < 16; ++i)
            if (may >> i & 1) list[at++] = lane + 32 * i;
          __syncwarp();
          id = lane < count ? list[lane] : 1 << 20;
          __syncwarp();
          double dm = 0.0, dinv = 1.0;
          if (!r.sigmoid) {
            dm = m;
            double s = 0.0;
#pragma unroll 1
            for (int e = lane; e < E; e += 32) s += lg[e] == lg[e] ? exp((double)lg[e] - dm) : 0.0;
#pragma unroll
            for (int off = 16; off; off >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, off);
            dinv = 1.0 / s;
          }
          const double d = lane < count ? score_of<double>(r, lg[id], dm, dinv) + (r.bias ? (double)r.bias[id] : 0.0)
                                        : -(double)INFINITY;
          int rank = 0;
          for (int i = 0; i < count; ++i) {
            const double o = __shfl_sync(0xFFFFFFFFu, d, i);
            const int oi = __shfl_sync(0xFFFFFFFFu, id, i);
            rank += o > d || (o == d && oi < id);
          }
          slot = lane < count && rank < k ? rank : -1;
        }
      }
    }
  }
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
    else
      w = expf(lw - big);
    w = slot >= 0 ? w : 0.0f;
    float s = w;
#pragma unroll
    for (int off = 16; off; off >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, off);
    w = w / s;
  } else {
    w = r.sigmoid && lw < 0.0f ? expf(lw) / (1.0f + expf(lw)) : score_of<float>(r, lw, m, inv);
  }
  if (slot >= 0) {
    ids[slot] = id;
    wts[slot] = w * r.scale;
    if (ids_copy) ids_copy[slot] = id;
  }
}

}  // namespace qg
