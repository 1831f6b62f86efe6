// Mixture-of-experts router (TurboEXL3 article §4.1 "Route": count each expert's tokens,
// group the tokens by expert, build the table of tiles -- one pass instead of a sort;
// §4.2: the router's top-k and softmax).
//
// Per token: the top-k experts by fp32 logit (ties to the lower expert index) and the
// softmax of the k kept logits.  Then every (token, slot) pair p = t*k + j is placed in
// grouped order -- experts ascending, tokens ascending within an expert -- giving
// counts[e], offsets[e] (exclusive prefix), pair_list[pos] = p, pair_pos[p] = pos, the
// ascending list of active experts, and a tile table of (expert, first position, count)
// with at most kRouteTile pairs per tile for the grouped prefill GEMM.  Everything is
// deterministic: ranks come from ordered scans, never from atomic arrival order.
//
// Up to 8 tokens (12 of more than 256 experts, two by a rule) take one CTA, up to 64 a cluster; more a launch of the top-k with counts of
// every block of tokens, one of the sums over the blocks where they are more than 16, and one of the placement.  In a graph, 512 experts,
// topk 10: 32 tokens 6.4 us (9.3 in one CTA), 64 7.1 (12 with four launches); behind another kernel 1000 13.0 (15.7), 8192 24 (27).
#include <cuda_runtime.h>

#include "qg_internal.h"
#include "qg_route.h"
#include "qg_route_by.cuh"
#include "qg_route_dev.cuh"
#include "qg_sync.cuh"

namespace qg {

// Tokens that one cluster routes, one a warp of its eight CTAs: 64 of 512 experts by softmax and bias 6.5 us, 7.2 with two launches, 32 6.1
// and 7.4; 128, two a warp, 9.7 against 8.
constexpr int kRouteCluster = 64;
// Tokens that one CTA alone routes without a rule.  One CTA and a cluster, in a graph behind another kernel, us: 9 tokens of 64 experts
// 4.6 and 4.2, of 256 5.0 and 4.9, of 384 5.0 and 5.4, of 512 5.9 and 6.3; 12 of 384 5.3 and 5.6, of 512 5.8 and 6.0; 16 of 384 5.9 and
// 5.8, of 512 6.6 and 6.2.
inline int route_small(int E) { return E > 256 ? 12 : 8; }
constexpr int kRouteBySmall = 2;  // tokens that one CTA alone routes by a rule: two 4.9 us, by a cluster of one 5.9

// Clear a shared array with 16-byte stores (bytes a multiple of 16, 16-byte aligned).
__device__ __forceinline__ void zero_shared(void* p, int bytes) {
  uint4* q = static_cast<uint4*>(p);
  for (int i = threadIdx.x; i < bytes / 16; i += blockDim.x) q[i] = make_uint4(0, 0, 0, 0);
}

// Block-wide exclusive scan of three counters (every thread of the block calls it;
// blockDim.x a multiple of 32, <= 1024); the totals go to *tot (shared memory).
__device__ __forceinline__ int3 block_scan3(int3 x, int3* tot) {
  __shared__ int3 wsum[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  int3 inc = x;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int a = __shfl_up_sync(0xFFFFFFFFu, inc.x, off), b = __shfl_up_sync(0xFFFFFFFFu, inc.y, off),
              c = __shfl_up_sync(0xFFFFFFFFu, inc.z, off);
    if (lane >= off) {
      inc.x += a;
      inc.y += b;
      inc.z += c;
    }
  }
  if (lane == 31) wsum[warp] = inc;
  __syncthreads();
  if (warp == 0) {
    const int3 w = lane < nw ? wsum[lane] : make_int3(0, 0, 0);
    int3 wi = w;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int a = __shfl_up_sync(0xFFFFFFFFu, wi.x, off), b = __shfl_up_sync(0xFFFFFFFFu, wi.y, off),
                c = __shfl_up_sync(0xFFFFFFFFu, wi.z, off);
      if (lane >= off) {
        wi.x += a;
        wi.y += b;
        wi.z += c;
      }
    }
    if (lane < nw) wsum[lane] = make_int3(wi.x - w.x, wi.y - w.y, wi.z - w.z);  // exclusive, per warp
    if (lane == 31) *tot = wi;
  }
  __syncthreads();
  const int3 base = wsum[warp];
  __syncthreads();
  return make_int3(base.x + inc.x - x.x, base.y + inc.y - x.y, base.z + inc.z - x.z);
}

// Large router, first launch: the experts and weights of a block of tokens, a warp a token, and how many of the block's
// pairs every expert has.  S: 32 S experts at most.
template <int S, bool BY>
__global__ void __launch_bounds__(256, 3) route_topk_kernel(const float* logits, int64_t T, int E, int k, int tokens, int32_t* ids,
                                                         float* wts, RouteView r, RouteRule rule) {
  __shared__ int hist[32 * S];
  __shared__ float cs[BY ? 8 : 1][BY ? 32 * S + 32 : 1];
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) pdl_launch_dependents();
  for (int e = threadIdx.x; e < E; e += 256) hist[e] = 0;
  __syncthreads();
  pdl_wait();
  const int64_t t0 = (int64_t)blockIdx.x * tokens, t1 = t0 + tokens < T ? t0 + tokens : T;
  if constexpr (BY) {
    for (int64_t t = t0 + warp; t < t1; t += 8)
      warp_route<S>(rule, logits + t * E, E, k, cs[warp], ids + t * k, wts + t * k, nullptr, hist);
  } else {
    for (int64_t t = t0 + warp; t < t1; t += 8) warp_topk<S>(logits + t * E, E, k, ids + t * k, wts + t * k, nullptr, hist);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += 256) r.block_counts[(size_t)blockIdx.x * E + e] = hist[e];
}

// Second launch, where the blocks are many: counts become the pairs in the blocks before, and the experts' totals.  A CTA has
// 32 experts, one a lane; its warps share the blocks.
__global__ void __launch_bounds__(1024) route_prefix_kernel(int E, int nblocks, RouteView r) {
  __shared__ int part[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, e = blockIdx.x * 32 + lane;
  if (threadIdx.x == 0) pdl_launch_dependents();
  pdl_wait();
  const int per = (nblocks + 31) / 32, b0 = min(nblocks, warp * per), b1 = min(nblocks, b0 + per);
  int sum = 0;
  if (e < E)
#pragma unroll 8
    for (int b = b0; b < b1; ++b) sum += r.block_counts[(size_t)b * E + e];
  part[warp][lane] = sum;
  __syncthreads();
  int run = 0, tot = 0;
#pragma unroll
  for (int w = 0; w < 32; ++w) {
    const int c = part[w][lane];
    run += w < warp ? c : 0;
    tot += c;
  }
  if (e >= E) return;
  if (warp == 0) r.counts[e] = tot;
#pragma unroll 8
  for (int b = b0; b < b1; ++b) {
    const int c = r.block_counts[(size_t)b * E + e];
    r.block_counts[(size_t)b * E + e] = run;
    run += c;
  }
}

// Last launch: offsets, active list and tile table (stored by block 0), and the stable placement of each block's pairs:
// experts ascending, pairs ascending within an expert.  `tokens` a block, `merged` blocks of the counts.  SUM: there was no second
// launch, the block adds the counts itself.  It does not ask for the next kernel's launch: where that is another call's top-k, its
// blocks would come to lie beside one another on the SMs that are free by then (1000 tokens, 512 experts, topk 16, call after call:
// 18.3 us, 15.1 so; behind another kernel 15.0 both ways).
template <bool SUM>
__global__ void __launch_bounds__(kRouteBlock) route_place_kernel(const int32_t* ids, int64_t P, int E, int k, int tokens, int merged,
                                                                  int nblocks, int tile, RouteView r) {
  __shared__ int3 totals;
  __shared__ int start[kMaxExperts], off[kMaxExperts], zid[kMaxExperts];
  __shared__ __align__(16) unsigned short wc[kRouteBlock / 32][kMaxExperts];  // pairs per (warp, expert)
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, b = blockIdx.x;
  zero_shared(&wc[0][0], sizeof(wc));
  pdl_wait();
  int tot = 0, before = 0;
  if (tid < E) {
    if (SUM) {
#pragma unroll 8
      for (int i = 0; i < nblocks; ++i) {
        const int c = r.block_counts[(size_t)i * E + tid];
        before += i < b * merged ? c : 0;
        tot += c;
      }
    } else {
      tot = r.counts[tid];
      before = r.block_counts[(size_t)b * merged * E + tid];
    }
  }
  const int64_t p = (int64_t)b * tokens * k + tid;
  const bool valid = tid < tokens * k && p < P;
  const int e = valid ? ids[p] : -1;
  const int3 ex = block_scan3(make_int3(tot, (tot + tile - 1) / tile, tot > 0 ? 1 : 0), &totals);
  if (tid < E) {
    start[tid] = ex.x + before;
    off[tid] = ex.x;
    zid[tid] = ex.z;
    if (b == 0) {
      r.counts[tid] = tot;
      r.offsets[tid] = ex.x;
      if (tot > 0) {
        r.active[ex.z] = tid;
        r.zidx[tid] = ex.z;
        reinterpret_cast<int4*>(r.groups + (size_t)ex.z * kGroupInts)[0] = make_int4(tid, ex.x, tot, 0);
      }
      for (int s = 0; s * tile < tot; ++s) {
        r.tiles[3 * (ex.y + s)] = tid;
        r.tiles[3 * (ex.y + s) + 1] = ex.x + s * tile;
        r.tiles[3 * (ex.y + s) + 2] = min(tile, tot - s * tile);
      }
    }
  }
  if (b == 0 && tid == 0) {
    r.offsets[E] = totals.x;
    r.meta[0] = totals.z;
    r.meta[1] = totals.y;
  }
  const unsigned mask = __match_any_sync(0xFFFFFFFFu, e);
  const int rank_in_warp = __popc(mask & ((1u << lane) - 1u));
  if (valid && rank_in_warp == 0) wc[warp][e] = (unsigned short)__popc(mask);
  __syncthreads();
  if (valid) {
    int at = start[e] + rank_in_warp;
    for (int w = 0; w < warp; ++w) at += wc[w][e];
    r.pair_list[at] = (int)p;
    r.pair_pos[p] = at;
    const int rank = at - off[e];
    if (rank < kGroupRows) r.groups[(size_t)zid[e] * kGroupInts + 4 + rank] = (int)(p / k);
  }
}

// Decode-sized routing (T <= route_small, or kRouteBySmall by a rule): every phase in one CTA, with
// the histogram, the scan and the placement in shared memory; only the results go to device
// memory.  BY: by a rule, of up to 32 BY experts; 0: without one.
template <int BY>
__global__ void __launch_bounds__(BY ? kMaxExperts : kRouteBlock) route_small_kernel(const float* logits, int T, int E, int k,
                                                                  int32_t* ids, float* wts, int tile, RouteView r,
                                                                  RouteRule rule) {
  __shared__ int s_ids[kRouteBlock];
  __shared__ int hist[kMaxExperts];
  __shared__ int off[kMaxExperts];
  __shared__ int zid[kMaxExperts];
  __shared__ int3 totals;
  __shared__ __align__(16) unsigned short wc[kRouteBlock / 32][kMaxExperts];  // pairs per (warp, expert)
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // The consumers of the routing wait for this grid to complete before reading it; the
  // logits may come from the preceding kernel.
  if (tid == 0) pdl_launch_dependents();
  for (int e = tid; e < E; e += blockDim.x) hist[e] = 0;
  zero_shared(&wc[0][0], sizeof(wc));
  pdl_wait();
  if constexpr (BY) {
    __shared__ float cs[kRouteBySmall][32 * BY + 32];
    if (warp < T)
      warp_route<BY>(rule, logits + (int64_t)warp * E, E, k, cs[warp], ids + warp * k, wts + warp * k, s_ids + warp * k, nullptr);
  } else {
    if (warp < T) warp_topk(logits + (int64_t)warp * E, E, k, ids + warp * k, wts + warp * k, s_ids + warp * k);
  }
  __syncthreads();
  // pairs p = t*k + j: histogram (order-free integer counts) and rank within the warp
  const int P = T * k;
  const bool valid = tid < P;
  const int e = valid ? s_ids[tid] : -1;
  if (valid) atomicAdd(&hist[e], 1);
  const unsigned mask = __match_any_sync(0xFFFFFFFFu, e);
  const int rank_in_warp = __popc(mask & ((1u << lane) - 1u));
  if (valid && rank_in_warp == 0) wc[warp][e] = (unsigned short)__popc(mask);
  __syncthreads();
  // totals, exclusive offsets, active list and tile table (one thread per expert)
  const int tot = tid < E ? hist[tid] : 0;
  const int3 ex = block_scan3(make_int3(tot, (tot + tile - 1) / tile, tot > 0 ? 1 : 0), &totals);
  if (tid < E) {
    r.counts[tid] = tot;
    r.offsets[tid] = ex.x;
    off[tid] = ex.x;
    zid[tid] = ex.z;
    if (tot > 0) {
      r.active[ex.z] = tid;
      r.zidx[tid] = ex.z;
      reinterpret_cast<int4*>(r.groups + (size_t)ex.z * kGroupInts)[0] = make_int4(tid, ex.x, tot, 0);
    }
    for (int s = 0; s * tile < tot; ++s) {
      r.tiles[3 * (ex.y + s)] = tid;
      r.tiles[3 * (ex.y + s) + 1] = ex.x + s * tile;
      r.tiles[3 * (ex.y + s) + 2] = min(tile, tot - s * tile);
    }
  }
  if (tid == 0) {
    r.offsets[E] = totals.x;
    r.meta[0] = totals.z;
    r.meta[1] = totals.y;
  }
  __syncthreads();
  // stable placement: experts ascending, pairs ascending within an expert
  if (valid) {
    int before = 0;
    for (int w = 0; w < warp; ++w) before += wc[w][e];
    const int pos = off[e] + before + rank_in_warp;
    r.pair_list[pos] = tid;
    r.pair_pos[tid] = pos;
    const int rank = before + rank_in_warp;
    if (rank < kGroupRows) r.groups[(size_t)zid[e] * kGroupInts + 4 + rank] = tid / k;
  }
}

// A batch of a few dozen tokens in one launch: a cluster of CTAs, a token to each of their warps, which read one another's counts from
// shared memory.
template <int S, bool BY>
__global__ void __launch_bounds__(256) route_cluster_kernel(const float* logits, int T, int E, int k, int32_t* ids, float* wts,
                                                            int tile, RouteView r, RouteRule rule) {
  __shared__ __align__(16) int hist[kMaxExperts];
  __shared__ float cs[BY ? 8 : 1][BY ? 32 * S + 32 : 1];
  __shared__ int s_ids[8 * kMaxTopk], start[kMaxExperts], off[kMaxExperts], zid[kMaxExperts];
  __shared__ __align__(16) unsigned short wc[8][kMaxExperts];  // pairs per (warp, expert)
  __shared__ int3 totals;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, b = blockIdx.x;
  if (tid == 0) pdl_launch_dependents();
  zero_shared(hist, sizeof(hist));
  zero_shared(&wc[0][0], sizeof(wc));
  __syncthreads();
  pdl_wait();
  const int t0 = b * 8, t1 = min(t0 + 8, T), t = t0 + warp;
  if (t < t1) {
    const float* lg = logits + (int64_t)t * E;
    if constexpr (BY) warp_route<S>(rule, lg, E, k, cs[warp], ids + t * k, wts + t * k, s_ids + warp * k, hist);
    else warp_topk<S>(lg, E, k, ids + t * k, wts + t * k, s_ids + warp * k, hist);
  }
  cluster_sync_all();
  // two experts a thread: their pairs in all CTAs and in those before
  int tot[2] = {0, 0}, before[2] = {0, 0};
  const int e0 = 2 * tid;
  for (int i = 0; i < (int)gridDim.x; ++i) {
    int a, c;
    asm volatile("ld.shared::cluster.v2.s32 {%0, %1}, [%2];" : "=r"(a), "=r"(c) : "r"(cluster_map(hist + e0, (uint32_t)i)));
    before[0] += i < b ? a : 0;
    before[1] += i < b ? c : 0;
    tot[0] += a;
    tot[1] += c;
  }
  const int tiles[2] = {(tot[0] + tile - 1) / tile, (tot[1] + tile - 1) / tile};
  int3 ex = block_scan3(make_int3(tot[0] + tot[1], tiles[0] + tiles[1], (tot[0] > 0) + (tot[1] > 0)), &totals);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int e = e0 + i, n = tot[i];
    start[e] = ex.x + before[i];
    off[e] = ex.x;
    zid[e] = ex.z;
    if (b == 0 && e < E) {
      r.counts[e] = n;
      r.offsets[e] = ex.x;
      if (n > 0) {
        r.active[ex.z] = e;
        r.zidx[e] = ex.z;
        reinterpret_cast<int4*>(r.groups + (size_t)ex.z * kGroupInts)[0] = make_int4(e, ex.x, n, 0);
      }
      for (int s = 0; s < tiles[i]; ++s) {
        r.tiles[3 * (ex.y + s)] = e;
        r.tiles[3 * (ex.y + s) + 1] = ex.x + s * tile;
        r.tiles[3 * (ex.y + s) + 2] = min(tile, n - s * tile);
      }
    }
    ex.x += n;
    ex.y += tiles[i];
    ex.z += n > 0;
  }
  if (b == 0 && tid == 0) {
    r.offsets[E] = totals.x;
    r.meta[0] = totals.z;
    r.meta[1] = totals.y;
  }
  // stable placement: experts ascending, pairs ascending within an expert
  const bool valid = tid < (t1 - t0) * k;
  const int e = valid ? s_ids[tid] : -1;
  const unsigned mask = __match_any_sync(0xFFFFFFFFu, e);
  const int rank_in_warp = __popc(mask & ((1u << lane) - 1u));
  if (valid && rank_in_warp == 0) wc[warp][e] = (unsigned short)__popc(mask);
  __syncthreads();
  if (valid) {
    const int p = t0 * k + tid;
    int at = start[e] + rank_in_warp;
    for (int w = 0; w < warp; ++w) at += wc[w][e];
    r.pair_list[at] = p;
    r.pair_pos[p] = at;
    const int rank = at - off[e];
    if (rank < kGroupRows) r.groups[(size_t)zid[e] * kGroupInts + 4 + rank] = t0 + tid / k;
  }
  cluster_sync_all();  // no CTA ends before the others have read its counts
}

RouteView route_view(void* ws, int64_t T, int E, int k) {
  const RouteLayout L = route_layout(T, E, k);
  uint8_t* b = static_cast<uint8_t*>(ws);
  RouteView v;
  v.meta = reinterpret_cast<int*>(b + L.meta);
  v.counts = reinterpret_cast<int*>(b + L.counts);
  v.offsets = reinterpret_cast<int*>(b + L.offsets);
  v.active = reinterpret_cast<int*>(b + L.active);
  v.pair_list = reinterpret_cast<int*>(b + L.pair_list);
  v.pair_pos = reinterpret_cast<int*>(b + L.pair_pos);
  v.tiles = reinterpret_cast<int*>(b + L.tiles);
  v.groups = reinterpret_cast<int*>(b + L.groups);
  v.zidx = reinterpret_cast<int*>(b + L.zidx);
  v.block_counts = reinterpret_cast<int*>(b + L.block_counts);
  return v;
}

// The large router: top-k and counts, the counts' sums where there are many blocks, placement.
template <int S, bool BY>
static int launch_large(const RouteRule& rule, const float* logits, int64_t T, int E, int k, int32_t* ids, float* wts,
                        const RouteView& r, cudaStream_t s) {
  const int tokens = route_block_tokens(T, k), place = route_place_tokens(T, k), merged = place / tokens;
  const int nb = (int)((T + tokens - 1) / tokens), np = (int)((T + place - 1) / place);
  const int64_t P = T * k;
  if (launch_pdl(route_topk_kernel<S, BY>, dim3(nb), dim3(256), 0, s, logits, T, E, k, tokens, ids, wts, r, rule) != cudaSuccess)
    return QG_ERR_CUDA;
  // up to 16 blocks' counts every placing block adds in less time than a launch takes
  if (nb <= 16) {
    if (launch_pdl(route_place_kernel<true>, dim3(np), dim3(kRouteBlock), 0, s, ids, P, E, k, place, merged, nb, (int)kRouteTile, r) !=
        cudaSuccess)
      return QG_ERR_CUDA;
  } else if (launch_pdl(route_prefix_kernel, dim3((E + 31) / 32), dim3(1024), 0, s, E, nb, r) != cudaSuccess ||
             launch_pdl(route_place_kernel<false>, dim3(np), dim3(kRouteBlock), 0, s, ids, P, E, k, place, merged, nb, (int)kRouteTile,
                        r) != cudaSuccess) {
    return QG_ERR_CUDA;
  }
  return cudaGetLastError() == cudaSuccess ? QG_OK : QG_ERR_CUDA;
}

template <int S, bool BY>
static int launch_cluster(const RouteRule& rule, const float* logits, int64_t T, int E, int k, int32_t* ids, float* wts,
                          const RouteView& r, cudaStream_t s) {
  const int ctas = (int)((T + 7) / 8);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, route_cluster_kernel<S, BY>, logits, (int)T, E, k, ids, wts, (int)kRouteTile, r, rule) ==
                     cudaSuccess && cudaGetLastError() == cudaSuccess
             ? QG_OK
             : QG_ERR_CUDA;
}

template <int S>
static int launch_batch(const float* logits, int64_t T, int E, int k, int32_t* ids, float* wts, const RouteView& r, cudaStream_t s) {
  return T <= kRouteCluster ? launch_cluster<S, false>(RouteRule(), logits, T, E, k, ids, wts, r, s)
                            : launch_large<S, false>(RouteRule(), logits, T, E, k, ids, wts, r, s);
}

int launch_route(const float* logits, int64_t T, int E, int k, int32_t* ids, float* wts, void* ws, void* stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  RouteView r = route_view(ws, T, E, k);
  if (T > route_small(E))
    return E <= 128 ? launch_batch<4>(logits, T, E, k, ids, wts, r, s)
           : E <= 256 ? launch_batch<8>(logits, T, E, k, ids, wts, r, s) : launch_batch<16>(logits, T, E, k, ids, wts, r, s);
  return launch_pdl(route_small_kernel<0>, dim3(1), dim3(kRouteBlock), 0, s, logits, (int)T, E, k, ids, wts, (int)kRouteTile, r,
                    RouteRule()) == cudaSuccess && cudaGetLastError() == cudaSuccess
             ? QG_OK
             : QG_ERR_CUDA;
}

template <int S>
static int launch_by(const RouteRule& rule, const float* logits, int64_t T, int E, int k, int32_t* ids, float* wts,
                     const RouteView& r, cudaStream_t s) {
  // by a rule a token takes a warp some 3 us, and one SM's warps share its issue slots: more tokens go to more SMs
  if (T > kRouteBySmall && T <= kRouteCluster) return launch_cluster<S, true>(rule, logits, T, E, k, ids, wts, r, s);
  if (T > kRouteBySmall) return launch_large<S, true>(rule, logits, T, E, k, ids, wts, r, s);
  return launch_pdl(route_small_kernel<S>, dim3(1), dim3(kMaxExperts), 0, s, logits, (int)T, E, k, ids, wts, (int)kRouteTile, r,
                    rule) == cudaSuccess && cudaGetLastError() == cudaSuccess
             ? QG_OK
             : QG_ERR_CUDA;
}

int launch_route_by(const RouteRule& rule, const float* logits, int64_t T, int E, int k, int32_t* ids, float* wts, void* ws,
                    void* stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  RouteView r = route_view(ws, T, E, k);
  return E <= 128 ? launch_by<4>(rule, logits, T, E, k, ids, wts, r, s)
         : E <= 256 ? launch_by<8>(rule, logits, T, E, k, ids, wts, r, s) : launch_by<16>(rule, logits, T, E, k, ids, wts, r, s);
}

}  // namespace qg
