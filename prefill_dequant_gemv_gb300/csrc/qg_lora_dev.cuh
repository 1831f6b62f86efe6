// Device functions shared by the low-rank adapters' kernels: the rows of every adapter as tiles,
// and the warp-level product.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "qg_lora.h"
#include "qg_sync.cuh"

namespace qg {

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float bf_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf_hi(uint32_t u) { return __uint_as_float(u & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {  // a in the low half
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// 16 (or 8) bytes global -> shared, those past the first `bytes` (0: none is read) as zeros.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy8(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// Bytes of a piece of eight elements of which `left` remain.
__device__ __forceinline__ int bytes_of(int left) { return 2 * max(0, min(8, left)); }

// The first of a value's two bf16 terms (in the upper half): the next one below its magnitude, so that the second has its sign and
// neither is 0 unless the value is.  Then an infinite element of B gives the infinity of the formula, not inf - inf or inf * 0, and
// a value beyond bf16's largest number stays finite.  (Below 2^-110 the second may be 0.)
__device__ __forceinline__ uint32_t first_term(float x) {
  const uint32_t u = __float_as_uint(x);
  return (u & 0x7FFFFFFFu) ? (u - 1u) & 0xFFFF0000u : u;
}
// Two h as two bf16 terms each: 16 bits of the value (the second is at most one step of the first, and rounds by 2^-16 of the value).
__device__ __forceinline__ void split_h2(float x, float y, uint32_t& top, uint32_t& rest) {
  const uint32_t a = first_term(x), b = first_term(y);
  top = b | a >> 16;
  rest = pack_bf16(x - __uint_as_float(a), y - __uint_as_float(b));
}
// scale times eight h, those from `valid` on (ranks past the adapter's) as zeros.
__device__ __forceinline__ void split_h(const float (&v)[8], float scale, int valid, uint4& top, uint4& rest) {
  uint32_t a[4], b[4];
#pragma unroll
  for (int j = 0; j < 4; ++j)
    split_h2(2 * j < valid ? v[2 * j] * scale : 0.0f, 2 * j + 1 < valid ? v[2 * j + 1] * scale : 0.0f, a[j], b[j]);
  top = make_uint4(a[0], a[1], a[2], a[3]);
  rest = make_uint4(b[0], b[1], b[2], b[3]);
}

// Exclusive prefix sum of one count a thread over a block of THREADS; the total in *total.
template <int THREADS>
__device__ __forceinline__ int block_prefix(int v, int* warp_sums, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int s = v;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int o = __shfl_up_sync(0xFFFFFFFFu, s, off);
    if (lane >= off) s += o;
  }
  if (lane == 31) warp_sums[warp] = s;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    const int c = warp_sums[w];
    before += w < warp ? c : 0;
    all += c;
  }
  __syncthreads();
  *total = all;
  return before + s - v;
}

// Adapter of a row, n_adapters for none (and for an id out of range).
__device__ __forceinline__ int bin_of(int id, int n_adapters) { return (unsigned)id < (unsigned)n_adapters ? id : n_adapters; }

// Rank of adapter e (0 for the rows without one), or kBadRank: out of range, to be taken as 0 and reported if a row names it.
constexpr int kBadRank = 255;
__device__ __forceinline__ int rank_or_bad(const LoraArgs& p, int e) {
  if (e >= p.n_adapters) return 0;
  const int r = p.ranks ? p.ranks[e] : p.max_rank;
  return r >= 0 && r <= p.max_rank ? r : kBadRank;
}
__device__ __forceinline__ void report_invalid(const LoraArgs& p) { atomicCAS(p.status, 0, kStatusInvalid); }
// Rank of the adapter e < n_adapters of a row; one out of range counts as 0 and is reported.
__device__ __forceinline__ int rank_of(const LoraArgs& p, int e) {
  const int r = p.ranks ? p.ranks[e] : p.max_rank;
  if (r >= 0 && r <= p.max_rank) return r;
  report_invalid(p);
  return 0;
}

// The rows of every adapter in tiles of T, adapter by adapter; first[e] is adapter e's first tile.
// first[n_adapters]: the rows without one; first[n_adapters + 1]: the number of tiles.
// Every CTA builds the same table: ids are few bytes beside x and y.
template <int THREADS>
struct Tiles {
  int first[kLoraMaxAdapters + 2];
  int warp_sums[THREADS / 32];
  uint8_t rank[kLoraMaxAdapters + 1];

  // Also notes every row's bin, and 0xFFFF up to `padded` rows.  A warp has every THREADS / 32nd run of 32 rows; 16 runs' loads before the first use.
  __device__ __forceinline__ void count(const LoraArgs& p, int T, uint16_t* bins_of_rows, int padded) {
    const int tid = threadIdx.x, lane = tid & 31, bins = p.n_adapters + 1;
    for (int e = tid; e <= bins; e += THREADS) first[e] = 0;
    for (int i = p.m + tid; i < padded; i += THREADS) bins_of_rows[i] = 0xFFFF;
    for (int e = tid; e <= p.n_adapters; e += THREADS) rank[e] = (uint8_t)rank_or_bad(p, e);
    __syncthreads();
    bool bad = false;
    for (int i0 = tid; i0 - lane < p.m; i0 += 16 * THREADS) {
      int e[16];
#pragma unroll
      for (int u = 0; u < 16; ++u) e[u] = i0 + u * THREADS < p.m ? p.ids[i0 + u * THREADS] : -1;
#pragma unroll
      for (int u = 0; u < 16; ++u) {
        const int i = i0 + u * THREADS;
        if (i - lane >= p.m) break;
        bad |= e[u] < -1 || e[u] >= p.n_adapters;
        e[u] = i < p.m ? bin_of(e[u], p.n_adapters) : -1;
        if (i < p.m) bins_of_rows[i] = (uint16_t)e[u];
        const int one = __shfl_sync(0xFFFFFFFFu, e[u], 0);
        unsigned same = 0xFFFFFFFFu;  // rows of one adapter in a run: one sum for it
        if (!__all_sync(0xFFFFFFFFu, e[u] == one)) same = __match_any_sync(0xFFFFFFFFu, e[u]);
        if (e[u] >= 0 && lane == __ffs(same) - 1) atomicAdd(&first[e[u]], __popc(same));  // integer counts: order-free
      }
    }
    if (bad) report_invalid(p);
    __syncthreads();
    constexpr int kPer = (kLoraMaxAdapters + 1 + THREADS - 1) / THREADS;
    const int per_bin = (bins + THREADS - 1) / THREADS, e0 = tid * per_bin;
    int c[kPer], sum = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      c[i] = i < per_bin && e0 + i < bins ? (first[e0 + i] + T - 1) / T : 0;
      if (i < per_bin && e0 + i < bins && rank[e0 + i] == kBadRank) {
        rank[e0 + i] = 0;
        if (c[i]) report_invalid(p);
      }
      if (e0 + i == p.n_adapters && p.out == p.y) c[i] = 0;  // in place: nothing to do without an adapter
      sum += c[i];
    }
    int total, at = block_prefix<THREADS>(sum, warp_sums, &total);
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (i < per_bin && e0 + i < bins) {
        first[e0 + i] = at;
        at += c[i];
      }
    if (tid == 0) first[bins] = total;
    __syncthreads();
  }
};

}  // namespace qg
