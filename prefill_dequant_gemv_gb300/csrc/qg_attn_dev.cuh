// Device helpers of the attention kernels: bounded waits, conversions between fp16 and E4M3, TMA of page
// boxes, and the E4M3 MMAs (tcgen05, kind::f8f6f4).
#pragma once

#include <cuda.h>
#include <stdint.h>

#include "qg_sync.cuh"

namespace qg {

constexpr float kLog2e = 1.4426950408889634f;

// mbar_wait_bounded in few instructions: this kernel's many roles share one instruction cache.
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, int* status) {
  if (mbar_try_wait(bar, parity)) return true;
  const unsigned long long t0 = global_ns();
  do {
    if (mbar_try_wait_sleep(bar, parity, 1000000u)) return true;
  } while (global_ns() - t0 < kWaitLimitNs);
  atomicExch(status, kStatusTimeout);
  return false;
}
// Ordinary accesses of global and shared memory before bulk copies of the same.
__device__ __forceinline__ void fence_proxy_async_all() { asm volatile("fence.proxy.async;" ::: "memory"); }
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t f16x2(float a, float b) {  // a in the low half
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}
__device__ __forceinline__ uint16_t e4m3x2(uint32_t h) {  // two fp16 -> two codes, the low half in the low byte
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(h));
  return r;
}
__device__ __forceinline__ uint32_t codes_f16x2(uint16_t c) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(c));
  return r;
}
__device__ __forceinline__ uint16_t e5m2x2(uint32_t h) {
  uint16_t r;
  asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;" : "=h"(r) : "r"(h));
  return r;
}
// F * (h - c) of two fp16 pairs, F 1, 16 or 32: exact where c is h rounded to fewer bits
template <int F>
__device__ __forceinline__ uint32_t rest(uint32_t h, uint32_t c) {
  static_assert(F == 1 || F == 16 || F == 32, "factor");
  uint32_t d, r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(h), "r"(c));
  if (F == 1) return d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(d), "r"(F == 16 ? 0x4C004C00u : 0x50005000u));
  return r;
}
__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, int c0, int c1, int c2, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::
          "r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void cp_async4(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}

// Shared-memory matrix descriptor (version 1) as its two halves: start and leading byte offset; stride
// byte offset and swizzle (0 none, 2 128 bytes, 4 64 bytes).  Adding bytes / 16 to the low half moves the start.
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr, uint32_t lbo) { return (addr & 0x3FFFFu) >> 4 | (lbo >> 4) << 16; }
constexpr uint32_t desc_hi(uint32_t sbo, uint32_t swizzle) { return sbo >> 4 | 1u << 14 | swizzle << 29; }
// kind::f8f6f4, E4M3 (A also E5M2) x E4M3 -> fp32, M = 128; ta, tb: A, B lie M- or N-contiguous.
__host__ __device__ constexpr uint32_t idesc_e4m3(int n, int ta, int tb, bool a_e5m2 = false) {
  return (1u << 4) | ((uint32_t)a_e5m2 << 7) | ((uint32_t)ta << 15) | ((uint32_t)tb << 16) | ((uint32_t)(n >> 3) << 17) | (8u << 24);
}
template <uint32_t AHI, uint32_t BHI, uint32_t IDESC>
__device__ __forceinline__ void mma_e4m3(uint32_t d, uint32_t alo, uint32_t blo, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\tsetp.ne.b32 p, %6, 0;\n\tmov.b64 da, {%1, %2};\n\tmov.b64 db, {%3, %4};\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], da, db, %5, p;\n\t}" ::"r"(d), "r"(alo), "n"(AHI), "r"(blo), "n"(BHI),
      "n"(IDESC), "r"(acc)
      : "memory");
}
// One lane of the warp, chosen so that the compiler knows the branch on it takes one thread.
__device__ __forceinline__ bool elect() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}
// Barrier of a softmax group's four warps that returns whether any thread's v is set.
__device__ __forceinline__ bool any_of(int group, bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %2, 0;\n\tbarrier.cta.red.or.pred q, %1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(1 + group), "r"((uint32_t)v)
      : "memory");
  return r != 0;
}
// One arrival for a warp, behind all its lanes' work: arrivals of 32 lanes are worked off one after the other.
__device__ __forceinline__ void warp_arrive(uint64_t* bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}
// Two fp32 operations an instruction, each rounded as the single one is.
__device__ __forceinline__ uint64_t pack2(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float* x, float* y) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(*x), "=f"(*y) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float warp_max(float v) {
  float r;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float rcp(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float lg2(float x) {
  float r;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// 16 elements of a query row (bf16 pairs) times the power of two `down`, as an E4M3 term and one for what is left of
// them, 8 units of a bf16's last place at most and so 3 significant bits with a sign: E5M2 (WIDE), or E4M3 scaled up by
// 2^5.  Exact for elements that `down` brings to 2^-6 or more, 2^-13 of the row's largest (which it brings to 2^7 at
// least); smaller ones, of which the first term has steps of 2^-9, are off by 2^-14 at most (E4M3: 2^-15), 2^-21 of
// the largest.
template <bool WIDE>
__device__ __forceinline__ void split_query(const uint4 (&x)[2], float down, uint4* hi, uint4* lo) {
  const uint32_t v[8] = {x[0].x, x[0].y, x[0].z, x[0].w, x[1].x, x[1].y, x[1].z, x[1].w};
  const uint32_t d = __byte_perm(__float_as_uint(down), 0, 0x3232);
  uint32_t h[4] = {0, 0, 0, 0}, l[4] = {0, 0, 0, 0};
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    uint32_t y;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(v[e]), "r"(d));
    const uint32_t f = f16x2(__uint_as_float(y << 16), __uint_as_float(y & 0xFFFF0000u));  // 11 bits hold a bf16's 8
    const uint16_t c = e4m3x2(f);
    h[e / 2] |= (uint32_t)c << (16 * (e & 1));
    const uint32_t left = codes_f16x2(c);
    l[e / 2] |= (uint32_t)(WIDE ? e5m2x2(rest<1>(f, left)) : e4m3x2(rest<32>(f, left))) << (16 * (e & 1));
  }
  *hi = make_uint4(h[0], h[1], h[2], h[3]);
  *lo = make_uint4(l[0], l[1], l[2], l[3]);
}
// The largest magnitude of 16 bf16 elements; NaN does not count.
__device__ __forceinline__ float query_max(const uint4 (&x)[2]) {
  const uint32_t v[8] = {x[0].x, x[0].y, x[0].z, x[0].w, x[1].x, x[1].y, x[1].z, x[1].w};
  uint32_t m = v[0] & 0x7FFF7FFFu;
#pragma unroll
  for (int e = 1; e < 8; ++e) asm("max.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(v[e] & 0x7FFF7FFFu));
  return fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xFFFF0000u));
}
// What brings a query row's largest element, amax < 2^(e2 + 8), to [128, 256).  An infinity makes every score of its row
// NaN (it meets a 0, or infinities of both signs, or none but equal ones), so the whole row becomes NaN here.
__device__ __forceinline__ float query_down(float amax, int e2) {
  return amax == INFINITY ? __int_as_float(0x7FFFFFFF) : __int_as_float((127 - e2) << 23);
}

// A NaN value code enters the output product of all rows, even times a weight of 0.  Where every row sees the key that is
// right; the codes of keys that only some rows see (behind the first row's position, before the last row's
// window) are looked at, a NaN becomes 0, and rows that do see it get their NaN in the end, from the cache.
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) {  // bit 7 of each byte that is 0x7F or 0xFF
  return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
}
__device__ __forceinline__ uint4 drop_nans(uint4 w, bool* found) {
  const uint32_t n[4] = {nan_bytes(w.x), nan_bytes(w.y), nan_bytes(w.z), nan_bytes(w.w)};
  if (n[0] | n[1] | n[2] | n[3]) *found = true;
  return make_uint4(w.x & ~((n[0] >> 7) * 255u), w.y & ~((n[1] >> 7) * 255u), w.z & ~((n[2] >> 7) * 255u),
                    w.w & ~((n[3] >> 7) * 255u));
}
// Bits of the 16 dims from d on (a multiple of 16) that are NaN in some key that the row at `pos` sees and not all rows do: all
// see the keys all0 .. all1.
static __device__ __noinline__ uint32_t nan_dims(const KvArgs& c, const int32_t* pages, int head, int head_dim, int d, int pos,
                                                 int window, int all0, int all1) {
  uint32_t bits = 0;
#pragma unroll 1
  for (int64_t t = max(pos - window + 1, 0); t <= pos; ++t) {
    if (t >= all0 && t <= all1) {
      t = all1;
      continue;
    }
    const int id = pages[t >> c.page_log2];
    if (id < 0 || id >= c.n_pages) continue;
    const int64_t tile = (int64_t)id * c.hkv + head, row = (tile << c.page_log2) + (t & ((1 << c.page_log2) - 1));
    if (c.ks[tile] == 0.0f) continue;
    const uint4 w = *reinterpret_cast<const uint4*>(c.v + row * head_dim + d);
    const uint32_t n[4] = {nan_bytes(w.x), nan_bytes(w.y), nan_bytes(w.z), nan_bytes(w.w)};
#pragma unroll
    for (int x = 0; x < 4; ++x)
      bits |= ((n[x] >> 7 & 1) | (n[x] >> 14 & 2) | (n[x] >> 21 & 4) | (n[x] >> 28 & 8)) << (4 * x);
  }
  return bits;
}
// Two codes of a word (its low or high half) -> two fp16 values.
__device__ __forceinline__ uint32_t codes_lo(uint32_t w) { return codes_f16x2((uint16_t)w); }
__device__ __forceinline__ uint32_t codes_hi(uint32_t w) { return codes_f16x2((uint16_t)(w >> 16)); }
__device__ __forceinline__ uint32_t bf16x2(float a, float b) {  // a in the low half
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}

}  // namespace qg
