// RMS norm with the residual's addition before it, its output in bf16 and / or in E4M3 codes
// with fp32 scales:
//   h = bf16(x + residual),  y = h / sqrt(mean(h^2) + eps) * (weight + weight_offset)
//   scale = max(amax / 448, 2^-100) of a group of y (or a row),  code = E4M3(y / scale)
//
// A row belongs to one CTA and a thread holds one or two vectors of eight of its elements in registers (a row of more than
// 16384: in shared memory), so that x and the residual are read once and the sum is written in the same pass.  CTAs stay
// for row after row, the next row's loads under way while one is summed and stored: what bounds many rows is HBM, and
// with codes the instructions (with one scale a row issue 73%), a few rows the chain load - sum - store.  The row's sum of squares
// (and, with one scale a row, its largest magnitude, of h * weight, as 1 / sqrt is not there yet) goes through warp
// shuffles and one shared-memory exchange whose slots alternate from row to row: one barrier a row, and every thread adds the warps'
// sums in the same order.  A group of 32, 64 or 128 elements lies in 4, 8 or 16 neighbouring lanes, so its scale needs shuffles only.
//
// Measured with residual, in a graph (share of the bytes at the copy rate, 6798 GB/s): one row of 5120 2.0 us, 64 to E4M3 in groups of
// 128 2.2; 4096 x 5120 27.5 us (90%), to E4M3 in groups 26.2 (82%), one scale a row 29.0 (74%); 18001 x 2048 48.2 (90%), 41.1 (92%) and
// 43.4 (87%); 2000 x 17408 48.1 (85%), 56.3 (64%) and 54.2 (66%).
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <atomic>

#include "qg_internal.h"
#include "qg_norm.h"
#include "qg_sync.cuh"

namespace qg {
namespace {

constexpr int kLongThreads = 768;  // for a row in shared memory: 2000 x 17408 to bf16 48 us (512 threads, three CTAs an SM: 50; 256: 52 to 58)
constexpr int kLongAhead = 2;      // and the vectors that a thread loads at a time (four: 52 us, fewer CTAs)
// of the longest row, rounded up to whole turns of the threads
constexpr size_t kLongBytes = (kNormMaxCols + 8 * kLongThreads - 1) / (8 * kLongThreads) * kLongThreads * 16;
constexpr float kMost = 448.0f;            // the largest code's value
constexpr float kLeast = kMost * 0x1p-100f;  // of a group's largest |y|: keeps 1 / scale finite for a group of zeros (448 * (1 / 448) is 1 in fp32)

struct Vec {
  uint32_t w[4];  // eight bf16
};

__device__ __forceinline__ float lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float hi(uint32_t u) { return __uint_as_float(u & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {  // a in the low half
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Eight elements from column c of a row of k elements; those past its end are 0 and are not read.  (A plain load: an output may lie on
// the row.)
__device__ __forceinline__ Vec load8(const uint16_t* row, int c, int k) {
  Vec v = {{0u, 0u, 0u, 0u}};
  if (c + 8 <= k) {
    const uint4 u = *reinterpret_cast<const uint4*>(row + c);
    v.w[0] = u.x, v.w[1] = u.y, v.w[2] = u.z, v.w[3] = u.w;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < k) v.w[i >> 1] |= (uint32_t)row[c + i] << (16 * (i & 1));
  }
  return v;
}
__device__ __forceinline__ void store8(uint16_t* row, int c, int k, const Vec& v) {
  if (c + 8 <= k) {
    *reinterpret_cast<uint4*>(row + c) = make_uint4(v.w[0], v.w[1], v.w[2], v.w[3]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < k) row[c + i] = (uint16_t)(v.w[i >> 1] >> (16 * (i & 1)));
  }
}

// Block-wide sum of one value a thread and, with MAX, the maximum of another (a magnitude), the same in every thread.  The
// slots hold a float per warp, 0 past the last warp; a caller that comes again alternates between two of them.
template <bool MAX>
__device__ __forceinline__ void block_reduce(float& v, float& m, float* sums, float* maxima) {
#pragma unroll
  for (int off = 16; off; off >>= 1) {
    v += __shfl_xor_sync(0xFFFFFFFFu, v, off);
    if (MAX) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, off));
  }
  const int warps = blockDim.x >> 5;
  if (warps == 1) return;
  if ((threadIdx.x & 31) == 0) {
    sums[threadIdx.x >> 5] = v;
    if (MAX) maxima[threadIdx.x >> 5] = m;
  }
  __syncthreads();
  v = m = 0.0f;
  for (int i = 0; i < warps; i += 4) {
    const float4 f = *reinterpret_cast<const float4*>(sums + i);
    v += (f.x + f.y) + (f.z + f.w);
    if (MAX) {
      const float4 g = *reinterpret_cast<const float4*>(maxima + i);
      m = fmaxf(fmaxf(m, g.x), fmaxf(g.y, fmaxf(g.z, g.w)));
    }
  }
}

// Eight elements as four pairs of fp32 (two bf16 of a word), and arithmetic on them: P, on a pair in one instruction, which
// pays where instructions are the bound, with one scale a row (18001 x 2048: 43.8 us, 45.1 without); the other forms lose
// by the pairs' registers (scales of groups of 128: 46 us, 41 without).
__device__ __forceinline__ float2 both(uint32_t u) { return make_float2(lo(u), hi(u)); }
__device__ __forceinline__ float2 twice(float a) { return make_float2(a, a); }
__device__ __forceinline__ uint64_t bits(float2 a) { return (uint64_t)__float_as_uint(a.y) << 32 | __float_as_uint(a.x); }
__device__ __forceinline__ float2 from_bits(uint64_t u) { return make_float2(__uint_as_float((uint32_t)u), __uint_as_float((uint32_t)(u >> 32))); }
template <bool P>
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  if (!P) return make_float2(a.x + b.x, a.y + b.y);
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(bits(a)), "l"(bits(b)));
  return from_bits(d);
}
template <bool P>
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  if (!P) return make_float2(a.x * b.x, a.y * b.y);
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(bits(a)), "l"(bits(b)));
  return from_bits(d);
}
// The squares of a, added to a sum in two parts, in one order in every form: y has the same bits whatever is stored beside it.
template <bool P>
__device__ __forceinline__ float2 add_squares(float2 a, float2 sum) {
  if (!P) return make_float2(fmaf(a.x, a.x, sum.x), fmaf(a.y, a.y, sum.y));
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %1, %2;" : "=l"(d) : "l"(bits(a)), "l"(bits(sum)));
  return from_bits(d);
}

// h (times f) times the weight.
template <bool P, bool BY>
__device__ __forceinline__ void scaled(const Vec& h, const Vec& w, float f, float woff, float2 (&v)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j)
    v[j] = mul2<P>(BY ? mul2<P>(both(h.w[j]), twice(f)) : both(h.w[j]), add2<P>(both(w.w[j]), twice(woff)));
}
// The largest magnitude of eight values, NaN and (finite) infinities left out.
__device__ __forceinline__ float largest(const float2 (&v)[4], bool finite) {
  float m = 0.0f;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    m = fmaxf(m, !finite || fabsf(v[j].x) < INFINITY ? fabsf(v[j].x) : 0.0f);
    m = fmaxf(m, !finite || fabsf(v[j].y) < INFINITY ? fabsf(v[j].y) : 0.0f);
  }
  return m;
}
// Eight E4M3 codes: nearest even, saturating at 448, NaN stays NaN.
template <bool P>
__device__ __forceinline__ void store_codes(const NormArgs& a, int64_t r, int c, int k, const float2 (&y)[4], float is) {
  uint32_t w[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const uint32_t p = __nv_cvt_float2_to_fp8x2(mul2<P>(y[2 * j], twice(is)), __NV_SATFINITE, __NV_E4M3);
    const uint32_t q = __nv_cvt_float2_to_fp8x2(mul2<P>(y[2 * j + 1], twice(is)), __NV_SATFINITE, __NV_E4M3);
    w[j] = p | q << 16;
  }
  uint8_t* row = a.codes + r * a.ldc;
  if (c + 8 <= k) {
    *reinterpret_cast<uint2*>(row + c) = make_uint2(w[0], w[1]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < k) row[c + i] = (uint8_t)(w[i >> 2] >> (8 * (i & 3)));
  }
}

// Of the values themselves, infinities left out; rare, so out of line.
__device__ __noinline__ float largest_value(Vec h, Vec w, float inv, float woff) {
  float2 v[4];
  scaled<false, true>(h, w, inv, woff, v);
  return largest(v, true);
}
// Whether the largest product of h and a weight, and the largest y that comes of it, are well inside fp32's range, and above the least.
__device__ __forceinline__ bool in_range(float amax, float ymax) { return amax >= 0x1p-100f && amax < INFINITY && ymax >= kLeast && ymax < INFINITY; }
// Over the `lanes` neighbouring lanes of a group.
__device__ __forceinline__ float group_max(float m, int lanes) {
  for (int off = lanes >> 1; off; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, off));
  return m;
}

// FP8: 0 bf16 only, 1 a scale a group, 2 a scale a row.  NV: vectors a thread; 0: the row lies in shared memory, as
// many a thread as it takes.
template <int NV, bool RES, int FP8>
__global__ void __launch_bounds__(NV ? 1024 : kLongThreads, NV ? 1 : 2) rms_norm_kernel(NormArgs a) {
  constexpr bool LONG = NV == 0;
  constexpr int kRegs = LONG ? kLongAhead : NV;
  __shared__ __align__(16) float slots[2][2][32];
  if (threadIdx.x < 128) (&slots[0][0][0])[threadIdx.x] = 0.0f;
  if (blockDim.x < 128)
    for (int i = threadIdx.x; i < 128; i += blockDim.x) (&slots[0][0][0])[i] = 0.0f;
  if (threadIdx.x == 0) pdl_launch_dependents();
  __syncthreads();
  pdl_wait();
  const int k = (int)a.k, T = blockDim.x, c0 = threadIdx.x * 8;
  constexpr bool P = FP8 == 2;
  constexpr bool kHold = !LONG && FP8 != 2;  // registers for the weights (one scale a row takes others)
  extern __shared__ __align__(16) Vec held[];  // LONG: a thread's own vectors
  const int n = LONG ? (int)((a.k + 8 * T - 1) / (8 * T)) : NV;
  Vec w[kHold ? kRegs : 1], x[kRegs], q[kRegs], h[LONG ? 1 : kRegs];
  auto load = [&](int64_t r, int i0) {
#pragma unroll
    for (int i = 0; i < kRegs; ++i) {
      x[i] = load8(a.x + r * a.ldx, c0 + (i0 + i) * T * 8, k);
      if (RES) q[i] = load8(a.res + r * a.ldr, c0 + (i0 + i) * T * 8, k);
    }
  };
  if (kHold) {
#pragma unroll
    for (int i = 0; i < kRegs; ++i) w[kHold ? i : 0] = load8(a.w, c0 + i * T * 8, k);
  }
  auto weight = [&](int i) { return kHold ? w[kHold ? i : 0] : load8(a.w, c0 + i * T * 8, k); };
  auto value = [&](int i) {
    if constexpr (LONG) return held[i * T + threadIdx.x];
    else return h[i];
  };
  if (!LONG) load(blockIdx.x, 0);
  int turn = 0;
  for (int64_t r = blockIdx.x; r < a.m; r += gridDim.x, turn ^= 1) {
    float2 sq2 = twice(0.0f);
    float amax = 0.0f;
    auto take = [&](int i, Vec& v) {  // vector i of the row, its residual added: stored, squared
      if (RES) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 f = add2<P>(both(x[i % kRegs].w[j]), both(q[i % kRegs].w[j]));
          v.w[j] = pack_bf16(f.x, f.y);
        }
      } else {
        v = x[i % kRegs];
      }
    };
    auto square = [&](int i, const Vec& v) {
      if (RES && a.sum) store8(a.sum + r * a.ldh, c0 + i * T * 8, k, v);
#pragma unroll
      for (int j = 0; j < 4; ++j) sq2 = add_squares<P>(both(v.w[j]), sq2);
    };
    if constexpr (LONG) {
      for (int i0 = 0; i0 < n; i0 += kRegs) {
        load(r, i0);
#pragma unroll
        for (int i = 0; i < kRegs; ++i) {
          if (i0 + i >= n) break;
          Vec v;
          take(i, v);
          held[(i0 + i) * T + threadIdx.x] = v;
          square(i0 + i, v);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < kRegs; ++i) take(i, h[i]);
      if (r + gridDim.x < a.m) load(r + gridDim.x, 0);  // while this row is summed and stored
#pragma unroll
      for (int i = 0; i < kRegs; ++i) square(i, h[i]);
    }
    float sq = sq2.x + sq2.y;
    if (FP8 == 2) {  // of h times the weight: 1 / sqrt is not there yet
#pragma unroll(LONG ? 2 : NV)
      for (int i = 0; i < n; ++i) {
        float2 v[4];
        scaled<P, false>(value(i), weight(i), 1.0f, a.woff, v);
        amax = fmaxf(amax, largest(v, false));
      }
    }
    block_reduce<FP8 == 2>(sq, amax, slots[0][turn], slots[1][turn]);
    const float inv = __frsqrt_rn(__fdiv_rn(sq, (float)k) + a.eps);
    // A code is that of h * weight * 448 / (the largest |h * weight|), in which 1 / sqrt cancels: two roundings, and the
    // same code whatever else the row holds.  Where the products h * weight pass fp32's range or come near its end, or the
    // scale is its least, h * inv * weight stands for them.
    float first = 1.0f, t = 0.0f;  // the value of a code is h * first * weight * t
    if (FP8 == 2) {
      float ymax = amax * inv;
      if (!in_range(amax, ymax)) {  // the same for the block
        first = inv, amax = kLeast;
#pragma unroll(LONG ? 1 : NV)
        for (int i = 0; i < n; ++i) amax = fmaxf(amax, largest_value(value(i), weight(i), inv, a.woff));
        float none = 0.0f;
        __syncthreads();
        block_reduce<true>(none, amax, slots[0][turn], slots[1][turn]);
        ymax = amax;
      }
      t = __fdiv_rn(kMost, amax);
      if (threadIdx.x == 0) a.scales[r * a.lds] = ymax * (1.0f / kMost);
    }
#pragma unroll(LONG ? 2 : NV)
    for (int i = 0; i < n; ++i) {
      const int c = c0 + i * T * 8;
      const Vec g = weight(i), f = value(i);
      float2 v[4];
      if (FP8 == 0 || a.y) {  // the same bits with codes and without
        scaled<P, true>(f, g, inv, a.woff, v);
        Vec o;
#pragma unroll
        for (int j = 0; j < 4; ++j) o.w[j] = pack_bf16(v[j].x, v[j].y);
        store8(a.y + r * a.ldy, c, k, o);
      }
      if (FP8 == 1) {
        // NaN does not enter a maximum.  What lies past the row's end is 0.
        scaled<P, false>(f, g, 1.0f, a.woff, v);
        amax = group_max(largest(v, false), a.group_lanes);
        float ymax = amax * inv;
        const bool far = !in_range(amax, ymax);  // the same for a group
        if (far) ymax = amax = kLeast;
        if (__any_sync(0xFFFFFFFFu, far && c < k)) {
          scaled<P, true>(f, g, far ? inv : 1.0f, a.woff, v);  // times 1: as before
          const float m = group_max(largest(v, true), a.group_lanes);
          if (far) ymax = amax = fmaxf(m, kLeast);
        }
        t = __fdiv_rn(kMost, amax);
        if ((threadIdx.x & (a.group_lanes - 1)) == 0 && c < k) a.scales[r * a.lds + (c >> a.group_log2)] = ymax * (1.0f / kMost);
      } else if (FP8 == 2) {
        scaled<P, true>(f, g, first, a.woff, v);
      }
      if (FP8) store_codes<P>(a, r, c, k, v, t);
    }
  }
}

template <int NV, bool RES, int FP8>
int launch(const NormArgs& a, const DeviceInfo& dev, int threads, cudaStream_t s) {
  // CTAs an SM by warps a CTA (NV 0: by vectors a thread), asked once; the GPUs that this is built for are alike
  static std::atomic<int> per_sm[33];
  static std::atomic<unsigned long long> allowed{0};
  const int vecs = NV ? 0 : (int)((a.k + 8 * threads - 1) / (8 * threads)), at = NV ? threads / 32 : vecs;
  const size_t smem = (size_t)vecs * threads * sizeof(Vec);
  if (NV == 0 && !allow_smem((const void*)rms_norm_kernel<NV, RES, FP8>, kLongBytes, allowed)) return QG_ERR_CUDA;
  int n = per_sm[at].load();
  if (n == 0) {
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, rms_norm_kernel<NV, RES, FP8>, threads, smem) != cudaSuccess || n < 1)
      return QG_ERR_CUDA;
    per_sm[at].store(n);
  }
  const int64_t resident = (int64_t)dev.sms * n;
  if (launch_pdl(rms_norm_kernel<NV, RES, FP8>, dim3((unsigned)std::min(a.m, resident)), dim3(threads), smem, s, a) != cudaSuccess)
    return QG_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? QG_OK : QG_ERR_CUDA;
}

template <int NV>
int launch_nv(const NormArgs& a, const DeviceInfo& dev, int threads, cudaStream_t s) {
  const int fp8 = !a.codes ? 0 : a.group_lanes ? 1 : 2;
  if (a.res)
    return fp8 == 0 ? launch<NV, true, 0>(a, dev, threads, s) : fp8 == 1 ? launch<NV, true, 1>(a, dev, threads, s)
                                                                         : launch<NV, true, 2>(a, dev, threads, s);
  return fp8 == 0 ? launch<NV, false, 0>(a, dev, threads, s) : fp8 == 1 ? launch<NV, false, 1>(a, dev, threads, s)
                                                                        : launch<NV, false, 2>(a, dev, threads, s);
}

}  // namespace

int launch_rms_norm(const NormArgs& a, const DeviceInfo& dev, void* stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int64_t vecs = (a.k + 7) / 8;
  // Two vectors a thread where rows queue up (4096 x 5120: 27 us, one vector 31, four 28); one where every row has a CTA of its
  // own (64 x 5120 to E4M3: 2.2 us, two vectors 3.4); by way of shared memory what 1024 threads do not hold so.
  const int nv = vecs <= 1024 && a.m <= dev.sms ? 1 : vecs <= 2048 ? 2 : 0;
  if (nv == 0) return launch_nv<0>(a, dev, kLongThreads, s);
  const int threads = (int)((vecs + nv - 1) / nv + 31) / 32 * 32;
  return nv == 1 ? launch_nv<1>(a, dev, threads, s) : launch_nv<2>(a, dev, threads, s);
}

}  // namespace qg
