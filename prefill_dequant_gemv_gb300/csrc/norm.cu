// RMS norm with the residual's addition before it, its output in bf16 and / or in E4M3 codes
// with fp32 scales:
//   h = bf16(x + residual),  y = h / sqrt(mean(h^2) + eps) * (weight + weight_offset)
//   scale = max(amax / 448, 2^-100) of a group of y (or a row),  code = E4M3(y * (1 / scale))
//
// A row belongs to one CTA and a thread holds NV vectors of eight of its elements in
// registers, so that x and the residual are read once and the sum is written in the same
// pass.  The row's sum of squares (and, with one scale a row, its largest magnitude) goes
// through warp shuffles and one shared-memory exchange whose slots alternate from row to
// row: one barrier a row and reduction, and every thread adds the warps' sums in the same
// order.  A group of 32, 64 or 128 elements lies in 4, 8 or 16 neighbouring lanes, so its
// scale needs shuffles only.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "qg_internal.h"
#include "qg_norm.h"
#include "qg_sync.cuh"

namespace qg {
namespace {

constexpr float kScaleMin = 0x1p-100f;  // keeps 1 / scale finite for a group of zeros

struct Vec {
  uint32_t w[4];  // eight bf16
};

__device__ __forceinline__ float lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float hi(uint32_t u) { return __uint_as_float(u & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {  // a in the low half
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Eight elements from column c of a row of k elements; those past its end are 0 and are not read.
__device__ __forceinline__ Vec load8(const uint16_t* row, int c, int k) {
  Vec v = {{0u, 0u, 0u, 0u}};
  if (c + 8 <= k) {
    const uint4 u = __ldg(reinterpret_cast<const uint4*>(row + c));
    v.w[0] = u.x, v.w[1] = u.y, v.w[2] = u.z, v.w[3] = u.w;
  } else {
    for (int i = 0; c + i < k; ++i) v.w[i >> 1] |= (uint32_t)row[c + i] << (16 * (i & 1));
  }
  return v;
}
__device__ __forceinline__ void store8(uint16_t* row, int c, int k, const Vec& v) {
  if (c + 8 <= k) {
    *reinterpret_cast<uint4*>(row + c) = make_uint4(v.w[0], v.w[1], v.w[2], v.w[3]);
  } else {
    for (int i = 0; c + i < k; ++i) row[c + i] = (uint16_t)(v.w[i >> 1] >> (16 * (i & 1)));
  }
}

// Block-wide sum or maximum of one value a thread, the same in every thread.  `slots` holds
// a float per warp; a caller that comes again alternates between two of them.
template <bool MAX>
__device__ __forceinline__ float block_reduce(float v, float* slots) {
#pragma unroll
  for (int off = 16; off; off >>= 1) {
    const float o = __shfl_xor_sync(0xFFFFFFFFu, v, off);
    v = MAX ? fmaxf(v, o) : v + o;
  }
  const int warps = blockDim.x >> 5;
  if (warps == 1) return v;
  if ((threadIdx.x & 31) == 0) slots[threadIdx.x >> 5] = v;
  __syncthreads();
  v = slots[0];
  for (int i = 1; i < warps; ++i) v = MAX ? fmaxf(v, slots[i]) : v + slots[i];
  return v;
}

// Eight E4M3 codes: nearest even, saturating at 448, NaN stays NaN.
__device__ __forceinline__ void store_codes(const NormArgs& a, int64_t r, int c, int k, const float (&y)[8], float is) {
  uint32_t w[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const uint32_t p = __nv_cvt_float2_to_fp8x2(make_float2(y[4 * j] * is, y[4 * j + 1] * is), __NV_SATFINITE, __NV_E4M3);
    const uint32_t q = __nv_cvt_float2_to_fp8x2(make_float2(y[4 * j + 2] * is, y[4 * j + 3] * is), __NV_SATFINITE, __NV_E4M3);
    w[j] = p | q << 16;
  }
  uint8_t* row = a.codes + r * a.ldc;
  if (c + 8 <= k) {
    *reinterpret_cast<uint2*>(row + c) = make_uint2(w[0], w[1]);
  } else {
    for (int i = 0; c + i < k; ++i) row[c + i] = (uint8_t)(w[i >> 2] >> (8 * (i & 3)));
  }
}

template <int NV, bool RES, int FP8>  // FP8: 0 bf16 only, 1 a scale a group, 2 a scale a row
__global__ void __launch_bounds__(1024) rms_norm_kernel(NormArgs a) {
  __shared__ float slots[2][2][32];
  if (threadIdx.x == 0) pdl_launch_dependents();
  pdl_wait();
  const int k = (int)a.k, T = blockDim.x;
  int turn = 0;
  for (int64_t r = blockIdx.x; r < a.m; r += gridDim.x, turn ^= 1) {
    Vec h[NV];
    float sq = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (threadIdx.x + i * T) * 8;
      h[i] = load8(a.x + r * a.ldx, c, k);
      if (RES) {
        const Vec q = load8(a.res + r * a.ldr, c, k);
#pragma unroll
        for (int j = 0; j < 4; ++j) h[i].w[j] = pack_bf16(lo(h[i].w[j]) + lo(q.w[j]), hi(h[i].w[j]) + hi(q.w[j]));
        if (a.sum) store8(a.sum + r * a.ldh, c, k, h[i]);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        sq = fmaf(lo(h[i].w[j]), lo(h[i].w[j]), sq);
        sq = fmaf(hi(h[i].w[j]), hi(h[i].w[j]), sq);
      }
    }
    sq = block_reduce<false>(sq, slots[0][turn]);
    const float inv = rsqrtf(sq * a.inv_k + a.eps);
    float y[NV][8];
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (threadIdx.x + i * T) * 8;
      const Vec w = load8(a.w, c, k);
      if (FP8 == 1) amax = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float f = j & 1 ? hi(h[i].w[j >> 1]) : lo(h[i].w[j >> 1]);
        const float g = (j & 1 ? hi(w.w[j >> 1]) : lo(w.w[j >> 1])) + a.woff;
        y[i][j] = f * inv * g;
        if (FP8) amax = fmaxf(amax, c + j < k && fabsf(y[i][j]) < INFINITY ? fabsf(y[i][j]) : 0.0f);
      }
      if (FP8 == 0 || a.y) {
        Vec o;
#pragma unroll
        for (int j = 0; j < 4; ++j) o.w[j] = pack_bf16(y[i][2 * j], y[i][2 * j + 1]);
        store8(a.y + r * a.ldy, c, k, o);
      }
      if (FP8 == 1) {
        for (int off = a.group_lanes >> 1; off; off >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, off));
        const float s = fmaxf(__fdiv_rn(amax, 448.0f), kScaleMin);
        if ((threadIdx.x & (a.group_lanes - 1)) == 0 && c < k) a.scales[r * a.lds + c / (a.group_lanes * 8)] = s;
        store_codes(a, r, c, k, y[i], __frcp_rn(s));
      }
    }
    if (FP8 == 2) {
      amax = block_reduce<true>(amax, slots[1][turn]);
      const float s = fmaxf(__fdiv_rn(amax, 448.0f), kScaleMin);
      if (threadIdx.x == 0) a.scales[r * a.lds] = s;
      const float is = __frcp_rn(s);
#pragma unroll
      for (int i = 0; i < NV; ++i) store_codes(a, r, (threadIdx.x + i * T) * 8, k, y[i], is);
    }
  }
}

template <int NV, bool RES, int FP8>
int launch(const NormArgs& a, const DeviceInfo& dev, int threads, cudaStream_t s) {
  const int64_t resident = (int64_t)dev.sms * std::max(1, 2048 / threads);
  if (launch_pdl(rms_norm_kernel<NV, RES, FP8>, dim3((unsigned)std::min(a.m, resident)), dim3(threads), 0, s, a) != cudaSuccess)
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
  const int nv = vecs <= 1024 ? 1 : vecs <= 2048 ? 2 : vecs <= 4096 ? 4 : 8;
  const int threads = (int)((vecs + nv - 1) / nv + 31) / 32 * 32;
  return nv == 1 ? launch_nv<1>(a, dev, threads, s) : nv == 2 ? launch_nv<2>(a, dev, threads, s)
         : nv == 4 ? launch_nv<4>(a, dev, threads, s) : launch_nv<8>(a, dev, threads, s);
}

}  // namespace qg
