// Low-rank adapters of many requests beside a shared projection:
//   out[i] = bf16(y[i] + scale_e * sum_j b_e[n][j] * h_j),  h_j = sum_k a_e[j][k] * x[i][k],  e = ids[i]
//
// One launch.  The rows of an adapter, wherever they lie, are taken T at a time (a tile); a
// cluster of CTAs works on a tile in two phases.  Phase 1: every CTA multiplies its share of
// the inputs (its warps split it further), the partial h are added in a fixed order, first
// in the CTA, then over the cluster through distributed shared memory, so that each CTA
// holds all of h.  Phase 2: every CTA multiplies its share of the outputs and adds y.  Both
// phases stream x, A, B, y and out once per tile; h never leaves the chip.
//
// Each CTA finds its tiles itself: it counts the rows of every adapter (ids are few bytes
// beside x and y), numbers the tiles adapter by adapter and collects its tile's rows in
// order.  So there is no plan to keep, nothing depends on the order of atomics, and rows of
// one adapter share its weights in whatever order the requests stand.
//
// Products are warp-level MMAs (m16n8k16, rows = tokens).  A lane loads 16 contiguous bytes
// of x and of A, eight inputs, and both operands take them as the fragment's k in the same
// order; which inputs make up a k16 step does not matter to the sum.  In phase 2 B's rows are
// dealt to the MMAs' columns so that a lane ends up with eight contiguous outputs of a row: y
// is read and written 16 bytes a lane.  h is split into two bf16 terms (16 bits of it), so the
// only rounding to 16 bits is the output's.
#include <algorithm>

#include "qg_lora_dev.cuh"

namespace qg {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;

// Eight elements of a row of k from column c, those past its end 0 and not read.
__device__ __forceinline__ uint4 load8(const uint16_t* row, int c, int k) {
  if (c + 8 <= k) return __ldg(reinterpret_cast<const uint4*>(row + c));
  uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (c + i < k) w[i >> 1] |= (uint32_t)row[c + i] << (16 * (i & 1));
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr));
  return v;
}

template <int R, int T>
struct Shape {
  static constexpr int kTiles = T / 16;                         // row tiles of 16
  static constexpr int kMt = T == 16 ? 1 : R <= 64 ? 2 : 1;     // of them in one warp, phase 1
  static constexpr int kKgroups = kWarps / (kTiles / kMt);      // warps that split the CTA's inputs
  static constexpr int kUnroll = R == 16 ? 4 : R == 32 ? 2 : 1;
  static constexpr int kPartRow = R + 4;                        // floats (16-byte rows)
  static constexpr int kHRow = R == 16 ? 48 : 2 * R + 32;       // bf16: fragments' rows in distinct banks
  static constexpr size_t kPartBytes = sizeof(float) * kKgroups * T * kPartRow;
  static constexpr size_t kHBytes = 2 * T * kHRow;
  static constexpr size_t kSmem = kPartBytes + kHBytes;
  static_assert((kTiles / kMt) * kKgroups == kWarps, "warps");
};

template <int R, int T>
__global__ void __launch_bounds__(kThreads) lora_kernel(LoraArgs p) {
  using S = Shape<R, T>;
  extern __shared__ __align__(16) uint8_t smem[];
  float* part = reinterpret_cast<float*>(smem);
  uint16_t* hs = reinterpret_cast<uint16_t*>(smem + S::kPartBytes);
  __shared__ Tiles<kThreads> tl;
  __shared__ int rows[T];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  uint32_t n_cta, rank;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(n_cta));
  rank = cluster_rank();
  const int cluster = blockIdx.x / n_cta, n_clusters = gridDim.x / n_cta;
  if (tid == 0) pdl_launch_dependents();
  pdl_wait();

  tl.count(p, T);
  const int n_tiles = tl.first[p.n_adapters + 1];
  for (int tile = cluster; tile < n_tiles; tile += n_clusters) {
    const int e = tl.collect(p, T, tile, rows), ra = rank_of(p, e);
    if (ra) {  // phase 1
      const uint16_t* ea = p.a + (int64_t)e * p.max_rank * p.lda;
      const int kg = warp % S::kKgroups, rg = warp / S::kKgroups;
      const int steps = (p.k + 31) / 32, groups = n_cta * S::kKgroups, me = rank * S::kKgroups + kg;
      const int s0 = (int)((int64_t)steps * me / groups), s1 = (int)((int64_t)steps * (me + 1) / groups);
      const uint16_t* xr[S::kMt][2];
#pragma unroll
      for (int i = 0; i < S::kMt; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int r = rows[(rg * S::kMt + i) * 16 + h * 8 + g];
          xr[i][h] = r < 0 ? nullptr : p.x + (int64_t)r * p.ldx;
        }
      float acc[S::kMt][R / 8][4] = {};
      for (int s = s0; s < s1; s += S::kUnroll) {
        uint4 xv[S::kUnroll][S::kMt][2], av[S::kUnroll][R / 8];
#pragma unroll
        for (int u = 0; u < S::kUnroll; ++u) {
          const int c = (s + u) * 32 + 8 * t;
          const int end = s + u < s1 ? p.k : 0;
#pragma unroll
          for (int j = 0; j < R / 8; ++j)
            av[u][j] = j * 8 + g < ra ? load8(ea + (int64_t)(j * 8 + g) * p.lda, c, end) : make_uint4(0, 0, 0, 0);
#pragma unroll
          for (int i = 0; i < S::kMt; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) xv[u][i][h] = xr[i][h] ? load8(xr[i][h], c, end) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int u = 0; u < S::kUnroll; ++u)
#pragma unroll
          for (int j = 0; j < R / 8; ++j)
#pragma unroll
            for (int i = 0; i < S::kMt; ++i) {
              mma16816(acc[i][j], xv[u][i][0].x, xv[u][i][1].x, xv[u][i][0].y, xv[u][i][1].y, av[u][j].x, av[u][j].y);
              mma16816(acc[i][j], xv[u][i][0].z, xv[u][i][1].z, xv[u][i][0].w, xv[u][i][1].w, av[u][j].z, av[u][j].w);
            }
      }
#pragma unroll
      for (int i = 0; i < S::kMt; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float* to = part + (kg * T + (rg * S::kMt + i) * 16 + h * 8 + g) * S::kPartRow + 2 * t;
#pragma unroll
          for (int j = 0; j < R / 8; ++j) *reinterpret_cast<float2*>(to + 8 * j) = make_float2(acc[i][j][2 * h], acc[i][j][2 * h + 1]);
        }
      __syncthreads();
      // the CTA's sum over its warps, then the cluster's over its CTAs, both in order
      for (int i = tid; i < T * R / 4; i += kThreads) {
        float* at = part + (i / (R / 4)) * S::kPartRow + (i % (R / 4)) * 4;
        float4 v = *reinterpret_cast<float4*>(at);
#pragma unroll
        for (int w = 1; w < S::kKgroups; ++w) {
          const float4 o = *reinterpret_cast<float4*>(at + w * T * S::kPartRow);
          v.x += o.x, v.y += o.y, v.z += o.z, v.w += o.w;
        }
        *reinterpret_cast<float4*>(at) = v;
      }
      if (n_cta > 1)
        cluster_sync_all();
      else
        __syncthreads();
      const float scale = p.scales[e];
      for (int i = tid; i < T * R / 8; i += kThreads) {
        const int row = i / (R / 8), col = (i % (R / 8)) * 8;
        const float* at = part + row * S::kPartRow + col;
        float v[8] = {};
        for (uint32_t c = 0; c < n_cta; ++c) {
          const uint32_t from = n_cta > 1 ? cluster_map(at, c) : 0;
          const float4 a0 = n_cta > 1 ? ld_cluster_f4(from) : *reinterpret_cast<const float4*>(at);
          const float4 a1 = n_cta > 1 ? ld_cluster_f4(from + 16) : *reinterpret_cast<const float4*>(at + 4);
          v[0] += a0.x, v[1] += a0.y, v[2] += a0.z, v[3] += a0.w;
          v[4] += a1.x, v[5] += a1.y, v[6] += a1.z, v[7] += a1.w;
        }
        uint4 top, rest;
        split_h(v, scale, ra - col, top, rest);
        *reinterpret_cast<uint4*>(hs + row * S::kHRow + col) = top;
        *reinterpret_cast<uint4*>(hs + row * S::kHRow + R + col) = rest;
      }
      __syncthreads();
    }

    {  // phase 2
      const uint16_t* eb = p.b + (int64_t)(e < p.n_adapters ? e : 0) * p.n * p.max_rank;
      const int chunks = (p.n + 31) / 32;
      const int c0 = (int)((int64_t)chunks * rank / n_cta), c1 = (int)((int64_t)chunks * (rank + 1) / n_cta);
      constexpr int kSteps = R == 16 ? 1 : R / 32;
      for (int ch = c0 + warp; ch < c1; ch += kWarps) {
        const int nb = ch * 32, col = nb + 8 * t;
        uint4 bv[kSteps][4];
#pragma unroll
        for (int q = 0; q < kSteps; ++q)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int nr = nb + 8 * (g >> 1) + 2 * j + (g & 1);
            const uint16_t* from = eb + (int64_t)nr * p.max_rank;
            bv[q][j] = make_uint4(0, 0, 0, 0);
            if (R == 16) {  // four ranks a lane
              const int c = 4 * t;
              if (nr < p.n && c < ra) {
                const uint2 v = __ldg(reinterpret_cast<const uint2*>(from + c));
                bv[q][j] = make_uint4(v.x, v.y, 0, 0);
                if (c + 4 > ra) bv[q][j] = keep_first(bv[q][j], ra - c);
              }
            } else {
              const int c = q * 32 + 8 * t;
              if (nr < p.n && c < ra) {
                bv[q][j] = __ldg(reinterpret_cast<const uint4*>(from + c));
                if (c + 8 > ra) bv[q][j] = keep_first(bv[q][j], ra - c);
              }
            }
          }
#pragma unroll
        for (int i = 0; i < S::kTiles; ++i) {
          float acc[4][4] = {};
          if (ra) {
            const uint16_t* h0 = hs + (i * 16 + g) * S::kHRow;
            const uint16_t* h1 = h0 + 8 * S::kHRow;
#pragma unroll
            for (int q = 0; q < kSteps; ++q)
#pragma unroll
              for (int term = 0; term < 2; ++term) {
                if (R == 16) {
                  const uint2 u = *reinterpret_cast<const uint2*>(h0 + term * R + 4 * t);
                  const uint2 v = *reinterpret_cast<const uint2*>(h1 + term * R + 4 * t);
#pragma unroll
                  for (int j = 0; j < 4; ++j) mma16816(acc[j], u.x, v.x, u.y, v.y, bv[q][j].x, bv[q][j].y);
                } else {
                  const uint4 u = *reinterpret_cast<const uint4*>(h0 + term * R + q * 32 + 8 * t);
                  const uint4 v = *reinterpret_cast<const uint4*>(h1 + term * R + q * 32 + 8 * t);
#pragma unroll
                  for (int j = 0; j < 4; ++j) {
                    mma16816(acc[j], u.x, v.x, u.y, v.y, bv[q][j].x, bv[q][j].y);
                    mma16816(acc[j], u.z, v.z, u.w, v.w, bv[q][j].z, bv[q][j].w);
                  }
                }
              }
          }
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int r = rows[i * 16 + h * 8 + g];
            if (r < 0 || col >= p.n) continue;
            const uint16_t* from = p.y + (int64_t)r * p.ldy + col;
            uint16_t* to = p.out + (int64_t)r * p.ldo + col;
            if (col + 8 <= p.n) {
              const uint4 v = *reinterpret_cast<const uint4*>(from);
              uint32_t w[4] = {v.x, v.y, v.z, v.w};
              if (ra)
#pragma unroll
                for (int j = 0; j < 4; ++j) w[j] = pack_bf16(bf_lo(w[j]) + acc[j][2 * h], bf_hi(w[j]) + acc[j][2 * h + 1]);
              *reinterpret_cast<uint4*>(to) = make_uint4(w[0], w[1], w[2], w[3]);
            } else {
#pragma unroll
              for (int c = 0; c < 8; ++c)
                if (col + c < p.n)
                  to[c] = ra ? (uint16_t)pack_bf16(bf_lo(from[c]) + acc[c >> 1][2 * h + (c & 1)], 0.0f) : from[c];
            }
          }
        }
      }
    }
    // no CTA writes its partial sums or rows again before every CTA has read them
    if (n_cta > 1)
      cluster_sync_all();
    else
      __syncthreads();
  }
}

template <int R, int T>
int launch(const LoraArgs& p, const DeviceInfo& dev, cudaStream_t s) {
  using S = Shape<R, T>;
  static std::atomic<unsigned long long> configured{0};
  if (!allow_smem((const void*)lora_kernel<R, T>, S::kSmem, configured)) return QG_ERR_CUDA;
  // about as many tiles as there are: full ones, or one for each adapter
  const int adapters = std::min(p.n_adapters + 1, p.m);
  const int full = (p.m + T - 1) / T, likely = std::max(full, std::min(p.n_adapters, p.m)), most = std::min(p.m, full + adapters);
  const int slots = 2 * dev.sms;
  int c = 8;
  while (c > 1 && likely * c > slots) c /= 2;
  const int clusters = std::max(1, std::min(most, slots / c));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(clusters * c);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = S::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = c;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  if (cudaLaunchKernelEx(&cfg, lora_kernel<R, T>, p) != cudaSuccess) return QG_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? QG_OK : QG_ERR_CUDA;
}

template <int T>
int launch_rank(const LoraArgs& p, const DeviceInfo& dev, cudaStream_t s) {
  if (p.max_rank <= 16) return launch<16, T>(p, dev, s);
  if (p.max_rank <= 32) return launch<32, T>(p, dev, s);
  if (p.max_rank <= 64) return launch<64, T>(p, dev, s);
  return launch<128, T>(p, dev, s);
}

}  // namespace

int launch_lora(const LoraArgs& p, const DeviceInfo& dev, void* stream) {
  return launch_rank<16>(p, dev, static_cast<cudaStream_t>(stream));
}

}  // namespace qg
