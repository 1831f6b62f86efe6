// Low-rank adapters for many rows, in two launches:
//   shrink: h[i] = a_e x[i] of every row, in fp32 parts;   expand: out[i] = bf16(y[i] + scale_e b_e h[i])
//
// Both stream their long operand once (x; y and out) and are bound by HBM; A, B and h
// come from L2.  Rows of one adapter are taken 64 at a time (a tile).  The tiles' inputs (shrink)
// or outputs (expand), cut into chunks, form one line of units that the CTAs, one an SM,
// share evenly whatever the sizes: a CTA's range may begin and end inside a tile.  In
// shrink that leaves a tile's h in parts, one for every CTA on it; CTA c's part of tile t is
// number c + t (each step along the line raises one of the two), and expand adds a tile's
// parts in that order, so results do not depend on timing.
//
// Rows lie anywhere, so a chunk of a tile is one bulk copy per row (512 bytes of a row in expand), into a
// ring in shared memory that one warp keeps filled; in expand the sum is written over y in the
// ring and leaves by bulk copies too.  Row pitches of 64 bytes past a multiple of 128 put the
// eight 16-byte pieces of a fragment's quarter into distinct banks.
//
// The products are warp-level MMAs (m16n8k16): 1024 multiply-adds a clock and SM.  A tile of 64 rows and
// rank 64 takes some 60% of that rate when HBM is saturated, h's two bf16 terms included, and the fragments'
// layout is what lets a lane hold eight contiguous outputs of a row (see lora.cu).
#include <algorithm>

#include "qg_lora_dev.cuh"

namespace qg {
namespace {

// A bounded wait with one answer for the warp.
__device__ __forceinline__ bool wait_warp(uint64_t* bar, int pass, int* status) {
  return __all_sync(0xFFFFFFFFu, mbar_wait_bounded(bar, pass & 1, status));
}

constexpr int T = 64;           // rows of a tile
constexpr int kBatch = 16;      // tiles whose rows a CTA lists at a time

// 1-D bulk copy shared -> global.
__device__ __forceinline__ void bulk_s2g(void* dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(smem_u32(src)), "r"(bytes) : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void bulk_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// The line of units: CTA c's range, and the CTA of a unit.  Never more CTAs than units.
__device__ __forceinline__ int64_t line_begin(int64_t units, int ctas, int c) { return units * c / ctas; }
__device__ __forceinline__ int line_owner(int64_t units, int ctas, int64_t u) { return (int)(((u + 1) * ctas - 1) / units); }

// ------------------------------------------------------------------ shrink
template <int R>
struct Shrink {
  static constexpr int kWidth = R <= 32 ? 256 : 128;  // inputs of a chunk
  static constexpr int kPitch = 2 * kWidth + 64;      // bytes
  static constexpr int kStages = R == 16 || R == 64 ? 4 : 3;
  static constexpr int kStage = (T + R) * kPitch;
  static constexpr int kSumRow = R + 4;               // floats
  static constexpr size_t kSmem = (size_t)kStages * kStage + T * kSumRow * 4;
  static constexpr int kThreads = 288;                // eight warps of products, one of copies
};

template <int R>
__global__ void __launch_bounds__(288, 1) lora_shrink_kernel(LoraArgs p, float* parts) {
  using S = Shrink<R>;
  extern __shared__ __align__(128) uint8_t smem[];
  float* sum = reinterpret_cast<float*>(smem + S::kStages * S::kStage);
  __shared__ Tiles<S::kThreads> tl;
  __shared__ int rows[kBatch][T];
  __shared__ int bins[kBatch], ranks[kBatch];
  __shared__ uint64_t full[S::kStages], empty[S::kStages];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  if (tid == 0) {
    for (int i = 0; i < S::kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 8);
    }
    fence_mbar_init();
  }
  pdl_wait();
  if (tid == 0) pdl_launch_dependents();  // after the wait: what this call reads is there for expand as well
  tl.count(p, T);
  const int chunks = (p.k + S::kWidth - 1) / S::kWidth, n_tiles = tl.first[p.n_adapters];
  const int64_t units = (int64_t)n_tiles * chunks;
  const int ctas = (int)min((int64_t)gridDim.x, units), c = blockIdx.x;
  if (c >= ctas) return;
  const int64_t u0 = line_begin(units, ctas, c), u1 = line_begin(units, ctas, c + 1);
  const int t_first = (int)(u0 / chunks), t_last = (int)((u1 - 1) / chunks);

  int it = 0;  // chunks so far: ring slot it % kStages, pass it / kStages
  bool ok = true;
  for (int t0 = t_first; t0 <= t_last; t0 += kBatch) {
    const int nt = min(kBatch, t_last + 1 - t0);
    for (int i = 0; i < nt; ++i) {
      const int e = tl.collect(p, T, t0 + i, rows[i]);
      if (tid == 0) {
        bins[i] = e;
        ranks[i] = rank_of(p, e);
      }
    }
    __syncthreads();
    for (int i = 0; i < nt; ++i) {
      const int tile = t0 + i, ra = ranks[i];
      const int k0 = (int)(max(u0, (int64_t)tile * chunks) - (int64_t)tile * chunks);
      const int k1 = (int)(min(u1, (int64_t)(tile + 1) * chunks) - (int64_t)tile * chunks);
      if (ra == 0) continue;
      if (warp == 8) {  // copies
        const uint16_t* ea = p.a + (int64_t)bins[i] * p.max_rank * p.lda;
        const int ra0 = rows[i][lane], ra1 = rows[i][lane + 32];
        const int live = __popc(__ballot_sync(0xFFFFFFFFu, ra0 >= 0)) + __popc(__ballot_sync(0xFFFFFFFFu, ra1 >= 0));
        for (int ch = k0; ch < k1 && ok; ++ch, ++it) {
          const int s = it % S::kStages;
          if (it >= S::kStages) ok = wait_warp(&empty[s], it / S::kStages - 1, p.status);
          if (!ok) break;
          uint8_t* st = smem + s * S::kStage;
          const int col = ch * S::kWidth;
          const uint32_t bytes = (uint32_t)(min(S::kWidth, p.k - col) + 7) / 8 * 16;  // up to the 16 bytes that hold the last
          if (lane == 0) mbar_arrive_expect_tx(&full[s], bytes * (uint32_t)(live + ra));
          __syncwarp();
          if (ra0 >= 0) bulk_g2s(st + lane * S::kPitch, p.x + ra0 * p.ldx + col, bytes, &full[s]);
          if (ra1 >= 0) bulk_g2s(st + (lane + 32) * S::kPitch, p.x + ra1 * p.ldx + col, bytes, &full[s]);
          for (int j = lane; j < ra; j += 32) bulk_g2s(st + (T + j) * S::kPitch, ea + (int64_t)j * p.lda + col, bytes, &full[s]);
        }
      } else {  // products: two halves of the rows, four quarters of a chunk's inputs
        const int half = warp & 1, part = warp >> 1;
        float acc[2][R / 8][4] = {};
        for (int ch = k0; ch < k1 && ok; ++ch, ++it) {
          const int s = it % S::kStages;
          ok = wait_warp(&full[s], it / S::kStages, p.status);
          if (!ok) break;
          const uint8_t* st = smem + s * S::kStage;
          const int left = p.k - ch * S::kWidth;  // inputs from the chunk's start on
#pragma unroll
          for (int q = 0; q < S::kWidth / 128; ++q) {
            const int col = part * (S::kWidth / 4) + q * 32 + 8 * t;
            const int valid = left - col;
            uint4 xv[2][2];
#pragma unroll
            for (int i2 = 0; i2 < 2; ++i2)
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                xv[i2][h] = *reinterpret_cast<const uint4*>(st + (half * 32 + i2 * 16 + h * 8 + g) * S::kPitch + 2 * col);
                if (valid < 8) xv[i2][h] = keep_first(xv[i2][h], valid);
              }
#pragma unroll
            for (int j = 0; j < R / 8; ++j) {
              if (j * 8 >= ra) break;
              uint4 av = *reinterpret_cast<const uint4*>(st + (T + j * 8 + g) * S::kPitch + 2 * col);
              if (valid < 8 || j * 8 + g >= ra) av = keep_first(av, j * 8 + g < ra ? valid : 0);
#pragma unroll
              for (int i2 = 0; i2 < 2; ++i2) {
                mma16816(acc[i2][j], xv[i2][0].x, xv[i2][1].x, xv[i2][0].y, xv[i2][1].y, av.x, av.y);
                mma16816(acc[i2][j], xv[i2][0].z, xv[i2][1].z, xv[i2][0].w, xv[i2][1].w, av.z, av.w);
              }
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&empty[s]);
        }
        // the four quarters' sums, one after the other: 3 to 2, 2 to 1, 1 to 0
        float* mine = sum + (half * 32 + g) * S::kSumRow + 2 * t;
#pragma unroll
        for (int from = 3; from >= 1; --from) {
          if (part == from) {
#pragma unroll
            for (int i2 = 0; i2 < 2; ++i2)
#pragma unroll
              for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int j = 0; j < R / 8; ++j)
                  *reinterpret_cast<float2*>(mine + (i2 * 16 + h * 8) * S::kSumRow + j * 8) =
                      make_float2(acc[i2][j][2 * h], acc[i2][j][2 * h + 1]);
          }
          named_sync(1, 256);
          if (part == from - 1) {
#pragma unroll
            for (int i2 = 0; i2 < 2; ++i2)
#pragma unroll
              for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int j = 0; j < R / 8; ++j) {
                  const float2 v = *reinterpret_cast<float2*>(mine + (i2 * 16 + h * 8) * S::kSumRow + j * 8);
                  acc[i2][j][2 * h] += v.x;
                  acc[i2][j][2 * h + 1] += v.y;
                }
          }
          named_sync(1, 256);
        }
        if (part == 0) {
          float* to = parts + ((int64_t)(c + tile) * T + half * 32 + g) * R + 2 * t;
#pragma unroll
          for (int i2 = 0; i2 < 2; ++i2)
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int j = 0; j < R / 8; ++j)
                *reinterpret_cast<float2*>(to + (i2 * 16 + h * 8) * R + j * 8) = make_float2(acc[i2][j][2 * h], acc[i2][j][2 * h + 1]);
        }
      }
    }
    __syncthreads();  // the lists are written again
  }
  if (warp == 8)  // after a wait that gave up, copies may be in flight: not past the CTA's end
    for (int i = max(0, it - S::kStages); i < it; ++i) wait_warp(&full[i % S::kStages], i / S::kStages, p.status);
}

// ------------------------------------------------------------------ expand
template <int R>
struct Expand {
  static constexpr int kWidth = 256;              // outputs of a chunk
  static constexpr int kPitch = 2 * kWidth + 64;  // bytes
  static constexpr int kStages = 4;
  static constexpr int kAhead = 2;                // chunks between a load and its use
  static constexpr int kStage = T * kPitch;
  static constexpr int kHRow = R == 16 ? 48 : 2 * R + 32;  // bf16
  static constexpr size_t kSmem = (size_t)kStages * kStage + 2 * T * kHRow;
  static constexpr int kSplit = 1;                // groups of warps that share a tile's rows
  static constexpr int kWarps = 8 * kSplit;       // of products; one more of copies
  static constexpr int kThreads = 32 * kWarps + 32;
  static constexpr int kMt = T / 16 / kSplit;     // row tiles of 16 a warp
  static constexpr int kHalf = R <= 64 ? R : 64;  // ranks of B in registers at a time
  static constexpr int kSteps = kHalf == 16 ? 1 : kHalf / 32;
};

// B's fragments: 32 outputs from nb, kHalf ranks from r0, of an adapter of rank ra.
template <int R>
__device__ __forceinline__ void load_b(const LoraArgs& p, const uint16_t* eb, int ra, int nb, int r0, int g, int t,
                                       uint4 (&bv)[Expand<R>::kSteps][4]) {
#pragma unroll
  for (int q = 0; q < Expand<R>::kSteps; ++q)
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
        const int c = r0 + q * 32 + 8 * t;
        if (nr < p.n && c < ra) {
          bv[q][j] = __ldg(reinterpret_cast<const uint4*>(from + c));
          if (c + 8 > ra) bv[q][j] = keep_first(bv[q][j], ra - c);
        }
      }
    }
}

template <int R>
__global__ void __launch_bounds__(Expand<R>::kThreads, 1) lora_expand_kernel(LoraArgs p, const float* parts, int shrink_ctas, int shrink_width) {
  using S = Expand<R>;
  extern __shared__ __align__(128) uint8_t smem[];
  uint16_t* hs = reinterpret_cast<uint16_t*>(smem + S::kStages * S::kStage);
  __shared__ Tiles<S::kThreads> tl;
  __shared__ int rows[kBatch][T];
  __shared__ int bins[kBatch], ranks[kBatch];
  __shared__ uint64_t full[S::kStages], done[S::kStages];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  if (tid == 0) {
    for (int i = 0; i < S::kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&done[i], S::kWarps);
    }
    fence_mbar_init();
    pdl_launch_dependents();
  }
  tl.count(p, T);
  const int chunks = (p.n + S::kWidth - 1) / S::kWidth, n_tiles = tl.first[p.n_adapters + 1];
  const int64_t units = (int64_t)n_tiles * chunks;
  const int ctas = (int)min((int64_t)gridDim.x, units), c = blockIdx.x;
  if (c >= ctas) {
    pdl_wait();  // this grid's end stands for the one before it
    return;
  }
  const int64_t u0 = line_begin(units, ctas, c), u1 = line_begin(units, ctas, c + 1);
  const int t_first = (int)(u0 / chunks), t_last = (int)((u1 - 1) / chunks);
  const int k_chunks = (p.k + shrink_width - 1) / shrink_width;
  const int64_t k_units = (int64_t)tl.first[p.n_adapters] * k_chunks;
  const int k_ctas = (int)min((int64_t)shrink_ctas, k_units);

  int it = 0;
  bool ok = true, waited = false;
  for (int t0 = t_first; t0 <= t_last; t0 += kBatch) {
    const int nt = min(kBatch, t_last + 1 - t0);
    for (int i = 0; i < nt; ++i) {
      const int e = tl.collect(p, T, t0 + i, rows[i]);
      if (tid == 0) {
        bins[i] = e;
        ranks[i] = rank_of(p, e);
      }
    }
    __syncthreads();
    if (warp == S::kWarps) {  // copies: loads kAhead chunks before the stores
      const int64_t b0 = max(u0, (int64_t)t0 * chunks), b1 = min(u1, (int64_t)(t0 + nt) * chunks);
      const int n = (int)(b1 - b0);
      for (int j = 0; j < n + S::kAhead && ok; ++j) {
        if (j >= S::kAhead) {  // chunk j - kAhead leaves
          const int64_t u = b0 + j - S::kAhead;
          const int i = (int)(u / chunks) - t0, col = (int)(u % chunks) * S::kWidth, at = it + j - S::kAhead, s = at % S::kStages;
          ok = wait_warp(&done[s], at / S::kStages, p.status);
          if (!ok) break;
          const uint32_t bytes = (uint32_t)min(S::kWidth, p.n - col) / 8 * 16;  // whole vectors; the products' warps store the rest
          if (bytes && (ranks[i] || p.out != p.y))
            for (int r = lane; r < T; r += 32)
              if (rows[i][r] >= 0) bulk_s2g(p.out + rows[i][r] * p.ldo + col, smem + s * S::kStage + r * S::kPitch, bytes);
          bulk_commit();
        }
        if (j < n) {  // chunk j comes; the slot's last chunk, j - kStages, left kStages - kAhead stores ago
          const int64_t u = b0 + j;
          const int i = (int)(u / chunks) - t0, col = (int)(u % chunks) * S::kWidth, s = (it + j) % S::kStages;
          bulk_wait_read<S::kStages - S::kAhead>();
          __syncwarp();
          const uint32_t bytes = (uint32_t)(min(S::kWidth, p.n - col) + 7) / 8 * 16;
          const int r0 = rows[i][lane], r1 = rows[i][lane + 32];
          const int live = __popc(__ballot_sync(0xFFFFFFFFu, r0 >= 0)) + __popc(__ballot_sync(0xFFFFFFFFu, r1 >= 0));
          if (lane == 0) mbar_arrive_expect_tx(&full[s], bytes * live);
          __syncwarp();
          if (r0 >= 0) bulk_g2s(smem + s * S::kStage + lane * S::kPitch, p.y + r0 * p.ldy + col, bytes, &full[s]);
          if (r1 >= 0) bulk_g2s(smem + s * S::kStage + (lane + 32) * S::kPitch, p.y + r1 * p.ldy + col, bytes, &full[s]);
        }
      }
      it += n;
    } else {  // products: eight groups of 32 outputs
      const int group = warp & 7, half = warp >> 3;
      if (!waited) pdl_wait();  // shrink has ended: its parts are there
      waited = true;
      for (int i = 0; i < nt && ok; ++i) {
        const int tile = t0 + i, e = bins[i], ra = ranks[i];
        const int c0 = (int)(max(u0, (int64_t)tile * chunks) - (int64_t)tile * chunks);
        const int c1 = (int)(min(u1, (int64_t)(tile + 1) * chunks) - (int64_t)tile * chunks);
        const uint16_t* eb = p.b + (int64_t)(e < p.n_adapters ? e : 0) * p.n * p.max_rank;
        uint4 bv[S::kSteps][4];
        if (ra) {
          load_b<R>(p, eb, ra, c0 * S::kWidth + group * 32, 0, g, t, bv);
          named_sync(1, 32 * S::kWarps);  // every warp is done with the last tile's h
          const int p0 = line_owner(k_units, k_ctas, (int64_t)tile * k_chunks),
                    p1 = line_owner(k_units, k_ctas, (int64_t)(tile + 1) * k_chunks - 1);
          const float scale = p.scales[e];
          for (int x = tid; x < T * R / 4; x += 32 * S::kWarps) {
            const int row = x / (R / 4), col = (x % (R / 4)) * 4;
            const float* from = parts + ((int64_t)(p0 + tile) * T + row) * R + col;
            float4 v = __ldcg(reinterpret_cast<const float4*>(from));
            for (int q = p0 + 1; q <= p1; ++q) {
              const float4 o = __ldcg(reinterpret_cast<const float4*>(from + (int64_t)(q - p0) * T * R));
              v.x += o.x, v.y += o.y, v.z += o.z, v.w += o.w;
            }
            uint2 top, rest;
            split_h(v, scale, top, rest);
            *reinterpret_cast<uint2*>(hs + row * S::kHRow + col) = top;
            *reinterpret_cast<uint2*>(hs + row * S::kHRow + R + col) = rest;
          }
          named_sync(1, 32 * S::kWarps);
        }
        for (int ch = c0; ch < c1; ++ch, ++it) {
          const int s = it % S::kStages, nb = ch * S::kWidth + group * 32, col = nb + 8 * t;
          ok = wait_warp(&full[s], it / S::kStages, p.status);
          if (!ok) break;
          if (ra && nb < p.n) {
            float acc[S::kMt][4][4] = {};
#pragma unroll
            for (int r0 = 0; r0 < R; r0 += S::kHalf) {
              uint4 cur[S::kSteps][4];
#pragma unroll
              for (int q = 0; q < S::kSteps; ++q)
#pragma unroll
                for (int j = 0; j < 4; ++j) cur[q][j] = bv[q][j];
              if (r0 + S::kHalf < R)  // the next fragments come during this step's products
                load_b<R>(p, eb, ra, nb, r0 + S::kHalf, g, t, bv);
              else if (ch + 1 < c1)
                load_b<R>(p, eb, ra, nb + S::kWidth, 0, g, t, bv);
#pragma unroll
              for (int i2 = 0; i2 < S::kMt; ++i2) {
                const uint16_t* h0 = hs + (half * (T / S::kSplit) + i2 * 16 + g) * S::kHRow + r0;
                const uint16_t* h1 = h0 + 8 * S::kHRow;
#pragma unroll
                for (int q = 0; q < S::kSteps; ++q)
#pragma unroll
                  for (int term = 0; term < 2; ++term) {
                    if (R == 16) {
                      const uint2 u = *reinterpret_cast<const uint2*>(h0 + term * R + 4 * t);
                      const uint2 v = *reinterpret_cast<const uint2*>(h1 + term * R + 4 * t);
#pragma unroll
                      for (int j = 0; j < 4; ++j) mma16816(acc[i2][j], u.x, v.x, u.y, v.y, cur[q][j].x, cur[q][j].y);
                    } else {
                      const uint4 u = *reinterpret_cast<const uint4*>(h0 + term * R + q * 32 + 8 * t);
                      const uint4 v = *reinterpret_cast<const uint4*>(h1 + term * R + q * 32 + 8 * t);
#pragma unroll
                      for (int j = 0; j < 4; ++j) {
                        mma16816(acc[i2][j], u.x, v.x, u.y, v.y, cur[q][j].x, cur[q][j].y);
                        mma16816(acc[i2][j], u.z, v.z, u.w, v.w, cur[q][j].z, cur[q][j].w);
                      }
                    }
                  }
              }
            }
#pragma unroll
            for (int i2 = 0; i2 < S::kMt; ++i2)
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const int r = half * (T / S::kSplit) + i2 * 16 + h * 8 + g;
                uint4* at = reinterpret_cast<uint4*>(smem + s * S::kStage + r * S::kPitch + 2 * (group * 32 + 8 * t));
                const uint4 v = *at;
                uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int j = 0; j < 4; ++j)
                  w[j] = pack_bf16(bf_lo(w[j]) + acc[i2][j][2 * h], bf_hi(w[j]) + acc[i2][j][2 * h + 1]);
                *at = make_uint4(w[0], w[1], w[2], w[3]);
              }
          }
          if (col < p.n && col + 8 > p.n && (ra || p.out != p.y))  // the row's last outputs, fewer than a vector
            for (int r = g; r < T / S::kSplit; r += 8) {
              const int row = rows[i][half * (T / S::kSplit) + r];
              const uint16_t* from = reinterpret_cast<const uint16_t*>(smem + s * S::kStage + (half * (T / S::kSplit) + r) * S::kPitch) + group * 32 + 8 * t;
              if (row >= 0)
                for (int x = 0; col + x < p.n; ++x) p.out[row * p.ldo + col + x] = from[x];
            }
          fence_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&done[s]);
        }
      }
    }
    __syncthreads();
  }
  if (warp == S::kWarps) {
    for (int i = max(0, it - S::kStages); i < it; ++i) wait_warp(&full[i % S::kStages], i / S::kStages, p.status);
    bulk_wait_all();
  }
}

template <int R>
int launch(const LoraArgs& p, const DeviceInfo& dev, float* parts, cudaStream_t s) {
  static std::atomic<unsigned long long> a{0}, b{0};
  if (!allow_smem((const void*)lora_shrink_kernel<R>, Shrink<R>::kSmem, a) ||
      !allow_smem((const void*)lora_expand_kernel<R>, Expand<R>::kSmem, b))
    return QG_ERR_CUDA;
  if (launch_pdl(lora_shrink_kernel<R>, dim3(dev.sms), dim3(Shrink<R>::kThreads), Shrink<R>::kSmem, s, p, parts) != cudaSuccess ||
      launch_pdl(lora_expand_kernel<R>, dim3(dev.sms), dim3(Expand<R>::kThreads), Expand<R>::kSmem, s, p,
                 static_cast<const float*>(parts), dev.sms, Shrink<R>::kWidth) != cudaSuccess)
    return QG_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? QG_OK : QG_ERR_CUDA;
}

int padded_rank(int max_rank) { return max_rank <= 16 ? 16 : max_rank <= 32 ? 32 : max_rank <= 64 ? 64 : 128; }

}  // namespace

size_t lora_rows_bytes(int n_adapters, int max_rank, int64_t m, const DeviceInfo& dev) {
  const int64_t rows = std::min<int64_t>(m, kLoraRowsAtOnce);
  const int64_t tiles = (rows + T - 1) / T + std::min<int64_t>(rows, n_adapters);
  return (size_t)(tiles + dev.sms) * T * padded_rank(max_rank) * sizeof(float);
}

int launch_lora_rows(const LoraArgs& all, const DeviceInfo& dev, void* parts, void* stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  float* f = static_cast<float*>(parts);
  for (int64_t at = 0; at < all.m; at += kLoraRowsAtOnce) {
    LoraArgs p = all;
    p.m = (int)std::min<int64_t>(kLoraRowsAtOnce, all.m - at);
    p.ids += at;
    p.x += at * p.ldx;
    p.y += at * p.ldy;
    p.out += at * p.ldo;
    const int r = padded_rank(p.max_rank);
    const int st = r == 16 ? launch<16>(p, dev, f, s) : r == 32 ? launch<32>(p, dev, f, s)
                   : r == 64 ? launch<64>(p, dev, f, s) : launch<128>(p, dev, f, s);
    if (st != QG_OK) return st;
  }
  return QG_OK;
}

}  // namespace qg
