// Low-rank adapters for many rows, in two launches:
//   shrink: h[i] = a_e x[i] of every row, in fp32 parts;   expand: out[i] = bf16(y[i] + scale_e b_e h[i])
//
// Both stream their long operand once (x; y and out) and are bound by HBM; A, B and h
// come from L2.  Rows of one adapter are taken 64 at a time (a tile).  The tiles' inputs (shrink)
// or outputs (expand), cut into chunks, form one line of units that the CTAs
// share evenly whatever the sizes: a CTA's range may begin and end inside a tile.  In
// shrink that leaves a tile's h in parts, one for every CTA on it; CTA c's part of tile t is
// number c + t (each step along the line raises one of the two), and expand adds a tile's
// parts in that order, so results do not depend on timing.
//
// Every lane copies the 16-byte pieces that it will multiply itself, into slots of shared memory of its
// own, some chunks ahead (cp.async): rows may lie anywhere, nothing waits for another warp,
// what lies past a row's end comes as zeros, and the loads in flight take no registers.
//
// The products are warp-level MMAs (m16n8k16): 1024 multiply-adds a clock and SM, measured.  A tile of 64 rows
// and rank 64 takes some 75% of that rate when HBM is saturated, h's two bf16 terms included, and the
// fragments' layout is what lets a lane hold eight contiguous outputs of a row (see lora.cu).
#include <algorithm>

#include "qg_lora_dev.cuh"

namespace qg {
namespace {

constexpr int T = 64;           // rows of a tile
constexpr int kBatch = 16;      // tiles whose rows a CTA lists at a time

// 16 bytes global -> shared, those past the first `bytes` (0: none is read) as zeros.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
// The same by way of L1, for what another warp of the CTA reads as well.
__device__ __forceinline__ void copy16_l1(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ int bytes_of(int left) { return 2 * max(0, min(8, left)); }

// The line of units: CTA c's range, and the CTA of a unit.  Never more CTAs than units.
__device__ __forceinline__ int64_t line_begin(int64_t units, int ctas, int c) { return units * c / ctas; }
__device__ __forceinline__ int line_owner(int64_t units, int ctas, int64_t u) { return (int)(((u + 1) * ctas - 1) / units); }

// The tiles of a batch: rows (past the last the first again: what is computed of them is not stored), how many,
// adapter and rank.
template <int THREADS>
struct Batch {
  int rows[kBatch][T];
  int live[kBatch], bins[kBatch], ranks[kBatch];
  __device__ __forceinline__ void fill(const LoraArgs& p, Tiles<THREADS>& tl, int t0, int nt) {
    for (int i = 0; i < nt; ++i) {
      const int e = tl.collect(p, T, t0 + i, rows[i]);
      const int r = threadIdx.x < T ? rows[i][threadIdx.x] : 0;
      const int n = __syncthreads_count(threadIdx.x < T && r >= 0);
      if (r < 0) rows[i][threadIdx.x] = rows[i][0];
      if (threadIdx.x == 0) {
        live[i] = n;
        bins[i] = e;
        ranks[i] = rank_of(p, e);
      }
    }
    __syncthreads();
  }
};

// ------------------------------------------------------------------ shrink
template <int R>
struct Shrink {
  static constexpr int kThreads = R <= 32 ? 512 : 256, kWarps = kThreads / 32;
  static constexpr int kSplit = 2;                        // groups of warps that share a tile's rows
  static constexpr int kParts = kWarps / kSplit;          // warps that share a chunk's inputs, 32 each
  static constexpr int kMt = T / 16 / kSplit;             // row tiles of 16 a warp
  static constexpr int kWidth = 32 * kParts;              // inputs of a chunk
  static constexpr int kPieces = 2 * kMt + R / 8;         // of 16 bytes a lane and chunk
  static constexpr int kAhead = R <= 64 ? 3 : 2;          // chunks in flight: slots of a lane
  static constexpr int kSumRow = R + 4;                   // floats
  static constexpr size_t kRing = (size_t)kWarps * kAhead * kPieces * 512;
  static constexpr size_t kSmem = kRing + T * kSumRow * 4;
};

template <int R>
__global__ void __launch_bounds__(Shrink<R>::kThreads) lora_shrink_kernel(LoraArgs p, float* parts) {
  using S = Shrink<R>;
  extern __shared__ __align__(128) uint8_t smem[];
  float* sum = reinterpret_cast<float*>(smem + S::kRing);
  __shared__ Tiles<S::kThreads> tl;
  __shared__ Batch<S::kThreads> b;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  pdl_wait();
  if (tid == 0) pdl_launch_dependents();  // after the wait: what this call reads is there for expand as well
  tl.count(p, T);
  const int chunks = (p.k + S::kWidth - 1) / S::kWidth, n_tiles = tl.first[p.n_adapters];
  const int64_t units = (int64_t)n_tiles * chunks;
  const int ctas = (int)min((int64_t)gridDim.x, units), c = blockIdx.x;
  if (c >= ctas) return;
  const int64_t u0 = line_begin(units, ctas, c), u1 = line_begin(units, ctas, c + 1);
  const int t_first = (int)(u0 / chunks), t_last = (int)((u1 - 1) / chunks);
  const int half = warp % S::kSplit, part = warp / S::kSplit, row0 = half * (T / S::kSplit) + g;
  uint8_t* mine = smem + (size_t)warp * S::kAhead * S::kPieces * 512 + lane * 16;
  const uint32_t mine_at = smem_u32(mine);
  constexpr uint32_t kSlot = S::kPieces * 512, kSlots = S::kAhead * kSlot;

  for (int t0 = t_first; t0 <= t_last; t0 += kBatch) {
    const int nt = min(kBatch, t_last + 1 - t0);
    b.fill(p, tl, t0, nt);
    const int64_t b0 = max(u0, (int64_t)t0 * chunks);
    const int n = (int)(min(u1, (int64_t)(t0 + nt) * chunks) - b0);
    // the copies' state: tile, input and pointers of the next chunk
    int fi = (int)(b0 / chunks) - t0, col = (int)(b0 % chunks) * S::kWidth + part * 32 + 8 * t, ra_f = 0;
    uint32_t slot_f = 0;
    const uint16_t *xp[2 * S::kMt], *ap;
    auto aim = [&]() {
      ra_f = b.ranks[fi];
#pragma unroll
      for (int i = 0; i < 2 * S::kMt; ++i) xp[i] = p.x + (int64_t)b.rows[fi][row0 + 8 * i] * p.ldx + col;
      ap = p.a + ((int64_t)(ra_f ? b.bins[fi] : 0) * p.max_rank + (g < p.max_rank ? g : 0)) * p.lda + col;
    };
    aim();
    auto fetch = [&](int j) {
      if (j < n) {
        const int left = bytes_of(p.k - col);
        const uint32_t to = mine_at + slot_f;
        slot_f = slot_f + kSlot == kSlots ? 0 : slot_f + kSlot;
        if (left && ra_f) {
#pragma unroll
          for (int i = 0; i < 2 * S::kMt; ++i) copy16(to + i * 512, xp[i], left);
#pragma unroll
          for (int i = 0; i < R / 8; ++i)
            if (i * 8 < ra_f) {
              const bool in = i * 8 + g < ra_f;
              copy16_l1(to + (2 * S::kMt + i) * 512, in ? ap + (int64_t)(i * 8) * p.lda : p.a, in ? left : 0);
            }
        } else {  // past the row's end: zeros
#pragma unroll
          for (int i = 0; i < S::kPieces; ++i) copy16(to + i * 512, p.x, 0);
        }
        col += S::kWidth;
        if (col - 8 * t >= chunks * S::kWidth) {
          col = part * 32 + 8 * t;
          if (++fi < nt) aim();
        } else {
#pragma unroll
          for (int i = 0; i < 2 * S::kMt; ++i) xp[i] += S::kWidth;
          ap += S::kWidth;
        }
      }
      copy_commit();
    };
#pragma unroll
    for (int j = 0; j < S::kAhead; ++j) fetch(j);
    int i = (int)(b0 / chunks) - t0, ch = (int)(b0 % chunks), ra = b.ranks[i];
    uint32_t slot = 0;
    float acc[S::kMt][R / 8][4] = {};
    for (int j = 0; j < n; ++j) {
      copy_wait<S::kAhead - 1>();
      const uint8_t* from = mine + slot;
      slot = slot + kSlot == kSlots ? 0 : slot + kSlot;
      uint4 xv[S::kMt][2];
#pragma unroll
      for (int m = 0; m < S::kMt; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) xv[m][h] = *reinterpret_cast<const uint4*>(from + (2 * m + h) * 512);
#pragma unroll
      for (int q = 0; q < R / 8; ++q)
        if (q * 8 < ra) {
          const uint4 av = *reinterpret_cast<const uint4*>(from + (2 * S::kMt + q) * 512);
#pragma unroll
          for (int m = 0; m < S::kMt; ++m) {
            mma16816(acc[m][q], xv[m][0].x, xv[m][1].x, xv[m][0].y, xv[m][1].y, av.x, av.y);
            mma16816(acc[m][q], xv[m][0].z, xv[m][1].z, xv[m][0].w, xv[m][1].w, av.z, av.w);
          }
        }
      fetch(j + S::kAhead);  // into the slot whose pieces the products have taken
      if (++ch < chunks && j + 1 < n) continue;
      // the tile's end, or the CTA's: the warps' sums over their inputs, one after the other
      if (ra) {
        float* at = sum + row0 * S::kSumRow + 2 * t;
#pragma unroll 1
        for (int w = 0; w < S::kParts; ++w) {
          if (part == w) {
#pragma unroll
            for (int m = 0; m < S::kMt; ++m)
#pragma unroll
              for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int q = 0; q < R / 8; ++q) {
                  float2* to = reinterpret_cast<float2*>(at + (m * 16 + h * 8) * S::kSumRow + q * 8);
                  float2 v = make_float2(acc[m][q][2 * h], acc[m][q][2 * h + 1]);
                  if (w) v.x += to->x, v.y += to->y;
                  *to = v;
                }
          }
          __syncthreads();
        }
        float* to = parts + (int64_t)(c + t0 + i) * T * R;
        for (int x = tid; x < T * R / 4; x += S::kThreads)
          reinterpret_cast<float4*>(to)[x] = *reinterpret_cast<const float4*>(sum + x / (R / 4) * S::kSumRow + x % (R / 4) * 4);
        __syncthreads();
      }
#pragma unroll
      for (int m = 0; m < S::kMt; ++m)
#pragma unroll
        for (int q = 0; q < R / 8; ++q)
#pragma unroll
          for (int x = 0; x < 4; ++x) acc[m][q][x] = 0.0f;
      ch = 0;
      if (++i < nt) ra = b.ranks[i];
    }
    copy_wait<0>();
    __syncthreads();  // the lists are written again
  }
}

// ------------------------------------------------------------------ expand
template <int R>
struct Expand {
  static constexpr int kThreads = 512, kWarps = kThreads / 32;
  static constexpr int kSplit = 2;                // groups of warps that share a tile's rows
  static constexpr int kWidth = 32 * kWarps / kSplit;  // outputs of a chunk
  static constexpr int kMt = T / 16 / kSplit;
  static constexpr int kAhead = 3;
  static constexpr int kHRow = R == 16 ? 48 : 2 * R + 32;  // bf16: a fragment's pieces in distinct banks
  static constexpr size_t kRing = (size_t)kWarps * kAhead * 2 * kMt * 512;
  static constexpr size_t kSmem = kRing + 2 * T * kHRow;
  static constexpr int kHalf = R <= 64 ? R : 64;  // ranks of B in registers at a time
  static constexpr int kSteps = kHalf == 16 ? 1 : kHalf / 32;
};

// B's fragments of 32 outputs, kHalf ranks from r0, of an adapter of rank ra: bp is the lane's place in the row of its first
// output, whose others lie two outputs apart; `outs` of them exist.
template <int R>
__device__ __forceinline__ void load_b(const uint16_t* bp, int max_rank, int ra, int outs, int r0, int t,
                                       uint4 (&bv)[Expand<R>::kSteps][4]) {
  constexpr int kLane = R == 16 ? 4 : 8;  // ranks a lane
#pragma unroll
  for (int q = 0; q < Expand<R>::kSteps; ++q) {
    const int c = r0 + q * 32 + kLane * t;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      bv[q][j] = make_uint4(0, 0, 0, 0);
      if (c < ra && 2 * j < outs) {
        const uint16_t* from = bp + 2 * j * max_rank + r0 + q * 32;
        if (R == 16) {
          const uint2 v = __ldg(reinterpret_cast<const uint2*>(from));
          bv[q][j] = make_uint4(v.x, v.y, 0, 0);
        } else {
          bv[q][j] = __ldg(reinterpret_cast<const uint4*>(from));
        }
      }
    }
    if (ra & (kLane - 1)) {  // the rank ends inside a piece
#pragma unroll
      for (int j = 0; j < 4; ++j) bv[q][j] = keep_first(bv[q][j], ra - c);
    }
  }
}

template <int R>
__global__ void __launch_bounds__(Expand<R>::kThreads) lora_expand_kernel(LoraArgs p, const float* parts, int shrink_ctas,
                                                                          int shrink_width) {
  using S = Expand<R>;
  extern __shared__ __align__(128) uint8_t smem[];
  uint16_t* hs = reinterpret_cast<uint16_t*>(smem + S::kRing);
  __shared__ Tiles<S::kThreads> tl;
  __shared__ Batch<S::kThreads> b;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  if (tid == 0) pdl_launch_dependents();
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
  const int half = warp % S::kSplit, group = warp / S::kSplit, row0 = half * (T / S::kSplit) + g;
  uint8_t* mine = smem + (size_t)warp * S::kAhead * 2 * S::kMt * 512 + lane * 16;
  const uint32_t mine_at = smem_u32(mine);
  constexpr uint32_t kSlot = 2 * S::kMt * 512, kSlots = S::kAhead * kSlot;
  const bool in_place = p.out == p.y;

  for (int t0 = t_first; t0 <= t_last; t0 += kBatch) {
    const int nt = min(kBatch, t_last + 1 - t0);
    b.fill(p, tl, t0, nt);
    const int64_t b0 = max(u0, (int64_t)t0 * chunks);
    const int n = (int)(min(u1, (int64_t)(t0 + nt) * chunks) - b0);
    int i = (int)(b0 / chunks) - t0, ch = (int)(b0 % chunks);
    // the copies' state: tile, output and pointers of the next chunk
    int fi = i, fc = ch * S::kWidth + group * 32 + 8 * t;
    uint32_t slot_f = 0, slot = 0;
    const uint16_t* yp[2 * S::kMt];
    auto aim = [&]() {
#pragma unroll
      for (int m = 0; m < 2 * S::kMt; ++m) yp[m] = p.y + (int64_t)b.rows[fi][row0 + 8 * m] * p.ldy + fc;
    };
    aim();
    auto fetch = [&](int j) {
      if (j < n) {
        const int left = bytes_of(p.n - fc);
        const uint32_t to = mine_at + slot_f;
        slot_f = slot_f + kSlot == kSlots ? 0 : slot_f + kSlot;
        if (left) {
#pragma unroll
          for (int m = 0; m < 2 * S::kMt; ++m) copy16(to + m * 512, yp[m], left);
        }
        fc += S::kWidth;
        if (fc - 8 * t >= chunks * S::kWidth) {
          fc = group * 32 + 8 * t;
          if (++fi < nt) aim();
        } else {
#pragma unroll
          for (int m = 0; m < 2 * S::kMt; ++m) yp[m] += S::kWidth;
        }
      }
      copy_commit();
    };
#pragma unroll
    for (int j = 0; j < S::kAhead; ++j) fetch(j);
    if (t0 == t_first) pdl_wait();  // shrink has ended: its parts are there, and stores may begin
    bool fresh = true;  // a tile begins
    int ra = 0, live = 0, nb = 0;
    uint16_t* op[2 * S::kMt];
    const uint16_t* bp = p.b;
    const int bg = 8 * (g >> 1) + (g & 1);  // the lane's outputs in B: bg, bg + 2, bg + 4, bg + 6
    for (int j = 0; j < n; ++j) {
      if (fresh) {
        const int e = b.bins[i], tile = t0 + i;
        ra = b.ranks[i];
        live = b.live[i] - row0;  // row m of this lane exists if 8 m < live
        nb = ch * S::kWidth + group * 32;
#pragma unroll
        for (int m = 0; m < 2 * S::kMt; ++m) op[m] = p.out + (int64_t)b.rows[i][row0 + 8 * m] * p.ldo + nb + 8 * t;
        if (ra) {
          bp = p.b + ((int64_t)e * p.n + nb + bg) * p.max_rank + (R == 16 ? 4 : 8) * t;
          __syncthreads();  // every warp is done with the last tile's h
          const int p0 = line_owner(k_units, k_ctas, (int64_t)tile * k_chunks),
                    p1 = line_owner(k_units, k_ctas, (int64_t)(tile + 1) * k_chunks - 1);
          const float scale = p.scales[e];
          for (int x = tid; x < T * R / 4; x += S::kThreads) {
            const int row = x / (R / 4), at = (x % (R / 4)) * 4;
            const float* from = parts + ((int64_t)(p0 + tile) * T + row) * R + at;
            float4 v = __ldcg(reinterpret_cast<const float4*>(from));
            for (int q = p0 + 1; q <= p1; ++q) {
              const float4 o = __ldcg(reinterpret_cast<const float4*>(from + (int64_t)(q - p0) * T * R));
              v.x += o.x, v.y += o.y, v.z += o.z, v.w += o.w;
            }
            uint2 top, rest;
            split_h(v, scale, top, rest);
            *reinterpret_cast<uint2*>(hs + row * S::kHRow + at) = top;
            *reinterpret_cast<uint2*>(hs + row * S::kHRow + R + at) = rest;
          }
          __syncthreads();
        }
      }
      const bool last = ch + 1 == chunks;  // of the tile
      float acc[S::kMt][4][4] = {};
      if (ra && nb < p.n) {
#pragma unroll
        for (int r0 = 0; r0 < R; r0 += S::kHalf) {
          uint4 bv[S::kSteps][4];
          load_b<R>(bp, p.max_rank, ra, p.n - nb - bg, r0, t, bv);
#pragma unroll
          for (int m = 0; m < S::kMt; ++m) {
            const uint16_t* h0 = hs + (row0 + m * 16) * S::kHRow + r0;
            const uint16_t* h1 = h0 + 8 * S::kHRow;
#pragma unroll
            for (int q = 0; q < S::kSteps; ++q)
#pragma unroll
              for (int term = 0; term < 2; ++term) {
                if (R == 16) {
                  const uint2 u = *reinterpret_cast<const uint2*>(h0 + term * R + 4 * t);
                  const uint2 v = *reinterpret_cast<const uint2*>(h1 + term * R + 4 * t);
#pragma unroll
                  for (int x = 0; x < 4; ++x) mma16816(acc[m][x], u.x, v.x, u.y, v.y, bv[q][x].x, bv[q][x].y);
                } else {
                  const uint4 u = *reinterpret_cast<const uint4*>(h0 + term * R + q * 32 + 8 * t);
                  const uint4 v = *reinterpret_cast<const uint4*>(h1 + term * R + q * 32 + 8 * t);
#pragma unroll
                  for (int x = 0; x < 4; ++x) {
                    mma16816(acc[m][x], u.x, v.x, u.y, v.y, bv[q][x].x, bv[q][x].y);
                    mma16816(acc[m][x], u.z, v.z, u.w, v.w, bv[q][x].z, bv[q][x].w);
                  }
                }
              }
          }
        }
      }
      copy_wait<S::kAhead - 1>();
      const uint8_t* from = mine + slot;
      slot = slot + kSlot == kSlots ? 0 : slot + kSlot;
      const int left = p.n - nb - 8 * t;
#pragma unroll
      for (int m = 0; m < S::kMt; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (16 * m + 8 * h >= live || left <= 0 || (ra == 0 && in_place)) continue;
          const uint4 v = *reinterpret_cast<const uint4*>(from + (2 * m + h) * 512);
          uint32_t w[4] = {v.x, v.y, v.z, v.w};
          if (ra)
#pragma unroll
            for (int x = 0; x < 4; ++x)
              w[x] = pack_bf16(bf_lo(w[x]) + acc[m][x][2 * h], bf_hi(w[x]) + acc[m][x][2 * h + 1]);
          uint16_t* to = op[2 * m + h];
          if (left >= 8) {
            *reinterpret_cast<uint4*>(to) = make_uint4(w[0], w[1], w[2], w[3]);
          } else {
#pragma unroll
            for (int x = 0; x < 8; ++x)
              if (x < left) to[x] = (uint16_t)(w[x >> 1] >> (16 * (x & 1)));
          }
        }
#pragma unroll
      for (int m = 0; m < 2 * S::kMt; ++m) op[m] += S::kWidth;
      nb += S::kWidth;
      bp += S::kWidth * p.max_rank;
      fetch(j + S::kAhead);
      fresh = last;
      ++ch;
      if (last) ch = 0, ++i;
    }
    copy_wait<0>();
    __syncthreads();  // the lists are written again
  }
}

// CTAs an SM: as many as fit.
template <int R>
struct PerSm {
  static constexpr int kShrink = 1, kExpand = 1;
};

template <int R>
int launch(const LoraArgs& p, const DeviceInfo& dev, float* parts, cudaStream_t s) {
  static std::atomic<unsigned long long> a{0}, b{0};
  if (!allow_smem((const void*)lora_shrink_kernel<R>, Shrink<R>::kSmem, a) ||
      !allow_smem((const void*)lora_expand_kernel<R>, Expand<R>::kSmem, b))
    return QG_ERR_CUDA;
  const int shrink = dev.sms * PerSm<R>::kShrink, expand = dev.sms * PerSm<R>::kExpand;
  if (launch_pdl(lora_shrink_kernel<R>, dim3(shrink), dim3(Shrink<R>::kThreads), Shrink<R>::kSmem, s, p, parts) != cudaSuccess ||
      launch_pdl(lora_expand_kernel<R>, dim3(expand), dim3(Expand<R>::kThreads), Expand<R>::kSmem, s, p,
                 static_cast<const float*>(parts), shrink, Shrink<R>::kWidth) != cudaSuccess)
    return QG_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? QG_OK : QG_ERR_CUDA;
}

int padded_rank(int max_rank) { return max_rank <= 16 ? 16 : max_rank <= 32 ? 32 : max_rank <= 64 ? 64 : 128; }

}  // namespace

size_t lora_rows_bytes(int n_adapters, int max_rank, int64_t m, const DeviceInfo& dev) {
  const int64_t rows = std::min<int64_t>(m, kLoraRowsAtOnce);
  const int64_t tiles = (rows + T - 1) / T + std::min<int64_t>(rows, n_adapters);
  return (size_t)(tiles + 2 * dev.sms) * T * padded_rank(max_rank) * sizeof(float);
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
