// Low-rank adapters of many requests beside a shared projection, few rows:
//   out[i] = bf16(y[i] + scale_e * sum_j b_e[n][j] * h_j),  h_j = sum_k a_e[j][k] * x[i][k],  e = ids[i]
//
// One launch.  The rows of an adapter, wherever they lie, are taken 16 at a time (a tile); a
// cluster of CTAs works on a tile in two phases.  Phase 1: every warp multiplies its share of
// the inputs, the partial h are added in a fixed order, first in the CTA, then over the cluster
// through distributed shared memory, so that each CTA holds all of h.  Phase 2: every warp
// multiplies its share of the outputs and adds y.  A and B are read once for a tile and are what
// the call is bound by, or the chain of its steps where they are small; so every lane copies the pieces
// that it will multiply itself into slots of shared memory of its own warp's (cp.async) as far ahead as there
// are slots, B and y while phase 1 and the sums of h are still under way.
//
// Each CTA finds its tiles itself, from the ids in its registers: there is no plan to keep, and
// rows of one adapter share its weights in whatever order the requests stand.
//
// Products are warp-level MMAs (m16n8k16, rows = tokens).  A lane copies 16 contiguous bytes
// of x and of A, eight inputs, and both operands take them as the fragment's k in the same
// order; which inputs make up a k16 step does not matter to the sum.  In phase 2 B's rows are
// dealt to the MMAs' columns so that a lane ends up with eight contiguous outputs of a row: y
// is read and written 16 bytes a lane.  h is split into two bf16 terms (16 bits of it), so the
// only rounding to 16 bits is the output's.
//
// Measured in a graph, 5120 inputs, 7168 outputs (us, rank 16 / 64; the bytes at the copy rate): one row 6.9 / 9.2 (0.5 / 1.9), 16 rows
// of 16 adapters - / 14 (- / 3.8), 64 of 48 15 / 22 (3.1 / 11.5), 256 of 48 16.5 / 23 (4.2 / 12.6).
#include <algorithm>
#include <cmath>

#include "qg_lora_dev.cuh"

namespace qg {
namespace {

constexpr int T = 16;  // rows of a tile
constexpr int kThreads = 256, kWarps = kThreads / 32;
static_assert(kThreads == kLoraFewRows, "a thread a row");

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr));
  return v;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

template <int R>
struct Shape {
  static constexpr int kHalves = R == 128 ? 2 : 1;              // warps that share the ranks of a step of phase 1
  static constexpr int kRanks = R / kHalves;                    // of a warp
  static constexpr int kLogGroups = R == 128 ? 2 : 3, kGroups = 1 << kLogGroups;  // warps that share the inputs
  static_assert(kGroups == kWarps / kHalves, "");
  static constexpr int kPieces = R / 8;                         // of 16 bytes in a row of B
  static constexpr int kSteps = R == 16 ? 1 : R / 32;           // of products over the ranks in phase 2
  // bytes a warp: 64 inputs of x's 16 rows and A's, or 64 outputs of y's rows and B's (rank 128: 32 outputs)
  static constexpr int kOuts = R == 128 ? 32 : 64;
  static constexpr int kSlot = 2048 + kRanks * 128;
  static constexpr int kAhead = R == 16 ? 6 : R == 32 ? 4 : 2;
  static constexpr int kPartRow = R + 4;                        // floats (16-byte rows)
  static constexpr int kHRow = R == 16 ? 48 : 2 * R + 32;       // bf16: fragments' rows in distinct banks
  static constexpr size_t kRing = (size_t)kWarps * kAhead * kSlot;
  static constexpr size_t kPartBytes = sizeof(float) * kGroups * T * kPartRow;
  static constexpr size_t kSmem = kRing + kPartBytes + 2 * T * kHRow;
};

// Place of piece `c` (16 bytes) of row r in a block of rows of PIECES pieces each: what a fragment's quarter of a warp reads
// together lies in distinct banks.
template <int PIECES>
__device__ __forceinline__ uint32_t piece_at(int r, int c) {
  if (PIECES == 2) return (32 * r + 16 * c) ^ ((r >> 3 & 1) << 6);
  if (PIECES == 4) return 64 * r + 16 * c;
  return 16 * PIECES * r + ((16 * c) ^ ((r & 1) << 6));
}

template <int R>
__global__ void __launch_bounds__(kThreads) lora_kernel(LoraArgs p) {
  using S = Shape<R>;
  extern __shared__ __align__(128) uint8_t smem[];
  float* part = reinterpret_cast<float*>(smem + S::kRing);
  uint16_t* hs = reinterpret_cast<uint16_t*>(smem + S::kRing + S::kPartBytes);
  __shared__ __align__(16) int ids[kThreads];
  __shared__ int warp_sums[kWarps], rows[T], found[2];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  uint32_t n_cta;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(n_cta));
  const int log_n = __ffs(n_cta) - 1, cluster = blockIdx.x >> log_n, n_clusters = gridDim.x >> log_n;  // a power of two
  uint8_t* mine = smem + (size_t)warp * S::kAhead * S::kSlot;
  const uint32_t mine_at = smem_u32(mine);
  const bool in_place = p.out == p.y;
  if (tid == 0) pdl_launch_dependents();
  pdl_wait();

  // Thread i has row i.  Its place among the rows of its adapter says whether it is the first of a tile; tiles are
  // numbered by their first rows.
  int id = -2;
  if (tid < p.m) {
    const int raw = p.ids[tid];
    if (raw < -1 || raw >= p.n_adapters) atomicCAS(p.status, 0, kStatusInvalid);
    id = (unsigned)raw < (unsigned)p.n_adapters ? raw : -1;
  }
  ids[tid] = id;
  __syncthreads();
  int place = 0;
  if (tid < p.m)
    for (int j = 0; j < tid; j += 4) {
      const int4 o = *reinterpret_cast<const int4*>(ids + j);
      place += (o.x == id) + (j + 1 < tid && o.y == id) + (j + 2 < tid && o.z == id) + (j + 3 < tid && o.w == id);
    }
  const bool first = tid < p.m && place % T == 0;
  int n_tiles;
  const int number = block_prefix<kThreads>(first, warp_sums, &n_tiles);

  // A cluster's CTAs work on one tile, or where there are more tiles than clusters in teams of half of them or fewer, each on
  // its own tile.  The teams of a cluster keep step (its barrier is the whole cluster's).
  int log_team = log_n;
  while (log_team > 0 && n_tiles > n_clusters << (log_n - log_team)) --log_team;
  const int team = 1 << log_team, rank = (int)cluster_rank() & (team - 1), lead = (int)cluster_rank() - rank;
  const int teams = n_clusters << (log_n - log_team);
  for (int at = 0; at < n_tiles; at += teams) {
    const int tile = at + (cluster << (log_n - log_team)) + (lead >> log_team);
    if (first && number == tile) found[0] = id, found[1] = place;
    if (tid == 0 && tile >= n_tiles) found[0] = -2, found[1] = 0;  // no tile
    if (tid < T) rows[tid] = -1;
    __syncthreads();
    const int e = found[0], place0 = found[1];
    if (e == -2) {
      if (team > 1) {
        cluster_arrive();
        cluster_wait();
        cluster_arrive();
        cluster_wait();
      }
      __syncthreads();
      continue;
    }
    if (id == e && place >= place0 && place < place0 + T) rows[place - place0] = tid;
    const int ra = e < 0 ? 0 : rank_of(p, e);
    __syncthreads();
    // phase 1 in steps of 64 inputs, phase 2 in chunks of kOuts outputs: this warp's
    const int half = warp % S::kHalves, group = warp / S::kHalves, rank0 = half * S::kRanks;
    const int steps = ra ? (p.k + 63) / 64 : 0, me = rank * S::kGroups + group, all = log_team + S::kLogGroups;
    const int s0 = steps * me >> all, n1 = (steps * (me + 1) >> all) - s0;
    const int chunks = (p.n + S::kOuts - 1) / S::kOuts;
    const int c0 = chunks * rank >> log_team, c1 = chunks * (rank + 1) >> log_team;
    // in place there is nothing to do without an adapter (such tiles count all the same: the teams are those of a call that is not)
    const int n2 = c0 + warp < c1 && !(ra == 0 && in_place) ? (c1 - c0 - warp + kWarps - 1) / kWarps : 0, n = n1 + n2;
    // The copies' state.  A lane copies piece lane % 8 of every fourth row of x, A and y, so that a copy takes whole lines; and
    // of B, whose rows are shorter or longer, every 32nd piece.  A pointer may run past its row's end, or stand on a row that is
    // not there: then no byte of it is read.
    const int64_t ee = e < 0 ? 0 : e;
    const int lr = lane >> 3, lc = lane & 7;
    constexpr int kBRows = 32 / S::kPieces > 0 ? 32 / S::kPieces : 1;  // rows of B in one copy
    const int br = lane / S::kPieces, bc = lane % S::kPieces;
    constexpr int kYLanes = S::kOuts / 8;                                // pieces of a row of y
    const int yr = lane / kYLanes, yc = lane % kYLanes;
    int left1 = p.k - s0 * 64 - 8 * lc, out1 = (c0 + warp) * S::kOuts;
    const uint16_t* ap = p.a + (ee * p.max_rank + rank0 + lr) * p.lda + s0 * 64 + 8 * lc;
    const uint16_t* xp[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) xp[i] = p.x + (int64_t)max(rows[lr + 4 * i], 0) * p.ldx + s0 * 64 + 8 * lc;
    const uint16_t* bp = p.b + (ee * p.n + out1 + br) * p.max_rank + 8 * bc;
    uint32_t to = mine_at;
    const uint32_t ring_end = mine_at + S::kAhead * S::kSlot;
    auto fetch1 = [&]() {
      const int bytes = bytes_of(left1);
#pragma unroll
      for (int i = 0; i < S::kRanks / 4; ++i)
        if ((4 * i & ~7) + rank0 < ra)
          copy16(to + 2048 + piece_at<8>(lr + 4 * i, lc), ap + (int64_t)(4 * i) * p.lda, rank0 + lr + 4 * i < ra ? bytes : 0);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if ((4 * i & ~7) == 0 || rows[8] >= 0)  // rows 8 to 15 only where there are any
          copy16(to + piece_at<8>(lr + 4 * i, lc), xp[i], rows[lr + 4 * i] >= 0 ? bytes : 0);
        xp[i] += 64;
      }
      ap += 64;
      left1 -= 64;
    };
    auto fetch2 = [&]() {
      const int ranks = 2 * max(0, min(8, ra - 8 * bc));  // bytes: ranks past the adapter's as zeros
      if (8 * bc < ((ra + 31) & ~31)) {  // (rank 16: always) what a step of products reads
#pragma unroll
        for (int i = 0; i < S::kOuts / kBRows; ++i)
          copy16(to + 2048 + piece_at<S::kPieces>(br + i * kBRows, bc), bp + (int64_t)(i * kBRows) * p.max_rank,
                 out1 + br + i * kBRows < p.n ? ranks : 0);
      }
      const int bytes = bytes_of(p.n - out1 - 8 * yc);
#pragma unroll
      for (int i = 0; i < T * kYLanes / 32; ++i) {
        const int r = rows[yr + i * (32 / kYLanes)];
        if (r >= 0 && bytes)
          copy16(to + piece_at<kYLanes>(yr + i * (32 / kYLanes), yc), p.y + (int64_t)r * p.ldy + out1 + 8 * yc, bytes);
      }
      bp += (int64_t)(S::kOuts * kWarps) * p.max_rank;
      out1 += S::kOuts * kWarps;
    };
    auto fetch = [&](int j) {
      __syncwarp();  // every lane is done with the slot
      if (j < n1)
        fetch1();
      else if (j < n)
        fetch2();
      copy_commit();
      to = to + S::kSlot == ring_end ? mine_at : to + S::kSlot;
    };
    const uint8_t* from = mine;
    auto arrived = [&]() {  // the oldest slot's pieces, every lane's
      copy_wait<S::kAhead - 1>();
      __syncwarp();
    };
    auto next = [&]() { from = from + S::kSlot == mine + S::kAhead * S::kSlot ? mine : from + S::kSlot; };
#pragma unroll 1
    for (int j = 0; j < S::kAhead; ++j) fetch(j);

    if (ra) {
      float acc[S::kRanks / 8][4] = {};
#pragma unroll 1
      for (int j = 0; j < n1; ++j) {
        arrived();
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const uint4 u = *reinterpret_cast<const uint4*>(from + piece_at<8>(g, 4 * q + t));
          uint4 v = make_uint4(0, 0, 0, 0);
          if (rows[8] >= 0) v = *reinterpret_cast<const uint4*>(from + piece_at<8>(g + 8, 4 * q + t));
#pragma unroll
          for (int i = 0; i < S::kRanks / 8; ++i)
            if (rank0 + i * 8 < ra) {
              const uint4 w = *reinterpret_cast<const uint4*>(from + 2048 + piece_at<8>(8 * i + g, 4 * q + t));
              mma16816(acc[i], u.x, v.x, u.y, v.y, w.x, w.y);
              mma16816(acc[i], u.z, v.z, u.w, v.w, w.z, w.w);
            }
        }
        fetch(j + S::kAhead);
        next();
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float* to_part = part + (group * T + h * 8 + g) * S::kPartRow + rank0 + 2 * t;
#pragma unroll
        for (int i = 0; i < S::kRanks / 8; ++i) *reinterpret_cast<float2*>(to_part + 8 * i) = make_float2(acc[i][2 * h], acc[i][2 * h + 1]);
      }
      __syncthreads();
      // the CTA's sum over its warps, then the team's over its CTAs, both in order; of the rows that there are
      const int live = __popc(__ballot_sync(0xFFFFFFFFu, rows[lane & 15] >= 0) & 0xFFFFu);
      for (int i = tid; i < live * R / 4; i += kThreads) {
        float* at = part + (i / (R / 4)) * S::kPartRow + (i % (R / 4)) * 4;
        float4 v = *reinterpret_cast<float4*>(at);
#pragma unroll
        for (int w = 1; w < S::kGroups; ++w) {
          const float4 o = *reinterpret_cast<float4*>(at + w * T * S::kPartRow);
          v.x += o.x, v.y += o.y, v.z += o.z, v.w += o.w;
        }
        *reinterpret_cast<float4*>(at) = v;
      }
      if (team > 1) {
        cluster_arrive();
        cluster_wait();
      } else {
        __syncthreads();
      }
      const float scale = p.scales[e];
      for (int i = tid; i < T * R / 8; i += kThreads) {
        const int r = i / (R / 8), col = (i % (R / 8)) * 8;
        uint4 top = make_uint4(0, 0, 0, 0), rest = top;
        if (r < live) {
          const float* at = part + r * S::kPartRow + col;
          float4 o[8][2];
#pragma unroll
          for (int c = 0; c < 8; ++c)  // a team has up to eight CTAs
            if (c < team) {
              const uint32_t there = cluster_map(at, (uint32_t)(lead + c));
              o[c][0] = ld_cluster_f4(there);
              o[c][1] = ld_cluster_f4(there + 16);
            }
          float v[8] = {};
#pragma unroll
          for (int c = 0; c < 8; ++c)
            if (c < team) {
              v[0] += o[c][0].x, v[1] += o[c][0].y, v[2] += o[c][0].z, v[3] += o[c][0].w;
              v[4] += o[c][1].x, v[5] += o[c][1].y, v[6] += o[c][1].z, v[7] += o[c][1].w;
            }
          split_h(v, scale, ra - col, top, rest);
        }
        *reinterpret_cast<uint4*>(hs + r * S::kHRow + col) = top;
        *reinterpret_cast<uint4*>(hs + r * S::kHRow + R + col) = rest;
      }
      __syncthreads();
    }
    if (ra == 0 && team > 1) {
      cluster_arrive();
      cluster_wait();
    }
    // no CTA writes its sums again, or ends, before every CTA has read them
    if (team > 1) cluster_arrive();

    const int row[2] = {rows[g], rows[g + 8]};
    int col = (c0 + warp) * S::kOuts + 8 * t;
#pragma unroll 1
    for (int j = n1; j < n; ++j) {
      arrived();
#pragma unroll
      for (int o = 0; o < S::kOuts / 32; ++o) {  // 32 outputs at a time
        float acc[4][4] = {};
        if (ra) {
          const uint16_t* h0 = hs + g * S::kHRow;
          const uint16_t* h1 = h0 + 8 * S::kHRow;
#pragma unroll
          for (int q = 0; q < S::kSteps; ++q) {
            if (q * 32 >= ra) break;
            if (R == 16) {
              uint2 w[4];
#pragma unroll
              for (int x = 0; x < 4; ++x)
                w[x] = *reinterpret_cast<const uint2*>(from + 2048 + piece_at<2>(32 * o + 8 * (g >> 1) + 2 * x + (g & 1), t >> 1) + 8 * (t & 1));
#pragma unroll
              for (int term = 0; term < 2; ++term) {
                const uint2 u = *reinterpret_cast<const uint2*>(h0 + term * R + 4 * t);
                const uint2 v = *reinterpret_cast<const uint2*>(h1 + term * R + 4 * t);
#pragma unroll
                for (int x = 0; x < 4; ++x) mma16816(acc[x], u.x, v.x, u.y, v.y, w[x].x, w[x].y);
              }
            } else {
              uint4 w[4];
#pragma unroll
              for (int x = 0; x < 4; ++x)
                w[x] = *reinterpret_cast<const uint4*>(from + 2048 + piece_at<S::kPieces>(32 * o + 8 * (g >> 1) + 2 * x + (g & 1), 4 * q + t));
#pragma unroll
              for (int term = 0; term < 2; ++term) {
                const uint4 u = *reinterpret_cast<const uint4*>(h0 + term * R + q * 32 + 8 * t);
                const uint4 v = *reinterpret_cast<const uint4*>(h1 + term * R + q * 32 + 8 * t);
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                  mma16816(acc[x], u.x, v.x, u.y, v.y, w[x].x, w[x].y);
                  mma16816(acc[x], u.z, v.z, u.w, v.w, w[x].z, w[x].w);
                }
              }
            }
          }
        }
        const int left = p.n - col - 32 * o;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (row[h] < 0 || left <= 0) continue;
          const uint4 v = *reinterpret_cast<const uint4*>(from + piece_at<kYLanes>(g + 8 * h, 4 * o + t));
          uint32_t w[4] = {v.x, v.y, v.z, v.w};
          if (ra)
#pragma unroll
            for (int x = 0; x < 4; ++x) w[x] = pack_bf16(bf_lo(w[x]) + acc[x][2 * h], bf_hi(w[x]) + acc[x][2 * h + 1]);
          uint16_t* op = p.out + (int64_t)row[h] * p.ldo + col + 32 * o;
          if (left >= 8) {
            *reinterpret_cast<uint4*>(op) = make_uint4(w[0], w[1], w[2], w[3]);
          } else {
#pragma unroll
            for (int x = 0; x < 8; ++x)
              if (x < left) op[x] = (uint16_t)(w[x >> 1] >> (16 * (x & 1)));
          }
        }
      }
      fetch(j + S::kAhead);
      next();
      col += S::kOuts * kWarps;
    }
    copy_wait<0>();
    if (team > 1) cluster_wait();
    __syncthreads();  // every warp is done with the tile's rows
  }
}

template <int R>
int launch(const LoraArgs& p, const DeviceInfo& dev, cudaStream_t s) {
  using S = Shape<R>;
  static std::atomic<unsigned long long> configured{0};
  if (!allow_smem((const void*)lora_kernel<R>, S::kSmem, configured)) return QG_ERR_CUDA;
  // The tiles are counted on the device.  About as many: full ones, or one for each adapter that is met where every row draws its
  // own.  The 152 SMs' partitions hold 15 clusters of eight CTAs and 36 of four (the occupancy query's answer for each of the four
  // forms, which all fill an SM's shared memory); more would wait for a turn of their own, and so would the last ones on a GPU that
  // holds fewer: slower, with the same results.
  const double met = p.n_adapters * -std::expm1(p.m * std::log1p(-1.0 / (p.n_adapters + 1)));
  const int full = (p.m + T - 1) / T, likely = std::max(full, std::min(p.m, (int)std::ceil(met)));
  const int most = std::min(p.m, full + std::min(p.n_adapters + 1, p.m));
  const int c = likely <= dev.sms / 10 ? 8 : 4, clusters = std::max(1, std::min(most, c == 8 ? dev.sms / 10 : dev.sms / 4 - 2));
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
  if (cudaLaunchKernelEx(&cfg, lora_kernel<R>, p) != cudaSuccess) return QG_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? QG_OK : QG_ERR_CUDA;
}

}  // namespace

int launch_lora(const LoraArgs& all, const DeviceInfo& dev, void* stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  for (int64_t at = 0; at < all.m; at += kLoraFewRows) {
    LoraArgs p = all;
    p.m = (int)std::min<int64_t>(kLoraFewRows, all.m - at);
    p.ids += at;
    p.x += at * p.ldx;
    p.y += at * p.ldy;
    p.out += at * p.ldo;
    const int st = p.max_rank <= 16 ? launch<16>(p, dev, s) : p.max_rank <= 32 ? launch<32>(p, dev, s)
                   : p.max_rank <= 64 ? launch<64>(p, dev, s) : launch<128>(p, dev, s);
    if (st != QG_OK) return st;
  }
  return QG_OK;
}

}  // namespace qg
