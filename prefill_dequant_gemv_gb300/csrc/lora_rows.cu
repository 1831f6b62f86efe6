// Low-rank adapters for many rows, in two launches:
//   shrink: h[i] = a_e x[i] of every row, in fp32 parts;   expand: out[i] = bf16(y[i] + scale_e b_e h[i])
//
// Both stream their long operand once (x; y and out) and are bound by HBM; A, B and h
// come from L2.  Rows of one adapter are taken 128 at a time (a tile), the M of a tcgen05 MMA.  The
// tiles' inputs (shrink) or outputs (expand), cut into chunks of 128, form one line of units that the
// CTAs, one an SM, share evenly whatever the sizes: a CTA's range may begin and end inside a
// tile.  In shrink that leaves a tile's h in parts, one for every CTA on it; CTA c's part of tile
// t is number c + t (each step along the line raises one of the two), and expand adds a tile's
// parts in that order, so results do not depend on timing.
//
// Rows may lie anywhere: the operands are copied 16 bytes a thread (cp.async), some chunks ahead,
// what lies past a row's end or an adapter's rank as zeros, into the 128-byte swizzled layout that
// the MMAs read.  In expand h's two bf16 terms are multiplied one after the other into the same
// accumulator, and the outputs of a chunk are dealt to the MMA's columns so that a lane that loads
// fragments of 16 rows x 8 columns from tensor memory holds eight contiguous outputs of a row: y comes
// and the sum leaves 16 bytes a lane, y by way of slots in shared memory that are the lane's own.
#include <algorithm>

#include "qg_lora_dev.cuh"
#include "qg_tc.cuh"

namespace qg {
namespace {

constexpr int T = 128;      // rows of a tile
constexpr int kWidth = 128;  // inputs or outputs of a chunk
constexpr int kBatch = 16;  // tiles whose rows a CTA lists at a time
constexpr uint32_t kAtom = T * 128;  // bytes of 128 rows of 64 bf16

// A bounded wait with one answer for the warp.
__device__ __forceinline__ bool wait_warp(uint64_t* bar, int pass, int* status) {
  return __all_sync(0xFFFFFFFFu, mbar_wait_bounded(bar, pass & 1, status));
}

// Fragments of 16 rows x 32 columns: lane 4 g + t has rows g and g + 8, columns 8 x + 2 t and the next of block x, in
// v[4 x], v[4 x + 1] and v[4 x + 2], v[4 x + 3].
__device__ __forceinline__ void tmem_ld_rows(uint32_t taddr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]), "=r"(v[9]),
        "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(taddr));
}

// The line of units: CTA c's range, and the CTA of a unit.  Never more CTAs than units.
__device__ __forceinline__ int64_t line_begin(int64_t units, int ctas, int c) { return units * c / ctas; }
__device__ __forceinline__ int line_owner(int64_t units, int ctas, int64_t u) { return (int)(((u + 1) * ctas - 1) / units); }
// Shrink's CTAs on the line: a tile of few goes into about eight parts at most, as expand reads them all.
__device__ __forceinline__ int shrink_ctas(int64_t units, int n_tiles, int grid) { return (int)min(units, (int64_t)min(grid, 8 * n_tiles)); }

// A tile as shrink describes it to expand: its rows (past the last the first again: what is computed of them is not
// stored), how many, adapter and rank.
struct Tile {
  int rows[T];
  int live, bin, rank, pad;
};
struct Table {
  int n_adapter, n_all, pad[62];  // tiles with an adapter, which come first, and all
  Tile tiles[1];
};

// ids -> one tile.
template <int THREADS>
__device__ __forceinline__ void describe(const LoraArgs& p, Tiles<THREADS>& tl, int tile, Tile& to) {
  const int e = tl.collect(p, T, tile, to.rows);
  const int r = threadIdx.x < T ? to.rows[threadIdx.x] : 0;
  const int n = __syncthreads_count(threadIdx.x < T && r >= 0);
  if (r < 0) to.rows[threadIdx.x] = to.rows[0];
  if (threadIdx.x == 0) {
    to.live = n;
    to.bin = e;
    to.rank = rank_of(p, e);
  }
}
__device__ __forceinline__ void store_tile(Table* table, int tile, const Tile& from) {
  if (threadIdx.x < sizeof(Tile) / 16)
    reinterpret_cast<int4*>(table->tiles + tile)[threadIdx.x] = reinterpret_cast<const int4*>(&from)[threadIdx.x];
}

__device__ __forceinline__ int up16(int rank) { return (rank + 15) & ~15; }

// ------------------------------------------------------------------ shrink
template <int ATOMS>  // of 64 ranks: 1 or 2
struct Shrink {
  static constexpr int kThreads = 416;  // eight warps of copies, one of MMAs, four that store h
  static constexpr int kRank = 64 * ATOMS;
  static constexpr int kStages = ATOMS == 1 ? 4 : 3;
  static constexpr uint32_t kAHalf = kRank * 128;                // 64 inputs of A
  static constexpr uint32_t kStage = 2 * kAtom + 2 * kAHalf;    // 128 inputs of x and of A
  static constexpr size_t kSmem = (size_t)kStages * kStage + 1024;
};

template <int ATOMS>
__global__ void __launch_bounds__(Shrink<ATOMS>::kThreads) lora_shrink_kernel(LoraArgs p, Table* table, float* parts, int pitch) {
  using S = Shrink<ATOMS>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Tiles<S::kThreads> tl;
  __shared__ __align__(16) Tile b[kBatch];
  __shared__ uint64_t full[S::kStages], empty[S::kStages], sum_full[2], sum_empty[2], fin;
  __shared__ uint32_t tmem_slot;
  const uint32_t ring = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < S::kStages; ++i) {
      mbar_init(&full[i], 256);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sum_full[i], 1);
      mbar_init(&sum_empty[i], 4);
    }
    mbar_init(&fin, 1);
    fence_mbar_init();
  }
  pdl_wait();
  tl.count(p, T);
  const int chunks = (p.k + kWidth - 1) / kWidth, n_tiles = tl.first[p.n_adapters], n_all = tl.first[p.n_adapters + 1];
  const int64_t units = (int64_t)n_tiles * chunks;
  const int ctas = shrink_ctas(units, n_tiles, gridDim.x), c = blockIdx.x;
  if (c == 0 && tid == 0) {
    table->n_adapter = n_tiles;
    table->n_all = n_all;
  }
  for (int tile = n_tiles + c; tile < n_all; tile += gridDim.x) {  // rows without an adapter are expand's alone
    describe(p, tl, tile, b[0]);
    __syncthreads();
    store_tile(table, tile, b[0]);
    __syncthreads();
  }
  if (c >= ctas) return;
  if (warp == 8) {
    tmem_alloc(&tmem_slot, 2 * S::kRank);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  if (tid == 0) pdl_launch_dependents();  // not before this CTA has its tensor memory
  const int64_t u0 = line_begin(units, ctas, c), u1 = line_begin(units, ctas, c + 1);
  const int t_first = (int)(u0 / chunks), t_last = (int)((u1 - 1) / chunks);

  int it = 0, sums = 0;  // chunks and tiles so far
  bool ok = true;
  for (int t0 = t_first; t0 <= t_last; t0 += kBatch) {
    const int nt = min(kBatch, t_last + 1 - t0);
    for (int i = 0; i < nt; ++i) describe(p, tl, t0 + i, b[i]);
    __syncthreads();
    for (int i = 0; i < nt; ++i)  // for expand, by the CTA of the tile's first chunk
      if ((int64_t)(t0 + i) * chunks >= u0) store_tile(table, t0 + i, b[i]);
    for (int i = 0; i < nt; ++i) {
      const int tile = t0 + i, ra = b[i].rank;
      const int k0 = (int)(max(u0, (int64_t)tile * chunks) - (int64_t)tile * chunks);
      const int k1 = (int)(min(u1, (int64_t)(tile + 1) * chunks) - (int64_t)tile * chunks);
      if (ra == 0) continue;
      if (warp < 8) {  // copies: a thread has one of a row's 16 pieces and every 16th row
        const int piece = tid & 15, r0 = tid >> 4;
        int col = k0 * kWidth + 8 * piece;
        const uint32_t at = r0 * 128 + (((piece & 7) ^ (r0 & 7)) << 4);
        const uint16_t* xp[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) xp[j] = p.x + (int64_t)b[i].rows[r0 + 16 * j] * p.ldx + col;
        const uint16_t* ap = p.a + ((int64_t)b[i].bin * p.max_rank + min(r0, p.max_rank - 1)) * p.lda + col;
        for (int ch = k0; ch < k1; ++ch, ++it) {
          const int s = it % S::kStages;
          if (it >= S::kStages) ok = ok && wait_warp(&empty[s], it / S::kStages - 1, p.status);
          if (!ok) break;
          const int left = bytes_of(p.k - col);
          const uint32_t xs = ring + s * S::kStage + (piece >> 3) * kAtom + at;
          const uint32_t as = ring + s * S::kStage + 2 * kAtom + (piece >> 3) * S::kAHalf + at;
#pragma unroll
          for (int j = 0; j < 8; ++j) copy16(xs + j * 2048, left ? xp[j] : p.x, left);
#pragma unroll
          for (int j = 0; j < S::kRank / 16; ++j)
            if (16 * j < ra) {
              const bool in = r0 + 16 * j < ra && left;
              copy16(as + j * 2048, in ? ap + (int64_t)(16 * j) * p.lda : p.a, in ? left : 0);
            }
          cp_async_arrive_noinc(&full[s]);
          col += kWidth;
          ap += kWidth;
#pragma unroll
          for (int j = 0; j < 8; ++j) xp[j] += kWidth;
        }
      } else if (warp == 8) {  // MMAs: x's rows by A's
        if (lane == 0) {
          const int buf = sums & 1;
          if (sums >= 2) ok = ok && mbar_wait_bounded(&sum_empty[buf], (sums / 2 - 1) & 1, p.status);
          tc_fence_after();
          const uint32_t idesc = idesc_bf16_f32(T, up16(ra)), d = tmem + buf * S::kRank;
          for (int ch = k0; ch < k1 && ok; ++ch, ++it) {
            const int s = it % S::kStages;
            ok = mbar_wait_bounded(&full[s], (it / S::kStages) & 1, p.status);
            if (!ok) break;
            tc_fence_after();
            fence_proxy_async_smem();  // the copies' writes before the tensor cores' reads
            const uint32_t xs = ring + s * S::kStage, as = xs + 2 * kAtom;
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
              mma_bf16_ss(d, sw128_desc(xs + (kk >> 2) * kAtom + (kk & 3) * 32), sw128_desc(as + (kk >> 2) * S::kAHalf + (kk & 3) * 32),
                          idesc, ch > k0 || kk);
            mma_commit(&empty[s]);
          }
          if (ok) mma_commit(&sum_full[buf]);
        }
        __syncwarp();
        ++sums;
      } else {  // h's part: lane = row
        const int buf = sums & 1, quad = warp & 3;
        ok = ok && wait_warp(&sum_full[buf], sums / 2, p.status);
        if (ok) {
          tc_fence_after();
          float* to = parts + ((int64_t)(c + tile) * T + quad * 32 + lane) * pitch;
          for (int j = 0; j < ra; j += 16) {
            uint32_t v[16];
            tmem_ld16(tmem + (quad << 21) + buf * S::kRank + j, v);
            tmem_ld_wait16(v);
#pragma unroll
            for (int x = 0; x < 4; ++x)
              reinterpret_cast<uint4*>(to + j)[x] = make_uint4(v[4 * x], v[4 * x + 1], v[4 * x + 2], v[4 * x + 3]);
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sum_empty[buf]);
        }
        ++sums;
      }
    }
    __syncthreads();  // the lists are written again
  }
  // leave nothing in flight: copies into this CTA's shared memory, MMAs that read it
  if (warp < 8) cp_async_wait_all();
  if (warp == 8) {
    if (lane == 0) {
      mma_commit(&fin);
      mbar_wait_bounded(&fin, 0, p.status);
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 8) tmem_dealloc(tmem, 2 * S::kRank);
}

// ------------------------------------------------------------------ expand
template <int ATOMS>
struct Expand {
  static constexpr int kWarps = 16;                    // of copies and sums; one more of MMAs
  static constexpr int kThreads = 32 * kWarps + 32;
  static constexpr int kAhead = ATOMS == 1 ? 3 : 2;    // chunks in flight
  static constexpr uint32_t kTerm = ATOMS * kAtom;     // one term of h
  static constexpr uint32_t kB = ATOMS * kAtom;        // 128 outputs of B
  static constexpr uint32_t kY = 4 * 512;              // a warp's share of y: 32 rows x 32 outputs
  static constexpr size_t kSmem = 2 * kTerm + kAhead * (kB + kWarps * kY) + 1024;
};

template <int ATOMS>
__global__ void __launch_bounds__(Expand<ATOMS>::kThreads) lora_expand_kernel(LoraArgs p, const Table* table, const float* parts, int pitch,
                                                                             int shrink_grid) {
  using S = Expand<ATOMS>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(16) Tile b[kBatch];
  __shared__ uint64_t b_full[S::kAhead], d_full[2], d_empty[2], h_full, fin;
  __shared__ uint32_t tmem_slot;
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t hs = smem_u32(smem), bs = hs + 2 * S::kTerm, ys = bs + S::kAhead * S::kB;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  if (tid == 0) {
    for (int i = 0; i < S::kAhead; ++i) mbar_init(&b_full[i], 32 * S::kWarps);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&d_full[i], 1);
      mbar_init(&d_empty[i], S::kWarps);
    }
    mbar_init(&h_full, S::kWarps);
    mbar_init(&fin, 1);
    fence_mbar_init();
  }
  pdl_wait();
  const int chunks = (p.n + kWidth - 1) / kWidth;
  const int n_adapter = __ldcg(&table->n_adapter), n_tiles = __ldcg(&table->n_all);
  const int64_t units = (int64_t)n_tiles * chunks;
  const int ctas = (int)min((int64_t)gridDim.x, units), c = blockIdx.x;
  if (c >= ctas) return;
  if (warp == S::kWarps) {
    tmem_alloc(&tmem_slot, 2 * kWidth);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  if (tid == 0) pdl_launch_dependents();  // not before this CTA has its tensor memory
  const int64_t u0 = line_begin(units, ctas, c), u1 = line_begin(units, ctas, c + 1);
  const int t_first = (int)(u0 / chunks), t_last = (int)((u1 - 1) / chunks);
  const int k_chunks = (p.k + kWidth - 1) / kWidth;
  const int64_t k_units = (int64_t)n_adapter * k_chunks;
  const int k_ctas = shrink_ctas(k_units, n_adapter, shrink_grid);
  const bool in_place = p.out == p.y;

  int mm = 0, tiles_h = 0;  // chunks multiplied and tiles whose h was laid out so far
  bool ok = true;
  for (int t0 = t_first; t0 <= t_last; t0 += kBatch) {
    const int nt = min(kBatch, t_last + 1 - t0);
    for (int x = tid; x < nt * (int)(sizeof(Tile) / 16); x += S::kThreads)
      reinterpret_cast<int4*>(b)[x] = __ldcg(reinterpret_cast<const int4*>(table->tiles + t0) + x);
    __syncthreads();
    const int64_t b0 = max(u0, (int64_t)t0 * chunks);
    const int n = (int)(min(u1, (int64_t)(t0 + nt) * chunks) - b0);
    int i = (int)(b0 / chunks) - t0, ch = (int)(b0 % chunks);
    if (warp == S::kWarps) {  // MMAs: h's rows, both terms, by B's
      if (lane == 0) {
        bool fresh = true;
        for (int j = 0; j < n && ok; ++j) {
          const int ra = b[i].rank;
          if (ra) {
            const int buf = mm & 1, s = mm % S::kAhead;
            if (fresh) ok = mbar_wait_bounded(&h_full, tiles_h++ & 1, p.status);
            if (mm >= 2) ok = ok && mbar_wait_bounded(&d_empty[buf], (mm / 2 - 1) & 1, p.status);
            ok = ok && mbar_wait_bounded(&b_full[s], (mm / S::kAhead) & 1, p.status);
            if (!ok) break;
            tc_fence_after();
            fence_proxy_async_smem();  // the copies' writes before the tensor cores' reads
            const uint32_t idesc = idesc_bf16_f32(T, kWidth), d = tmem + buf * kWidth;
            for (int term = 0; term < 2; ++term)
              for (int kk = 0; 16 * kk < ra; ++kk)
                mma_bf16_ss(d, sw128_desc(hs + term * S::kTerm + (kk >> 2) * kAtom + (kk & 3) * 32),
                            sw128_desc(bs + s * S::kB + (kk >> 2) * kAtom + (kk & 3) * 32), idesc, term || kk);
            mma_commit(&d_full[buf]);
            ++mm;
          }
          fresh = ++ch == chunks;
          if (fresh) ch = 0, ++i;
        }
      }
      __syncwarp();
    } else {
      const int quad = warp & 3, group = warp >> 2, row0 = quad * 32 + g;
      uint8_t* mine = smem + 2 * S::kTerm + S::kAhead * S::kB + warp * S::kY + lane * 16;
      const uint32_t mine_at = ys + warp * S::kY + lane * 16;
      // the copies' state: tile, output and pointers of the next chunk
      constexpr int kRow = 8 * ATOMS, kPass = 32 * S::kWarps / kRow;  // pieces of a row of B, rows of B in one pass of the threads
      const int piece = tid % kRow, o = tid / kRow;
      // output o of each 32 stands in the MMA's column 8 x + 2 a + i, o = 8 a + 2 x + i
      const int place = (o & ~31) + 8 * ((o >> 1) & 3) + 2 * ((o >> 3) & 3) + (o & 1);
      const uint32_t b_at = (piece >> 3) * kAtom + place * 128 + (((piece & 7) ^ (place & 7)) << 4);
      int fi = i, fc = ch * kWidth, ra_f = 0, slot_y = 0, slot_b = mm % S::kAhead;
      const uint16_t *yp[4], *bp = p.b;
      auto aim = [&]() {
        ra_f = b[fi].rank;
#pragma unroll
        for (int m = 0; m < 4; ++m) yp[m] = p.y + (int64_t)b[fi].rows[row0 + 8 * m] * p.ldy + fc + group * 32 + 8 * t;
        if (ra_f) bp = p.b + ((int64_t)b[fi].bin * p.n + fc + o) * p.max_rank + 8 * piece;
      };
      aim();
      auto fetch = [&](int j) {
        if (j < n) {
          if (ra_f) {
            const int bytes = bytes_of(ra_f - 8 * piece);  // ranks past the adapter's as zeros
            if (8 * piece < up16(ra_f)) {
#pragma unroll
              for (int x = 0; x < kWidth / kPass; ++x) {
                const bool in = fc + o + x * kPass < p.n && bytes;
                copy16(bs + slot_b * S::kB + b_at + x * kPass * 128, in ? bp + (int64_t)x * kPass * p.max_rank : p.b, in ? bytes : 0);
              }
            }
            cp_async_arrive_noinc(&b_full[slot_b]);
            slot_b = slot_b + 1 == S::kAhead ? 0 : slot_b + 1;
          }
          const int left = bytes_of(p.n - fc - group * 32 - 8 * t);
          const uint32_t to = mine_at + slot_y * S::kWarps * S::kY;
          slot_y = slot_y + 1 == S::kAhead ? 0 : slot_y + 1;
          if (left) {
#pragma unroll
            for (int m = 0; m < 4; ++m) copy16(to + m * 512, yp[m], left);
          }
          fc += kWidth;
          if (fc >= chunks * kWidth) {
            fc = 0;
            if (++fi < nt) aim();
          } else {
#pragma unroll
            for (int m = 0; m < 4; ++m) yp[m] += kWidth;
            bp += kWidth * p.max_rank;
          }
        }
        copy_commit();
      };
#pragma unroll
      for (int j = 0; j < S::kAhead; ++j) fetch(j);
      bool fresh = true;  // a tile begins
      int ra = 0, live = 0, nb = 0, slot = 0;
      uint16_t* op[4];
      for (int j = 0; j < n; ++j) {
        if (fresh) {
          const int e = b[i].bin, tile = t0 + i;
          ra = b[i].rank;
          live = b[i].live - row0;  // row m of this lane exists if 8 m < live
          nb = ch * kWidth + group * 32;
#pragma unroll
          for (int m = 0; m < 4; ++m) op[m] = p.out + (int64_t)b[i].rows[row0 + 8 * m] * p.ldo + nb + 8 * t;
          if (ra) {  // h's terms; the last tile's MMAs have ended, as this warp has had their sums
            const int p0 = line_owner(k_units, k_ctas, (int64_t)tile * k_chunks),
                      p1 = line_owner(k_units, k_ctas, (int64_t)(tile + 1) * k_chunks - 1), pieces = up16(ra) / 8;
            const float scale = p.scales[e];
            const int64_t step = (int64_t)T * pitch;
            for (int x = tid; x < T * pieces; x += 32 * S::kWarps) {
              const int row = x / pieces, pc = x - row * pieces;
              const float* from = parts + (int64_t)(p0 + tile) * step + row * pitch + 8 * pc;
              float v[8] = {};
              for (int q = p0; q <= p1; q += 4) {  // four parts' loads at a time
                float4 a[4][2];
#pragma unroll
                for (int y = 0; y < 4; ++y)
#pragma unroll
                  for (int z = 0; z < 2; ++z)
                    a[y][z] = q + y <= p1 ? __ldcg(reinterpret_cast<const float4*>(from + (q - p0 + y) * step) + z)
                                          : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                  v[0] += a[y][0].x, v[1] += a[y][0].y, v[2] += a[y][0].z, v[3] += a[y][0].w;
                  v[4] += a[y][1].x, v[5] += a[y][1].y, v[6] += a[y][1].z, v[7] += a[y][1].w;
                }
              }
              uint4 top, rest;
              split_h(v, scale, ra - 8 * pc, top, rest);
              uint8_t* to = smem + (pc >> 3) * kAtom + row * 128 + (((pc & 7) ^ (row & 7)) << 4);
              *reinterpret_cast<uint4*>(to) = top;
              *reinterpret_cast<uint4*>(to + S::kTerm) = rest;
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&h_full);
          }
        }
        const int buf = mm & 1, left = p.n - nb - 8 * t;
        if (ra) {
          ok = wait_warp(&d_full[buf], mm / 2, p.status);
          if (!ok) break;
          tc_fence_after();
          ++mm;
        }
        copy_wait<S::kAhead - 1>();
        const uint8_t* from = mine + slot * S::kWarps * S::kY;
        slot = slot + 1 == S::kAhead ? 0 : slot + 1;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t acc[16];
          if (ra) {
            tmem_ld_rows(tmem + (quad << 21) + (half << 20) + buf * kWidth + group * 32, acc);
            tmem_ld_wait16(acc);
            if (half == 1) {
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(&d_empty[buf]);
            }
          }
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int m = 2 * half + h;
            if (8 * m >= live || left <= 0 || (ra == 0 && in_place)) continue;
            const uint4 v = *reinterpret_cast<const uint4*>(from + m * 512);
            uint32_t w[4] = {v.x, v.y, v.z, v.w};
            if (ra)
#pragma unroll
              for (int x = 0; x < 4; ++x)
                w[x] = pack_bf16(bf_lo(w[x]) + __uint_as_float(acc[4 * x + 2 * h]), bf_hi(w[x]) + __uint_as_float(acc[4 * x + 2 * h + 1]));
            uint16_t* to = op[m];
            if (left >= 8) {
              *reinterpret_cast<uint4*>(to) = make_uint4(w[0], w[1], w[2], w[3]);
            } else {
#pragma unroll
              for (int x = 0; x < 8; ++x)
                if (x < left) to[x] = (uint16_t)(w[x >> 1] >> (16 * (x & 1)));
            }
          }
        }
#pragma unroll
        for (int m = 0; m < 4; ++m) op[m] += kWidth;
        nb += kWidth;
        fetch(j + S::kAhead);  // into the slots whose pieces have been taken
        fresh = ++ch == chunks;
        if (fresh) ch = 0, ++i;
      }
      copy_wait<0>();
    }
    __syncthreads();  // the lists are written again
  }
  if (warp == S::kWarps) {  // leave no MMA in flight
    if (lane == 0) {
      mma_commit(&fin);
      mbar_wait_bounded(&fin, 0, p.status);
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == S::kWarps) tmem_dealloc(tmem, 2 * kWidth);
}

// The scratch: the table, then h's parts, rows of `pitch` floats.
struct Layout {
  size_t parts, total;
  int pitch;
  Layout(int n_adapters, int max_rank, int64_t m, const DeviceInfo& dev) {
    const int64_t rows = std::min<int64_t>(m, kLoraRowsAtOnce);
    const int64_t tiles = (rows + T - 1) / T + std::min<int64_t>(rows, n_adapters) + 1;  // one partly filled an adapter, and without
    pitch = (max_rank + 15) / 16 * 16;
    parts = (sizeof(Table) + (size_t)tiles * sizeof(Tile) + 255) / 256 * 256;
    total = parts + (size_t)(tiles + dev.sms) * T * pitch * sizeof(float);
  }
};

template <int ATOMS>
int launch(const LoraArgs& p, const DeviceInfo& dev, Table* table, float* parts, int pitch, cudaStream_t s) {
  static std::atomic<unsigned long long> a{0}, b{0};
  if (!allow_smem((const void*)lora_shrink_kernel<ATOMS>, Shrink<ATOMS>::kSmem, a) ||
      !allow_smem((const void*)lora_expand_kernel<ATOMS>, Expand<ATOMS>::kSmem, b))
    return QG_ERR_CUDA;
  if (launch_pdl(lora_shrink_kernel<ATOMS>, dim3(dev.sms), dim3(Shrink<ATOMS>::kThreads), Shrink<ATOMS>::kSmem, s, p, table, parts,
                 pitch) != cudaSuccess ||
      launch_pdl(lora_expand_kernel<ATOMS>, dim3(dev.sms), dim3(Expand<ATOMS>::kThreads), Expand<ATOMS>::kSmem, s, p,
                 static_cast<const Table*>(table), static_cast<const float*>(parts), pitch, dev.sms) != cudaSuccess)
    return QG_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? QG_OK : QG_ERR_CUDA;
}

}  // namespace

size_t lora_rows_bytes(int n_adapters, int max_rank, int64_t m, const DeviceInfo& dev) {
  return Layout(n_adapters, max_rank, m, dev).total;
}

int launch_lora_rows(const LoraArgs& all, const DeviceInfo& dev, void* scratch, void* stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const Layout l(all.n_adapters, all.max_rank, all.m, dev);
  Table* table = static_cast<Table*>(scratch);
  float* parts = reinterpret_cast<float*>(static_cast<char*>(scratch) + l.parts);
  for (int64_t at = 0; at < all.m; at += kLoraRowsAtOnce) {
    LoraArgs p = all;
    p.m = (int)std::min<int64_t>(kLoraRowsAtOnce, all.m - at);
    p.ids += at;
    p.x += at * p.ldx;
    p.y += at * p.ldy;
    p.out += at * p.ldo;
    const int st = p.max_rank <= 64 ? launch<1>(p, dev, table, parts, l.pitch, s) : launch<2>(p, dev, table, parts, l.pitch, s);
    if (st != QG_OK) return st;
  }
  return QG_OK;
}

}  // namespace qg
