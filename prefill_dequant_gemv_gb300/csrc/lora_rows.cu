// Low-rank adapters for many rows, one cooperative launch of a CTA an SM in two phases:
//   shrink: h[i] = a_e x[i] of every row;   expand: out[i] = bf16(y[i] + scale_e b_e h[i])
//
// Both stream their long operand once (x; y and out) and are bound by HBM; A, B and h
// come from L2.  Rows of one adapter are taken 128 at a time (a tile), the M of a tcgen05 MMA.  The
// tiles' inputs (shrink) or outputs (expand), cut into chunks of 128, form one line of units that the
// CTAs share evenly whatever the sizes: a CTA's range may begin and end inside a
// tile.  In shrink that leaves a tile's h in parts, one for every CTA on it; CTA c's part of tile
// t is number c + t (each step along the line raises one of the two); a CTA that begins a tile in
// expand adds the tile's parts in that order once all are there, so results do not depend on timing.  It waits for its
// own tiles only (all CTAs run at once, and none waits before its share of shrink is done); y and B of its first chunks
// are on their way meanwhile.
//
// Rows may lie anywhere: the operands are copied 16 bytes a thread (cp.async), some chunks ahead,
// what lies past a row's end or an adapter's rank as zeros, into the 128-byte swizzled layout that
// the MMAs read.  (A bulk copy a row costs some 60 clocks each: a third of this rate.)  In expand h's two bf16 terms are
// multiplied one after the other into the same accumulator, and the outputs of a chunk are dealt to the MMA's columns
// so that a lane that loads fragments of 16 rows x 8 columns from tensor memory holds eight contiguous outputs of
// a row: y comes and the sum leaves 16 bytes a lane, y by way of slots in shared memory that are the lane's own.
//
// Measured in a graph (us; the bytes at the copy rate): 3999 rows of 5 adapters of rank 16, 6144 to 5120 38.7 (19.5); 8192 rows of 3
// of rank 64, a third each, 5120 to 5120 66 (37.6), to 17408 128 (97.5), the same with 5707 of the rows without an adapter and 1934 and 551
// of two 142; 2048 of rank 128, 5120 to 7168 46 (13.1); 300 rows of 4 of rank 16 18 to 19 (2.0).  In a stream of calls 3 us more.
// What is over the bytes: the rows' sorting, 7 to 9 us, and the chain from a tile's last input to its first output, some 10.
// y's first chunks sent for into L2 during that chain made it longer (39 -> 42, 133 -> 136).
#include <algorithm>

#include "qg_lora_dev.cuh"
#include "qg_tc.cuh"

namespace qg {
namespace {

constexpr int T = 128;      // rows of a tile
constexpr int kWidth = 128;  // inputs or outputs of a chunk
constexpr int kList = 16;    // tiles of a CTA in either phase
// Chunks of expand that take as long as a tile's h: by the rank, 3 at 16 and 8 at 64 (measured: 2.8 and 7.7; four at any rank
// leaves 8192 rows of rank 64 to 17408 outputs 133 us, this 129).
__device__ __forceinline__ int start_chunks(int pitch) { return 1 + (7 * pitch + 32) / 64; }
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

// The line of `units` shared by `ctas` CTAs, the first `more` of which have one more than `each`; never more CTAs than units.
// (32 bits: a 64-bit division takes some 600 clocks.)
struct Line {
  int ctas, each, more;
  __device__ __forceinline__ Line(int units, int most) {
    ctas = min(units, most);
    each = ctas ? units / ctas : 0;
    more = units - each * ctas;
  }
  __device__ __forceinline__ int begin(int c) const { return c < ctas ? c * each + min(c, more) : ctas * each + more; }
  __device__ __forceinline__ int owner(int u) const {
    const int wide = more * (each + 1);
    return u < wide ? u / (each + 1) : more + (u - wide) / each;
  }
};

// A tile: its rows, how many, adapter, rank.
struct Tile {
  int rows[T];
  int live, bin, rank, pad;
};

__device__ __forceinline__ int up16(int rank) { return (rank + 15) & ~15; }

// What the CTAs hand one another (device memory; the counters are zero between calls).
struct Scratch {
  int* done;      // CTAs that have ended
  int* tickets;   // [tile] warps whose share of a part is there, eight a part
  float* parts;   // [CTA + tile][T][pitch]
  int pitch;      // max_rank rounded up to 16
};

template <int ATOMS>  // of 64 ranks: 1 or 2
struct Shape {
  static constexpr int kWarps = 16;  // of work; one more of MMAs
  static constexpr int kThreads = 32 * kWarps + 32;
  static constexpr int kRank = 64 * ATOMS;
  // shrink
  static constexpr int kStages = ATOMS == 1 ? 4 : 3;
  static constexpr uint32_t kAHalf = kRank * 128;             // 64 inputs of A
  static constexpr uint32_t kStage = 2 * kAtom + 2 * kAHalf;  // 128 inputs of x and of A
  // expand
  static constexpr int kAhead = ATOMS == 1 ? 3 : 2;   // chunks in flight
  static constexpr uint32_t kTerm = ATOMS * kAtom;    // one term of h
  static constexpr uint32_t kB = ATOMS * kAtom;       // 128 outputs of B
  static constexpr uint32_t kY = 4 * 512;             // a warp's share of y: 32 rows x 32 outputs
  static constexpr size_t kShrink = (size_t)kStages * kStage, kExpand = 2 * kTerm + kAhead * (kB + kWarps * kY);
  static constexpr size_t kSmem = (kShrink > kExpand ? kShrink : kExpand) + 1024;
  static_assert(kShrink >= 2 * (kLoraRowsAtOnce + kThreads * 8), "the rows' bins lie there first");
};

// The bin that a tile belongs to: the last with first[e] <= tile (those without tiles share their successor's first).
__device__ __forceinline__ int bin_of_tile(const int* first, int n_adapters, int tile) {
  int e = 0;
  for (int step = 1024; step; step >>= 1)
    if (e + step <= n_adapters && first[e + step] <= tile) e += step;
  return e;
}

__device__ __forceinline__ int load_acquire(const int* p) {
  int v;
  asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ void red_release(int* p, int v) {
  asm volatile("red.release.gpu.global.add.s32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}
// Waits, up to the limit, for a counter to reach n; one answer for the warp.
__device__ __forceinline__ bool wait_count(const int* counter, int n, int* status) {
  bool up = false;
  if ((threadIdx.x & 31) == 0) {
    const unsigned long long t0 = global_ns();
    while (!(up = load_acquire(counter) >= n)) {
      __nanosleep(64);
      if (global_ns() - t0 > kWaitLimitNs) {
        atomicExch(status, kStatusTimeout);
        break;
      }
    }
  }
  up = __any_sync(0xFFFFFFFFu, up);
  __syncwarp();  // what the counter stands for is there for every lane
  return up;
}

template <int ATOMS>
__global__ void __launch_bounds__(Shape<ATOMS>::kThreads, 1) lora_rows_kernel(LoraArgs p, Scratch sc) {
  using S = Shape<ATOMS>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Tiles<S::kThreads> tl;
  __shared__ Tile in_list[kList], out_list[kList];
  __shared__ uint64_t full[S::kStages], empty[S::kStages], sum_full[2], sum_empty[2];
  __shared__ uint64_t b_full[S::kAhead], d_full[2], d_empty[2], h_full, ring_free, fin;
  __shared__ uint32_t tmem_slot;
  __shared__ int last_cta;
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t base = smem_u32(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, c = blockIdx.x;
  if (tid == 0) {
    for (int i = 0; i < S::kStages; ++i) {
      mbar_init(&full[i], 256);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sum_full[i], 1);
      mbar_init(&sum_empty[i], 8);
      mbar_init(&d_full[i], 1);
      mbar_init(&d_empty[i], S::kWarps);
    }
    for (int i = 0; i < S::kAhead; ++i) mbar_init(&b_full[i], 32 * S::kWarps);
    mbar_init(&h_full, S::kWarps);
    mbar_init(&ring_free, 1);
    mbar_init(&fin, 1);
    fence_mbar_init();
  }
  if (warp == S::kWarps) {
    tmem_alloc(&tmem_slot, 2 * kWidth);
    tmem_relinquish();
  }
  // the rows' bins, the tiles, this CTA's units in both phases and its tiles' rows
  uint16_t* bins = reinterpret_cast<uint16_t*>(smem);
  tl.count(p, T, bins, (p.m + 8 * S::kThreads - 1) / (8 * S::kThreads) * (8 * S::kThreads));
  const int n_adapter = tl.first[p.n_adapters], n_tiles = tl.first[p.n_adapters + 1];  // tiles with an adapter, which come first, and all
  const int k_chunks = (p.k + kWidth - 1) / kWidth, n_chunks = (p.n + kWidth - 1) / kWidth;
  // In shrink a tile of few goes into about eight parts at most, as one CTA adds them all.  In expand a tile begins with `start` units
  // of no chunk: the time that its h takes.
  const int start = start_chunks(sc.pitch);
  const Line in_line(n_adapter * k_chunks, min((int)gridDim.x, 8 * n_adapter)), out_line(n_tiles * (n_chunks + start), gridDim.x);
  const int ku0 = in_line.begin(c), ku1 = in_line.begin(c + 1), kt0 = ku0 / k_chunks, kt1 = ku1 > ku0 ? (ku1 - 1) / k_chunks + 1 : kt0;
  const int nu0 = out_line.begin(c), nu1 = out_line.begin(c + 1);
  int nt0 = nu0 / (n_chunks + start), ch = max(0, nu0 - nt0 * (n_chunks + start) - start);  // expand's first tile and chunk
  const int nt_last = nu1 / (n_chunks + start), ch_last = max(0, nu1 - nt_last * (n_chunks + start) - start);
  const int nt1 = nt_last + (ch_last > 0), n = (nt_last - nt0) * n_chunks + ch_last - ch;  // past its last tile; its chunks
  // Each adapter's rows in ascending order to the places that they have in this CTA's tiles.  A lane looks at eight rows side
  // by side, a warp at 256 (more than 4352 rows: a run of such blocks); how many there are before them comes from a sum
  // over the lanes and the warps.
  const int blocks = (p.m + 256 * (S::kWarps + 1) - 1) / (256 * (S::kWarps + 1));
  auto look = [&](int i, uint32_t e) {  // bit j: row i + j is e's
    const uint4 v = *reinterpret_cast<const uint4*>(bins + i);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t hits = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) hits |= ((w[j] & 0xFFFFu) == e ? 1u << 2 * j : 0u) | (w[j] >> 16 == e ? 2u << 2 * j : 0u);
    return hits;
  };
  int t = kt0;
  for (int phase = 0; phase < 2;) {  // (one copy of this code: it runs once, from cold instruction caches)
    const int end = phase ? nt1 : kt1;
    if (t >= end) {
      ++phase;
      t = nt0;
      continue;
    }
    const int e = bin_of_tile(tl.first, p.n_adapters, t), first = tl.first[e], row0 = warp * blocks * 256 + 8 * lane;
    t = tl.first[e + 1];
    if (phase && first < kt1 && t > kt0) continue;  // listed already
    int mine = 0;
#pragma unroll 1
    for (int u = 0; u < blocks; ++u) mine += __popc(look(row0 + 256 * u, e));
    const int all = __reduce_add_sync(0xFFFFFFFFu, mine);
    __syncthreads();
    if (lane == 0) tl.warp_sums[warp] = all;
    __syncthreads();
    const int v = lane < S::kWarps + 1 ? tl.warp_sums[lane] : 0;
    int at = __reduce_add_sync(0xFFFFFFFFu, lane < warp ? v : 0);
    const int total = __reduce_add_sync(0xFFFFFFFFu, v);
#pragma unroll 1
    for (int u = 0; u < blocks && all; ++u) {
      uint32_t h = look(row0 + 256 * u, e);
      int place = __popc(h);
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int o = __shfl_up_sync(0xFFFFFFFFu, place, off);
        if (lane >= off) place += o;
      }
      const int sum = __shfl_sync(0xFFFFFFFFu, place, 31);
      place += at - __popc(h);
      at += sum;
      for (; h; h &= h - 1, ++place) {
        const int row = row0 + 256 * u + __ffs(h) - 1, tile = first + place / T;
        if (tile >= kt0 && tile < kt1) in_list[tile - kt0].rows[place % T] = row;
        if (tile >= nt0 && tile < nt1) out_list[tile - nt0].rows[place % T] = row;
      }
    }
    if (tid < kt1 - kt0 || (tid >= 32 && tid - 32 < nt1 - nt0)) {
      const int tile = tid < 32 ? kt0 + tid : nt0 + tid - 32, left = total - (tile - first) * T;
      Tile& to = tid < 32 ? in_list[tid] : out_list[tid - 32];
      if (tile >= first && left > 0) {
        to.live = min(left, T);
        to.bin = e;
        to.rank = tl.rank[e];
      }
    }
  }
  __syncthreads();
  if (tid < T) {  // past a tile's last row: any
    for (int i = 0; i < kt1 - kt0; ++i)
      if (tid >= in_list[i].live) in_list[i].rows[tid] = 0;
    for (int i = 0; i < nt1 - nt0; ++i)
      if (tid >= out_list[i].live) out_list[i].rows[tid] = 0;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  bool ok = true;

  // ---------------------------------------------------------------- shrink
  int sums = 0;  // tiles so far
  {
    int it = 0;  // chunks so far
    for (int tile = kt0; tile < kt1; ++tile) {
      const Tile& b = in_list[tile - kt0];
      const int ra = b.rank;
      if (ra == 0) {  // no h; its flag is not waited for
        continue;
      }
      const int k0 = max(ku0 - tile * k_chunks, 0), k1 = min(ku1 - tile * k_chunks, k_chunks);
      if (warp < 8) {  // copies: a thread has one of a row's 16 pieces and every 16th row
        const int piece = tid & 15, r0 = tid >> 4;
        int col = k0 * kWidth + 8 * piece;
        const uint32_t at = r0 * 128 + (((piece & 7) ^ (r0 & 7)) << 4);
        const uint16_t* xp[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) xp[j] = p.x + (int64_t)b.rows[r0 + 16 * j] * p.ldx + col;
        const int live = b.live - r0;  // row 16 j of this thread exists if 16 j < live
        const uint16_t* ap = p.a + ((int64_t)b.bin * p.max_rank + min(r0, p.max_rank - 1)) * p.lda + col;
        for (int ch = k0; ch < k1; ++ch, ++it) {
          const int s = it % S::kStages;
          if (it >= S::kStages) ok = ok && wait_warp(&empty[s], it / S::kStages - 1, p.status);
          if (!ok) break;
          const int left = bytes_of(p.k - col);
          const uint32_t xs = base + s * S::kStage + (piece >> 3) * kAtom + at;
          const uint32_t as = base + s * S::kStage + 2 * kAtom + (piece >> 3) * S::kAHalf + at;
#pragma unroll
          for (int j = 0; j < 8; ++j) copy16(xs + j * 2048, left ? xp[j] : p.x, 16 * j < live ? left : 0);
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
        ++sums;
      } else if (warp == S::kWarps) {  // MMAs: x's rows by A's
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
            const uint32_t xs = base + s * S::kStage, as = xs + 2 * kAtom;
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
      } else {  // h's part: lane = row, 16 ranks a warp in turns; of the last part's CTA all of h
        const int buf = sums & 1, quad = warp & 3;
        ok = ok && wait_warp(&sum_full[buf], sums / 2, p.status);
        if (ok) {
          tc_fence_after();
          float* to = sc.parts + ((int64_t)(c + tile) * T + quad * 32 + lane) * sc.pitch;
          for (int j = (warp >> 2 & 1) * 16; j < ra; j += 32) {
            uint32_t v[16];
            tmem_ld16(tmem + (quad << 21) + buf * S::kRank + j, v);
            tmem_ld_wait16(v);
#pragma unroll
            for (int x = 0; x < 4; ++x)
              __stcg(reinterpret_cast<uint4*>(to + j) + x, make_uint4(v[4 * x], v[4 * x + 1], v[4 * x + 2], v[4 * x + 3]));
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&sum_empty[buf]);
            red_release(&sc.tickets[tile], 1);
          }
        }
        ++sums;
      }
    }
  }
  if (tid == 32 * S::kWarps) mma_commit(&ring_free);  // every MMA that reads shrink's ring has ended

  // ---------------------------------------------------------------- expand
  const uint32_t hs = base, bs = hs + 2 * S::kTerm, ys = bs + S::kAhead * S::kB;
  int i = 0, mm = 0;  // tile, chunks multiplied so far
  if (warp == S::kWarps) {  // MMAs: h's rows, both terms, by B's
    if (lane == 0) {
      // the sums of shrink have left tensor memory
      if (sums >= 1) ok = ok && mbar_wait_bounded(&sum_empty[(sums - 1) & 1], ((sums - 1) / 2) & 1, p.status);
      if (sums >= 2) ok = ok && mbar_wait_bounded(&sum_empty[sums & 1], ((sums - 2) / 2) & 1, p.status);
      int tiles_h = 0;
      bool fresh = true;
      for (int j = 0; j < n && ok; ++j) {
        const int ra = out_list[i].rank;
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
        fresh = ++ch == n_chunks;
        if (fresh) ch = 0, ++i;
      }
      mma_commit(&fin);  // leave no MMA in flight
      mbar_wait_bounded(&fin, 0, p.status);
    }
    __syncwarp();
  } else {
    ok = ok && wait_warp(&ring_free, 0, p.status);
    const int g = lane >> 2, t = lane & 3, quad = warp & 3, group = warp >> 2, row0 = quad * 32 + g;
    const bool in_place = p.out == p.y;
    uint8_t* mine = smem + 2 * S::kTerm + S::kAhead * S::kB + warp * S::kY + lane * 16;
    const uint32_t mine_at = ys + warp * S::kY + lane * 16;
    // the copies' state: tile, output and pointers of the next chunk
    constexpr int kRow = 8 * ATOMS, kPass = 32 * S::kWarps / kRow;  // pieces of a row of B, rows of B in one pass of the threads
    const int piece = tid % kRow, o = tid / kRow;
    // output o of each 32 stands in the MMA's column 8 x + 2 a + i, o = 8 a + 2 x + i
    const int place = (o & ~31) + 8 * ((o >> 1) & 3) + 2 * ((o >> 3) & 3) + (o & 1);
    const uint32_t b_at = (piece >> 3) * kAtom + place * 128 + (((piece & 7) ^ (place & 7)) << 4);
    int fi = 0, fc = ch * kWidth, ra_f = 0, live_f = 0, slot_y = 0, slot_b = 0;
    const uint16_t *yp[4], *bp = p.b;
    auto aim = [&]() {
      const Tile& b = out_list[fi];
      ra_f = b.rank;
      live_f = b.live - row0;  // row m of this lane exists if 8 m < live
#pragma unroll
      for (int m = 0; m < 4; ++m) yp[m] = p.y + (int64_t)b.rows[row0 + 8 * m] * p.ldy + fc + group * 32 + 8 * t;
      if (ra_f) bp = p.b + ((int64_t)b.bin * p.n + fc + o) * p.max_rank + 8 * piece;
    };
    if (n) aim();
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
#pragma unroll
        for (int m = 0; m < 4; ++m)
          if (left && 8 * m < live_f) copy16(to + m * 512, yp[m], left);
        fc += kWidth;
        if (fc >= n_chunks * kWidth) {
          fc = 0;
          if (++fi < nt1 - nt0) aim();
        } else {
#pragma unroll
          for (int m = 0; m < 4; ++m) yp[m] += kWidth;
          bp += kWidth * p.max_rank;
        }
      }
      copy_commit();
    };
    if (ok) {
#pragma unroll
      for (int j = 0; j < S::kAhead; ++j) fetch(j);
    }
    bool fresh = true;  // a tile begins
    int ra = 0, live = 0, nb = 0, slot = 0;
    uint16_t* op[4];
    for (int j = 0; j < n && ok; ++j) {
      if (fresh) {
        const Tile& b = out_list[i];
        ra = b.rank;
        live = b.live - row0;
        nb = ch * kWidth + group * 32;
#pragma unroll
        for (int m = 0; m < 4; ++m) op[m] = p.out + (int64_t)b.rows[row0 + 8 * m] * p.ldo + nb + 8 * t;
        if (ra) {  // h's terms; the last tile's MMAs have ended, as this warp has had their sums
          const int tile = nt0 + i, pieces = up16(ra) / 8;
          const int p0 = in_line.owner(tile * k_chunks), n_parts = in_line.owner((tile + 1) * k_chunks - 1) - p0 + 1;
          const int64_t step = (int64_t)T * sc.pitch;
          const float scale = p.scales[b.bin];
          ok = wait_count(&sc.tickets[tile], 8 * n_parts, p.status);
          if (!ok) break;
          for (int x = tid; x < T * pieces; x += 32 * S::kWarps) {
            const int row = x / pieces, pc = x - row * pieces;
            const float* from = sc.parts + (p0 + tile) * step + row * sc.pitch + 8 * pc;
            float v[8] = {};
            for (int q = 0; q < n_parts; q += 4) {  // four parts' loads at a time
              float4 a[4][2];
#pragma unroll
              for (int y = 0; y < 4; ++y)
#pragma unroll
                for (int z = 0; z < 2; ++z)
                  a[y][z] = q + y < n_parts ? __ldcg(reinterpret_cast<const float4*>(from + (q + y) * step) + z)
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
      fresh = ++ch == n_chunks;
      if (fresh) ch = 0, ++i;
    }
    cp_async_wait_all();  // leave no copy in flight
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == S::kWarps) tmem_dealloc(tmem, 2 * kWidth);
  // the last CTA leaves the counters at zero
  if (tid == 0) last_cta = ticket_add(sc.done, 1) == (int)gridDim.x - 1;
  __syncthreads();
  if (last_cta) {
    for (int x = tid; x < n_adapter; x += S::kThreads) sc.tickets[x] = 0;
    if (tid == 0) *sc.done = 0;
  }
}

// The scratch after the status word: counters, at one place and of one size whatever the call's, as they are to be zero before the
// next call of any sizes; then h's parts.
constexpr int kTickets = (int)kLoraRowsAtOnce / T + kLoraMaxAdapters + 1;  // tiles at most
struct Layout {
  size_t tickets, parts, total;
  int pitch;
  Layout(int n_adapters, int max_rank, int64_t m, const DeviceInfo& dev) {
    const int64_t rows = std::min<int64_t>(m, kLoraRowsAtOnce);
    const int64_t tiles = (rows + T - 1) / T + std::min<int64_t>(rows, n_adapters) + 1;  // one partly filled an adapter, and without
    pitch = (max_rank + 15) / 16 * 16;
    const auto up = [](size_t b) { return (b + 255) / 256 * 256; };
    tickets = 256;  // the CTAs' counter before
    parts = tickets + up(kTickets * sizeof(int));
    total = parts + (size_t)(tiles + dev.sms) * T * pitch * sizeof(float);
  }
};

template <int ATOMS>
int launch(const LoraArgs& p, const DeviceInfo& dev, const Scratch& sc, cudaStream_t s) {
  static std::atomic<unsigned long long> done{0};
  if (!allow_smem((const void*)lora_rows_kernel<ATOMS>, Shape<ATOMS>::kSmem, done)) return QG_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(dev.sms);
  cfg.blockDim = dim3(Shape<ATOMS>::kThreads);
  cfg.dynamicSmemBytes = Shape<ATOMS>::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;  // all CTAs at once
  attr[0].val.cooperative = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, lora_rows_kernel<ATOMS>, p, sc) != cudaSuccess) return QG_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? QG_OK : QG_ERR_CUDA;
}

}  // namespace

size_t lora_rows_bytes(int n_adapters, int max_rank, int64_t m, const DeviceInfo& dev) {
  return Layout(n_adapters, max_rank, m, dev).total;
}

int launch_lora_rows(const LoraArgs& all, const DeviceInfo& dev, void* scratch, void* stream) {
  const Layout l(all.n_adapters, all.max_rank, all.m, dev);
  char* b = static_cast<char*>(scratch);
  const Scratch sc = {reinterpret_cast<int*>(b), reinterpret_cast<int*>(b + l.tickets), reinterpret_cast<float*>(b + l.parts),
                      l.pitch};
  for (int64_t at = 0; at < all.m; at += kLoraRowsAtOnce) {
    LoraArgs p = all;
    p.m = (int)std::min<int64_t>(kLoraRowsAtOnce, all.m - at);
    p.ids += at;
    p.x += at * p.ldx;
    p.y += at * p.ldy;
    p.out += at * p.ldo;
    const int st = p.max_rank <= 64 ? launch<1>(p, dev, sc, static_cast<cudaStream_t>(stream))
                                    : launch<2>(p, dev, sc, static_cast<cudaStream_t>(stream));
    if (st != QG_OK) return st;
  }
  return QG_OK;
}

}  // namespace qg
