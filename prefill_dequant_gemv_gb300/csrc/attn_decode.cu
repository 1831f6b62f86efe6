// Attention of a few rows a KV head over the 8-bit paged cache (decode, speculative
// verification): the R = new * G query rows of one (sequence, KV head) pair, at most 32, against
// all its keys.
//
// The mathematics.  With codes k, v, page scales ks, vs and s_j = scale * ks_j * (q . k_j) * log2(e), each
// row keeps t_j = s_j + log2(vs_j), a reference m near their maximum and P_j = 2^(t_j - m + 6):
//   out = sum_j P_j v_j / sum_j P_j / vs_j.
// The value scale sits in the exponent, so P is rounded relative to the largest contribution
// whatever the scales' spread.  m need not be the maximum: it moves only when some t_j passes it by
// 2.8, so few tiles but the first reduce anything over their keys.
//
// Bound by HBM: each key and value code is used for R rows only.  So nothing converts them: both
// products run on the E4M3 tensor cores with the codes as they lie in the cache, and the 16-bit side
// is split into E4M3 terms instead, which is little work for few rows:
//   scores   S^T[key][row]  = K[128 keys x D]   * Q^T      (A: the key tile, B: the rows, N = 2 terms x rows)
//   outputs  O^T[dim][row] += V^T[D x 128 keys] * P^T      (A: the value tile read transposed, N = 3 terms x rows)
// A query row over a power of two is the sum of two E4M3 terms (bf16 has 8 significant bits, a term 4 and a sign), the second
// scaled up by 2^5: exact but for elements below 2^-13 of the row's largest, off by 2^-21 of it at most.  P, rounded to
// fp16's 11 bits, is the sum of three, the second and third scaled up by 2^4 and 2^9; each term has its own
// accumulator columns, so the scaling comes out at the end.  The third ends at steps of 2^-18, so a P below 2^-7 keeps
// fewer bits: it is off by 2^-19 at most, 2^-25 of the row's largest weight, which is 2^6 at least.  Keys as the M
// dimension fill it whatever R is.  Accumulation and statistics are fp32.
//
//   * The pairs' keys, in tiles of 128, lie on one line, which the CTAs (one an SM) share out evenly
//     whatever the lengths; a pair cut between CTAs leaves partial (m, l, O) rows in the workspace, and the
//     CTA that finishes last adds them in order.  One launch.
//   * One or two warps copy key tiles into a ring by TMA and as many value tiles into another, two bring a
//     pair's query rows, two issue the MMAs (scores, outputs), and groups of four warps turn S into P, a key a
//     thread: its column of R scores comes from tensor memory, its terms go to shared memory as 16-byte rows.
//     The sums of P stay per thread until the pair ends.  A tile's way through these steps is a chain of about
//     2500 cycles, several times what its bytes take to arrive; so several groups work on as many tiles at once,
//     each with its own reference and accumulators, joined at the pair's end.
//
// Measured (GB300; bytes are the codes and scales that the rows see, queries and outputs): 64 sequences of up to
// 8193 tokens, 40/8 heads of 128: 110 us, 5.1 TB/s; one of 131001 tokens, 24/4 heads of 256: 59 us,
// 4.55 TB/s; 16 x 4 rows on 8004 tokens, 24/4 of 256: 45 us, 2.45 TB/s; one token on 777, 40/8 of 128:
// 14.4 us.  Long calls run at the memory's pace but for some 12 us: launch, first tiles
// (2 us until the CTAs are ready, 1.5 until the first copy has landed), the chain of the last tile, and the join of cut
// pairs (5 us); a few short pairs are such a chain alone, of whose 14 us some 6 are not accounted for.  The forms of 80
// registers (16 rows, heads of 64 and 128) spill some 370 bytes.
// Batches of more than 32 sequences read each further one's lengths from memory on their way (Walk).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>

#include "qg_attn.h"
#include "qg_attn_dev.cuh"
#include "qg_sync.cuh"
#include "qg_tc.cuh"

namespace qg {
namespace {

constexpr int kTile = 128;           // keys a tile
constexpr int kMostCtas = 256;
constexpr float kBias = 6.0f;        // P of a key at the reference is 2^6 ...
constexpr float kHead = 2.8f;        // ... and at most 2^8.8 = 446, below E4M3's 448
constexpr float kNone = -3e38f;      // the reference of a row that has seen no key: -inf would make NaN of its masked scores

// D: head dimension; N: rows it is built for (16, 32).
template <int D, int N>
struct Cfg {
  // softmax groups of 128 threads (heads of 256: as many as the ring has stages)
  static constexpr int GROUPS = D == 256 && N == 16 ? 2 : 64 / N;
  static constexpr int THREADS = 128 * GROUPS + 256;
  // registers a thread: what the launch gives, what softmax threads take, what the other two warpgroups keep
  static constexpr int REGS = GROUPS == 4 ? 80 : 128, RSOFT = GROUPS == 4 ? 96 : 168, RREST = GROUPS == 4 ? 48 : 80;
  static_assert(128 * GROUPS * RSOFT + 256 * RREST <= THREADS * REGS && THREADS * REGS <= 65536, "registers");
  static constexpr int PW = D < 128 ? D : 128;       // bytes of a panel row (a TMA box row)
  static constexpr int NP = D / PW;                  // panels
  static constexpr int PANEL = kTile * PW;
  static constexpr int KV = kTile * D;               // bytes of a key (or value) tile
  static constexpr int Q = 2 * N * D;                // both terms of the query rows
  static constexpr int QPANEL = 2 * N * PW;
  static constexpr int QB = 2;                       // buffers of them
  static constexpr int P = 3 * N * kTile;            // a group's terms of P
  static constexpr int MB = NP;                      // M blocks of O (128 dims; D = 64 fills half of one)
  static constexpr int SCOL = 2 * N, OCOL = 3 * N;   // TMEM columns of a group's S and of a block of its O
  static constexpr int OSET = GROUPS * MB * OCOL;    // all groups' O
  static constexpr int OB = GROUPS * SCOL + 2 * OSET <= 512 ? 2 : 1;  // sets: two pairs can be at work
  static constexpr int PRODUCERS = D == 256 ? 1 : 2; // warps that copy keys, and values
  static constexpr int FIXED = 1024 + QB * Q + GROUPS * P + 9216;
  static constexpr int SLOTS = (232448 - FIXED) / KV;
  // key tiles are done with after the scores, value tiles a softmax later
  // (whole multiples of PRODUCERS: a stage is always filled by the same warp)
  static constexpr int SK0 = SLOTS * 2 / 5 < 2 ? 2 : SLOTS * 2 / 5, SK = (SK0 > 6 ? 6 : SK0) / PRODUCERS * PRODUCERS;
  static constexpr int SV = (SLOTS - SK > 8 ? 8 : SLOTS - SK) / PRODUCERS * PRODUCERS;
  static constexpr int METAS = 32;                   // tiles between a key tile's issue and its outputs: fewer
  static constexpr int SMEM = FIXED + (SK + SV) * KV;
  static_assert(SK >= 2 && SV >= 2 && GROUPS * SCOL + OB * OSET <= 512, "shared and tensor memory");
  static_assert(SK + 3 * GROUPS < METAS && SV + GROUPS < METAS, "tiles on their way");
};

// What a stage holds.
struct TileMeta {
  int tok0, len, after;  // after: tiles of its pair in this CTA before it
  int flags;             // 1: some of its rows hold no key; 2: some row of the pair does not see all of it; 4: the CTA's last
  float ks[8], vs[8];    // scales of its groups of 16 keys; key scale 0: the group holds no key that anyone sees
};
struct ValueMeta {
  int after, rows, groups;       // as above; rows before the sequence's end; bits of the groups that hold keys
  int set;                       // its O; 4: the CTA's last; 8: some of its keys are hidden, from all rows or some
  int all0, all1;                // every row of the pair sees the keys all0 .. all1 - 1 of the tile
};
// What a query buffer holds besides the rows.
template <int N>
struct PairMeta {
  int R, n_tiles, i0, i1;       // rows, tiles, and which of this CTA's tiles they are
  int first, skipped;           // its first tile's place on the line, and how many tiles of it earlier CTAs have
  int last, head;               // whether it is the CTA's last pair; its KV head
  const int32_t* pages;
  int64_t base;                 // its first row's output
  alignas(16) float rc[N];      // the row's power of two * scale * log2(e)
  int pos[N];
  int64_t off[N];               // the row's output, from the first one's
};
template <int D, int N>
struct Shared {
  using C = Cfg<D, N>;
  TileMeta tile[C::METAS];
  ValueMeta value[C::METAS];
  PairMeta<N> pair[C::QB];
  alignas(16) float ref[C::OB][C::GROUPS][N];
  alignas(16) float factor[C::GROUPS][N];  // of a group's O at the join
  alignas(16) float grow[C::GROUPS][N];    // what a group's O and sums are multiplied by when references move
  uint32_t moved[C::GROUPS];               // bits of the rows whose reference moves
  float sum[C::OB][C::GROUPS][N], red[C::GROUPS][4][N], inv[N];
  uint64_t kfull[C::SK], kfree[C::SK], vfull[C::SV], vfree[C::SV];
  uint64_t qfull[C::QB], qfree[C::QB];
  uint64_t sfull[C::GROUPS], sfree[C::GROUPS], pfull[C::GROUPS], pvdone[C::GROUPS];
  uint64_t summed[C::OB], joined[C::OB], ended[2], joinbar;
  uint32_t tmem;
  int poison;     // a NaN value code was dropped
  int joins;      // pairs whose parts this CTA has to join in the end, at most two
  int join[2][4];  // rows, first CTA, parts, whether the first part is its CTA's first pair
  int64_t join_base[2];
};

struct DecodeArgs {
  AttnArgs a;
  int* counters;   // one a CTA: the parts of the pair that begins in it and ends in another
  float2* part_ml; // [2 * grid][N]
  float* part_o;   // [2 * grid][N][D]
};

// First key that any row of the sequence sees, rounded down to a page; tiles of a pair (one at least where
// there are rows, so that rows without a key are written).
__device__ __forceinline__ int first_key(const Seq& s, const AttnArgs& a) {
  const int64_t p = (int64_t)s.len - s.rows + 1 - a.window;
  return p > 0 ? ((int)p >> a.c.page_log2) << a.c.page_log2 : 0;
}
// (the host keeps all of a call's tiles below 2^31)
__device__ __forceinline__ int tiles_of(const Seq& s, const AttnArgs& a) {
  return s.rows > 0 ? max(1, (s.len - first_key(s, a) + kTile - 1) / kTile) : 0;
}

// The line cut into even parts: CTA c's begins at begin(c); whose tile u is.
struct Share {
  int each, more;
  __device__ __forceinline__ int begin(int cta) const { return cta * each + min(cta, more); }
  __device__ __forceinline__ int owner(int u) const {
    const int big = more * (each + 1);
    return u < big ? u / (each + 1) : more + (u - big) / each;
  }
};

// A pair takes as long as its tiles and some six more (its rows, its end; 2, 3, 4, 6, 8 and 12 give 125, 117, 114,
// 110, 111 and 112 us for 64 ragged sequences, and 51, 48, 46, 45.5, 45.3 and 47 us for 16 x 4 rows): the line
// counts a pair's tiles and kPairCost places behind them, which no tile stands at.
constexpr int kPairCost = 6;
__device__ __forceinline__ int places_of(const Seq& s, const AttnArgs& a) {
  const int n = tiles_of(s, a);
  return n ? n + kPairCost : 0;
}

// A place on the line: tile k of head h of sequence b, whose pairs have n tiles.  A whole warp walks; lane
// b holds sequence b of the first 32.
struct Walk {
  int b, h, k, n, lo;
  Seq sq, mine;

  // places of all sequences, each counted once (all its KV heads have as many); most: of one pair
  __device__ __forceinline__ int count(const AttnArgs& a, int lane, bool* bad, int* most) {
    const KvArgs& c = a.c;
    mine = {0, 0, 0};
    if (lane < c.n_seqs) mine = seq_of(c, lane, bad);
    const int first = places_of(mine, a);
    int total = __reduce_add_sync(0xFFFFFFFFu, first);
    *most = __reduce_max_sync(0xFFFFFFFFu, first);  // of the first 32 sequences
    for (int base = 32; base < c.n_seqs; base += 32) {
      int t = 0;
      if (base + lane < c.n_seqs) t = places_of(seq_of(c, base + lane, bad), a);
      total += __reduce_add_sync(0xFFFFFFFFu, t);
    }
    return total;
  }
  // pair number `pair` of at most 32 sequences: its places [u0, u1)
  __device__ __forceinline__ void pair_of(const AttnArgs& a, int pair, int lane, int* u0, int* u1) const {
    const int here = places_of(mine, a), which = pair / a.c.hkv, head = pair - which * a.c.hkv;
    const int before = __reduce_add_sync(0xFFFFFFFFu, lane < which ? here : 0);
    const int n = which < 32 ? __shfl_sync(0xFFFFFFFFu, here, which & 31) : 0;
    *u0 = before * a.c.hkv + head * n;
    *u1 = *u0 + n;
  }
  __device__ __forceinline__ void take(const Seq& t, int who) {
    sq.start = __shfl_sync(0xFFFFFFFFu, t.start, who);
    sq.rows = __shfl_sync(0xFFFFFFFFu, t.rows, who);
    sq.len = __shfl_sync(0xFFFFFFFFu, t.len, who);
  }
  // the next pair; there is one
  __device__ __forceinline__ void next_pair(const AttnArgs& a) {
    k = 0;
    if (++h == a.c.hkv) {
      bool ignore = false;
      h = 0;
      do {
        ++b;
        if (b < 32)
          take(mine, b);
        else
          sq = seq_of(a.c, b, &ignore);
        n = tiles_of(sq, a);
      } while (n == 0);
      lo = first_key(sq, a);
    }
  }
  // To a CTA's first tile: the first at or behind place u0; returns its place, or u1 where there is none before u1.
  __device__ __forceinline__ int find(const AttnArgs& a, int u0, int u1, int lane) {
    const KvArgs& c = a.c;
    int left = u0;
    bool ignore = false;
    b = 0, n = 1;
    sq = {0, 0, 0};
    for (int base = 0; base < c.n_seqs; base += 32) {
      Seq t = mine;
      if (base) {
        t = {0, 0, 0};
        if (base + lane < c.n_seqs) t = seq_of(c, base + lane, &ignore);
      }
      const int un = places_of(t, a);
      int sum = un * c.hkv;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xFFFFFFFFu, sum, o);
        if (lane >= o) sum += v;
      }
      const int all = __shfl_sync(0xFFFFFFFFu, sum, 31);
      if (left < all) {
        const int who = __ffs(__ballot_sync(0xFFFFFFFFu, sum > left)) - 1;
        b = base + who;
        n = __shfl_sync(0xFFFFFFFFu, un, who);
        left -= __shfl_sync(0xFFFFFFFFu, sum, who) - n * c.hkv;
        take(t, who);
        break;
      }
      left -= all;
    }
    h = left / n;
    k = left - h * n;
    n -= kPairCost;
    lo = first_key(sq, a);
    if (u0 >= u1) return u1;
    if (k >= n) {  // behind a pair's tiles: on to the next one's
      u0 += n + kPairCost - k;
      if (u0 >= u1) return u1;
      next_pair(a);
    }
    return u0;
  }
};

// The joining of a pair's parts, in their order on the line, by the CTA that finished last: its softmax
// threads (the others have given up their registers).  A load of what other SMs have just written takes some 1900
// cycles, so the parts come by bulk copies into the rings, all of a round at once, and the weights meanwhile.
template <int D, int N>
__device__ __noinline__ void join_parts(const DecodeArgs& da, int R, int G, int64_t base, int c0, int parts, bool at_start,
                                        uint8_t* scratch, uint64_t* bar, uint32_t* phase) {
  using C = Cfg<D, N>;
  const AttnArgs& a = da.a;
  constexpr int T = 128 * C::GROUPS, W = T / 32, WT = kMostCtas * N * 4, ROOM = (C::SK + C::SV) * C::KV - WT;
  static_assert(ROOM >= kMostCtas * 128, "scratch");
  auto slot = [&](int q) { return (int64_t)(2 * (c0 + q) + (q == 0 && !at_start ? 1 : 0)); };
  float* wt = reinterpret_cast<float*>(scratch);  // [parts][N]: weights over the sum
  uint8_t* buf = scratch + WT;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int all = R * D, most = min(all, ROOM / parts / 16 * 4);  // floats of a part, and in one round
  bool dead = false;
#pragma unroll 1
  for (int f0 = 0; f0 < all; f0 += most) {
    const int floats = min(most, all - f0);
    fence_proxy_async_all();  // shared memory read, and the parts written, by ordinary accesses before
    named_sync(15, T);
    if (tid == 0) mbar_arrive_expect_tx(bar, (uint32_t)(parts * floats * 4));
    if (lane == 0)
      for (int q = warp; q < parts; q += W)
        bulk_g2s(buf + q * floats * 4, da.part_o + slot(q) * N * D + f0, (uint32_t)(floats * 4), bar);
    if (f0 == 0) {
      for (int row = warp; row < R; row += W) {  // a warp a row, a lane a part
        float m = -INFINITY, l = 0.0f;
#pragma unroll 2
        for (int q = lane; q < parts; q += 32) {
          const float2 z = __ldcg(&da.part_ml[slot(q) * N + row]);
          const float t = fmaxf(m, z.x);
          if (t != -INFINITY) l = fmaf(l, ex2(m - t), z.y * ex2(z.x - t));
          m = t;
          wt[q * N + row] = z.x;
        }
        const float top = warp_max(m);
        float sum = m == -INFINITY ? 0.0f : l * ex2(m - top);
#pragma unroll
        for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
        for (int q = lane; q < parts; q += 32) {
          const float z = wt[q * N + row];
          wt[q * N + row] = ex2(z - top) * inv;
        }
      }
      named_sync(15, T);
    }
    if (!dead && !wait(bar, *phase & 1, da.a.c.status)) dead = true;
    *phase += 1;
#pragma unroll 1
    for (int e = 4 * tid; e < floats && !dead; e += 4 * T) {
      const int row = (f0 + e) / D, d = (f0 + e) % D, t = row / G, g = row - t * G;
      float4 v = make_float4(0, 0, 0, 0);
#pragma unroll 4
      for (int q = 0; q < parts; ++q) {
        const float4 y = *reinterpret_cast<const float4*>(buf + (q * floats + e) * 4);
        const float f = wt[q * N + row];  // (a part of no weight may hold a NaN that its row sees)
        v.x = fmaf(y.x, f, v.x), v.y = fmaf(y.y, f, v.y), v.z = fmaf(y.z, f, v.z), v.w = fmaf(y.w, f, v.w);
      }
      const __nv_bfloat162 y0 = __floats2bfloat162_rn(v.x, v.y), y1 = __floats2bfloat162_rn(v.z, v.w);
      *reinterpret_cast<uint2*>(a.out + base + t * a.ldo + g * a.hso + d) =
          make_uint2(*reinterpret_cast<const uint32_t*>(&y0), *reinterpret_cast<const uint32_t*>(&y1));
    }
  }
}

// A key of a page whose key scale is 0, in any tile: its P is 0, but a NaN code times 0 is NaN, so its values become 0, once
// they are here.  (Keys that not all rows see the output warp looks after.  With that warp reading the scales of every
// tile 64 ragged sequences took up to 4 us more.)
template <int D, int N>
__device__ __noinline__ bool drop_values(uint8_t* vring, uint64_t* vfull, int i, int key, int* status) {
  using C = Cfg<D, N>;
  const bool ok = wait(&vfull[i % C::SV], (uint32_t)(i / C::SV) & 1u, status);
  uint8_t* at = vring + i % C::SV * C::KV + key * C::PW;
#pragma unroll 1
  for (int e = 0; e < C::NP * C::PW; e += 16)
    *reinterpret_cast<uint4*>(at + e / C::PW * C::PANEL + e % C::PW) = make_uint4(0, 0, 0, 0);
  return ok;
}

template <int D, int N>
__global__ void __launch_bounds__(Cfg<D, N>::THREADS, 1)
    attn_decode_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                       const DecodeArgs da) {
  using C = Cfg<D, N>;
  constexpr int NG = C::GROUPS, NPR = C::PRODUCERS, kMma = 4 * NG;
  static_assert(sizeof(Shared<D, N>) <= 9216 && C::SK <= 8 && C::SV <= 8, "shared memory");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* vring = ring + C::SK * C::KV;
  uint8_t* qbuf = vring + C::SV * C::KV;
  uint8_t* pbuf = qbuf + C::QB * C::Q;
  Shared<D, N>& sh = *reinterpret_cast<Shared<D, N>*>(pbuf + NG * C::P);
  const AttnArgs& a = da.a;
  const KvArgs& c = a.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = a.hq / c.hkv;

  {  // a thread an entry
    const int t = threadIdx.x;
    if (t < C::SK) mbar_init(&sh.kfull[t], 16), mbar_init(&sh.kfree[t], 1);
    if (t < C::SV) mbar_init(&sh.vfull[t], 8), mbar_init(&sh.vfree[t], 1);
    if (t < C::QB) mbar_init(&sh.qfull[t], 64), mbar_init(&sh.qfree[t], 1);
    if (t < NG) {
      mbar_init(&sh.sfull[t], 2);  // the MMAs' end, and the issuing thread's own arrival
      mbar_init(&sh.sfree[t], 4);
      mbar_init(&sh.pfull[t], 4);
      mbar_init(&sh.pvdone[t], 1);
    }
    if (t < C::OB) mbar_init(&sh.summed[t], NG), mbar_init(&sh.joined[t], 1);
    if (t < 2) mbar_init(&sh.ended[t], 1);
    if (t == 2) mbar_init(&sh.joinbar, 1);
    if (t < 8) fence_mbar_init();
  }
  if (warp == kMma) {
    tmem_alloc(&sh.tmem, 512);
    tmem_relinquish();
  }
  pdl_launch_dependents();  // the next kernel's CTAs may take the SMs that this one leaves free, and wait there
  pdl_wait();
  Walk w;
  bool bad = false;
  int most = 0;
  const int total = w.count(a, lane, &bad, &most) * c.hkv;  // places
  if (bad && warp == 0 && blockIdx.x == 0) atomicMax(c.status, kStatusInvalid);
  // with no more CTAs than places, each has one at least
  const int grid = min((int)gridDim.x, total), cta = blockIdx.x;
  const Share share = {total / max(grid, 1), total % max(grid, 1)};
  int u0 = cta < grid ? share.begin(cta) : 0, u1 = cta < grid ? share.begin(cta + 1) : 0;
  // A few short pairs: a CTA a pair.  Its groups take most tiles at once, and a join between CTAs costs more
  // than a second round (one sequence of 777 keys, 8 KV heads of 128: 14.4 us so, 15.1 cut into as many CTAs as there are places).
  if (most <= 2 * NG + kPairCost && c.n_seqs <= 32 && c.n_seqs * c.hkv <= (int)gridDim.x) w.pair_of(a, cta, lane, &u0, &u1);
  int place = u1;  // of this CTA's first tile
  if (warp > kMma && warp < kMma + 7) place = w.find(a, u0, u1, lane);
  if (threadIdx.x == 0) sh.joins = sh.poison = 0;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  const uint32_t otm = tmem + NG * C::SCOL;  // the groups' O follow their S

  if (u1 > u0 && warp >= kMma) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::RREST));
    if (warp > kMma && warp <= kMma + 2 * NPR) {  // -------------------------------- key tiles, value tiles
      // NPR warps for the keys, as many for the values, each with every NPR-th tile: a tile's copies take
      // one warp some 600 to 1100 cycles to issue.  Lanes 8q .. 8q + 7 look after one of four tiles: its eight
      // groups of 16 keys.  Four tiles' page ids are fetched by one load, while the four before them are issued.
      const bool keys = warp <= kMma + NPR;
      const int odd = NPR == 2 ? (warp - kMma - 1) & 1 : 0;
      const int stages = keys ? C::SK : C::SV;
      uint8_t* slots = keys ? ring : vring;
      uint64_t* full = keys ? sh.kfull : sh.vfull;
      uint64_t* free_ = keys ? sh.kfree : sh.vfree;
      const CUtensorMap* map = keys ? &kmap : &vmap;
      const int P = 1 << c.page_log2, box = min(P, kTile);
      int tok0 = 0, len = 0, head = 0, after = 0, id = -1, flags = 0, ready = 0, set = 0, pairs = 0, in_pair = 0, all0 = 0, all1 = 0;
      bool dead = false, done = place >= u1;
      int s = odd, i = odd, lap = 0;
      if (done && keys && odd == 0) {  // no tile for this CTA
        if (lane == 0) sh.tile[0].after = -1;
        __syncwarp();
        if (lane < 16) mbar_arrive(&full[0]);
      } else if (done && odd == 0) {
        if (lane == 0) sh.value[0].after = -1;
        __syncwarp();
        if (lane < 8) mbar_arrive(&full[0]);
      }
      do {
        const int ctok0 = tok0, clen = len, chead = head, cafter = after, cid = id, cflags = flags, cready = ready, cset = set;
        const int call0 = all0, call1 = all1;
        // the next four tiles (the first time, the first four)
        int b = w.b;
        len = 0;
        ready = 0;
        auto describe = [&](int q) {  // tile q places on, in the pair at hand
          const int k = w.k + q, at = place + q + 1;
          b = w.b, head = w.h, len = w.sq.len, tok0 = w.lo + k * kTile, after = in_pair + q, set = pairs % C::OB;
          // the rows stand at len - rows .. len - 1
          all0 = min(max(max(len - a.window, 0) - tok0, 0), kTile);
          all1 = min(max(len - w.sq.rows + 1 - tok0, 0), kTile);
          flags = all0 > 0 || all1 < kTile ? 2 : 0;
          if (at >= u1 || (k == w.n - 1 && at + kPairCost >= u1)) flags |= 4;
        };
        auto walk = [&](int q) {
          place += q;
          in_pair += q;
          w.k += q;
          if (w.k == w.n) {
            place += kPairCost;
            in_pair = 0;
            ++pairs;
            if (place < u1) w.next_pair(a);
          }
          done = place >= u1;
        };
        if (!done && w.k + 4 * NPR <= w.n && place + 4 * NPR <= u1) {  // all of one pair
          describe(NPR * (lane >> 3) + odd);
          ready = 4;
          walk(4 * NPR);
        } else {
#pragma unroll 1
          for (int q = 0; q < 4 * NPR && !done; ++q) {
            if (q % NPR == odd) {
              if (lane >> 3 == q / NPR) describe(0);
              ++ready;
            }
            walk(1);
          }
        }
        id = -1;
        const int64_t next = (int64_t)tok0 + 16 * (lane & 7);
        if (next < len) id = c.pages[(int64_t)b * c.page_stride + (next >> c.page_log2)];
#pragma unroll 1
        for (int q = 0; q < cready; ++q, i += NPR) {
          if (lap && !wait(&free_[s], (lap - 1) & 1, c.status)) dead = true;
          if (__any_sync(0xFFFFFFFFu, dead)) {
            dead = true;
            break;
          }
          if (lane >> 3 == q) {
            const int gl = lane & 7, tok = ctok0 + 16 * gl;
            bool ok = tok < clen;
            if (ok && (cid < 0 || cid >= c.n_pages)) {
              ok = false;
              atomicMax(c.status, kStatusInvalid);
            }
            const int64_t tile = (int64_t)cid * c.hkv + chead;
            TileMeta& m = sh.tile[i % C::METAS];
            if (keys) {  // written before this lane's arrival, which hands it over
              const bool cut = __any_sync(0xFFu << (8 * q), !ok || tok + 16 > clen);
              if (gl == 0) m.tok0 = ctok0, m.len = clen, m.after = cafter, m.flags = cflags | (cut ? 3 : 0);
              if (!ok) m.ks[gl] = m.vs[gl] = 0.0f;
            } else {
              const uint32_t groups = __ballot_sync(0xFFu << (8 * q), ok) >> (8 * q) & 0xFFu;
              if (gl == 0) {
                ValueMeta& vm = sh.value[i % C::METAS];
                const bool cut = groups != 0xFF || clen - ctok0 < kTile || (cflags & 2);
                vm.after = cafter, vm.rows = min(clen - ctok0, kTile), vm.groups = (int)groups;
                vm.set = cset | (cflags & 4) | (cut ? 8 : 0);
                vm.all0 = call0, vm.all1 = call1;
              }
            }
            if (ok && (16 * gl) % box == 0) {
              uint8_t* dst = slots + s * C::KV + 16 * gl * C::PW;
              mbar_arrive_expect_tx(&full[s], box * D);
#pragma unroll
              for (int x = 0; x < C::NP; ++x)
                tma_load_3d(dst + x * C::PANEL, map, x * 128, tok & (P - 1), (int)tile, &full[s]);
            } else {
              mbar_arrive(&full[s]);
            }
            if (keys) {
              if (ok) {
                cp_async4(&m.ks[gl], c.ks + tile);
                cp_async4(&m.vs[gl], c.vs + tile);
              }
              cp_async_arrive_noinc(&full[s]);
            }
          }
          __syncwarp();
          s += NPR;
          if (s >= stages) s -= stages, ++lap;
        }
      } while (!dead && (ready || !done));
      // no copy is left in flight into this CTA's shared memory when it ends: the last stages filled
#pragma unroll 1
      for (int j = max(odd, i - stages); j < i; j += NPR)
        wait(&full[j % stages], (uint32_t)(j / stages) & 1u, c.status);
    } else if (warp == kMma + 5 || warp == kMma + 6) {  // -------------------------- query rows
      // Two warps; D / 16 lanes a row, 16 elements each; the loads of four rows a lane group are issued together.
      // Rows past R stay as they are: their columns of S are not looked at.
      constexpr int TPR = D / 16, RPP = 32 / TPR;
      const int part = lane % TPR, mine = (warp - kMma - 5) * RPP + lane / TPR;
      bool dead = false;
      if (place >= u1) {  // no pair for this CTA
        if (lane == 0) sh.pair[0].i1 = 0;
        __syncwarp();
        mbar_arrive(&sh.qfull[0]);
      }
      for (int p = 0, i0 = 0; place < u1; ++p) {
        const int qb = p % C::QB;
        const int R = min(w.sq.rows * G, N), first_pos = w.sq.len - w.sq.rows;
        const int i1 = i0 + min(w.n - w.k, u1 - place), next = place + w.n - w.k + kPairCost;
        const int64_t qbase = (int64_t)w.sq.start * a.ldq + (int64_t)w.h * G * a.hsq + 16 * part;
        PairMeta<N>& m = sh.pair[qb];
        uint8_t* qd = qbuf + qb * C::Q;
        bool waited = p < C::QB;
#pragma unroll 1
        for (int r0 = mine; __any_sync(0xFFFFFFFFu, r0 < R); r0 += 8 * RPP) {
          uint4 x[4][2];
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const int row = r0 + 2 * RPP * y, i = row / G, g = row - i * G;
            x[y][0] = x[y][1] = make_uint4(0, 0, 0, 0);
            if (row < R) {
              const uint4* qp = reinterpret_cast<const uint4*>(a.q + qbase + i * a.ldq + g * a.hsq);
              x[y][0] = qp[0];
              x[y][1] = qp[1];
            }
          }
          if (!waited) {
            if (!wait(&sh.qfree[qb], (uint32_t)(p / C::QB - 1) & 1u, c.status)) dead = true;
            waited = true;
          }
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const int row = r0 + 2 * RPP * y;
            if (!__any_sync(0xFFFFFFFFu, row < R)) break;
            float amax = query_max(x[y]);
#pragma unroll
            for (int o = TPR / 2; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
            // a power of two that brings the row's largest element to [128, 256)
            const int e2 = min(max((__float_as_int(amax) >> 23) - 127 - 7, -125), 125);
            uint4 hi, lo;
            split_query<false>(x[y], query_down(amax, e2), &hi, &lo);
            if (row < R) {
              // rows of PW bytes in the swizzle of the key tiles: term, then row (N is a multiple of the swizzle's 8 rows)
              const int panel = part / (C::PW / 16), chunk = part % (C::PW / 16);
              const int at = panel * C::QPANEL + row * C::PW + (D == 64 ? chunk ^ ((row >> 1) & 3) : chunk ^ (row & 7)) * 16;
              *reinterpret_cast<uint4*>(qd + at) = hi;
              *reinterpret_cast<uint4*>(qd + at + N * C::PW) = lo;
              if (part == 0) {
                const int i = row / G, g = row - i * G;
                m.rc[row] = __int_as_float((127 + e2) << 23) * (a.scale * kLog2e);
                m.pos[row] = max(first_pos + i, -1);
                m.off[row] = i * a.ldo + g * a.hso;
              }
            }
          }
        }
        if (!waited && !wait(&sh.qfree[qb], (uint32_t)(p / C::QB - 1) & 1u, c.status)) dead = true;
        if (__any_sync(0xFFFFFFFFu, dead)) break;
        if (warp == kMma + 5 && lane == 0) {
          m.R = R, m.n_tiles = w.n, m.first = place - w.k, m.skipped = w.k;
          m.i0 = i0, m.i1 = i1, m.last = next >= u1;
          m.head = w.h, m.pages = c.pages + (int64_t)w.b * c.page_stride;
          m.base = (int64_t)w.sq.start * a.ldo + (int64_t)w.h * G * a.hso;
        }
        fence_proxy_async_smem();
        mbar_arrive(&sh.qfull[qb]);
        place = next;
        i0 = i1;
        if (place < u1) w.next_pair(a);
      }
    } else if (warp == kMma) {  // ---------------------------------------------------- score MMAs
      // One thread issues them, and its instructions set the pace: descriptors are one add each, and the output
      // MMAs have a warp of their own.
      constexpr uint32_t kSwz = D == 64 ? 4 : 2, kHi = desc_hi(8 * C::PW, kSwz), kQk = idesc_e4m3(2 * N, 0, 0);
      int ks = 0, g = 0, qb = -1;
      uint32_t kpar = 0, spar = 1, qpar = 1;
      const uint32_t k0 = desc_lo(smem_u32(ring), 16), q0 = desc_lo(smem_u32(qbuf), 16);
      bool dead = false, last = false;
#pragma unroll 1
      for (int i = 0; !last && !dead; ++i) {
        dead = !wait(&sh.kfull[ks], kpar, c.status);
        const int after = sh.tile[i % C::METAS].after;
        last = sh.tile[i % C::METAS].flags & 4;
        if (after < 0) break;
        if (!dead && after == 0) {
          if (++qb == C::QB) qb = 0;
          if (qb == 0) qpar ^= 1;
          dead = !wait(&sh.qfull[qb], qpar, c.status);
        }
        if (!dead && i >= NG) dead = !wait(&sh.sfree[g], spar, c.status);
        dead = __any_sync(0xFFFFFFFFu, dead);
        tc_fence_after();
        if (!dead && elect()) {
          const uint32_t ka = k0 + ks * (C::KV / 16), qa = q0 + qb * (C::Q / 16), d = tmem + g * C::SCOL;
#pragma unroll
          for (int x = 0; x < D / 32; ++x) {
            const uint32_t panel = x * 32 / C::PW, off = x * 32 % C::PW;
            mma_e4m3<kHi, kHi, kQk>(d, ka + (panel * C::PANEL + off) / 16, qa + (panel * C::QPANEL + off) / 16, x > 0);
          }
          mma_commit(&sh.sfull[g]);
          mbar_arrive(&sh.sfull[g]);  // passes the tile's description on to the softmax group
          mma_commit(&sh.kfree[ks]);
        }
        __syncwarp();
        if (++ks == C::SK) ks = 0, kpar ^= 1;
        if (++g == NG) g = 0, spar ^= 1;
      }
      // every MMA has ended before the CTA's memory goes
      if (elect()) {
        mma_commit(&sh.ended[0]);
        wait(&sh.ended[0], 0, c.status);
      }
      __syncwarp();
    } else if (warp == kMma + 7) {  // ------------------------------------------------ output MMAs
      // A: V^T, dims contiguous: groups of 8 keys 8 * PW bytes apart; for D = 64 the upper 64 of the
      // 128 rows are the next 8 KB (in the ring or right behind it): lanes that nobody reads.
      // B: P^T, rows contiguous in groups of 16, no swizzle: groups of 8 keys 128 bytes apart
      constexpr uint32_t kHi = desc_hi(8 * C::PW, D == 64 ? 4 : 2), kPHi = desc_hi(kTile * 16, 0);
      constexpr uint32_t kPv = idesc_e4m3(3 * N, 1, 1);
      int vs = 0, g = 0;
      uint32_t vpar = 0, ppar = 0;
      const uint32_t v0 = desc_lo(smem_u32(vring), C::PANEL), p0 = desc_lo(smem_u32(pbuf), 128);
      bool dead = false, last = false;
#pragma unroll 1
      for (int i = 0; !last && !dead; ++i) {
        dead = !wait(&sh.vfull[vs], vpar, c.status);
        dead = __any_sync(0xFFFFFFFFu, dead);
        if (dead) break;
        const ValueMeta m = sh.value[i % C::METAS];
        if (m.after < 0) break;
        last = m.set & 4;
        // rows without a key hold anything, NaN codes too: numbers for P = 0
        if (m.set & 8) {
          uint8_t* vt = vring + vs * C::KV;
          bool found = false;
#pragma unroll 1
          for (int side = 0; side < 2; ++side) {  // keys before and behind those that every row sees
#pragma unroll 1
            for (int e = (side ? m.all1 * (C::PW / 16) : 0) + lane; e < (side ? m.rows : m.all0) * (C::PW / 16); e += 32)
#pragma unroll
              for (int x = 0; x < C::NP; ++x) {
                uint4* at = reinterpret_cast<uint4*>(vt + x * C::PANEL + e * 16);
                *at = drop_nans(*at, &found);
              }
          }
          if (found) sh.poison = 1;
          __syncwarp();
#pragma unroll 1
          for (int gr = 0; gr < 8; ++gr) {  // groups of 16 rows: from row `from` of each on
            const int from = (m.groups >> gr & 1) ? min(max(m.rows - 16 * gr, 0), 16) : 0;
#pragma unroll 4
            for (int e = from * (C::PW / 16) + lane; e < C::PW; e += 32)
#pragma unroll
              for (int x = 0; x < C::NP; ++x)
                *reinterpret_cast<uint4*>(vt + x * C::PANEL + (gr * C::PW + e) * 16) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
          __syncwarp();
        }
        dead = !wait(&sh.pfull[g], ppar, c.status);
        dead = __any_sync(0xFFFFFFFFu, dead);
        tc_fence_after();
        const uint32_t acc = m.after >= NG;  // not the group's first tile of the pair
        if (!dead && elect()) {
          const uint32_t va = v0 + vs * (C::KV / 16), pa = p0 + g * (C::P / 16);
          const uint32_t d = otm + (m.set & 3) * C::OSET + g * (C::MB * C::OCOL);
#pragma unroll
          for (int mb = 0; mb < C::MB; ++mb)
#pragma unroll
            for (int x = 0; x < kTile / 32; ++x)
              mma_e4m3<kHi, kPHi, kPv>(d + mb * C::OCOL, va + (mb * C::PANEL + x * 32 * C::PW) / 16, pa + x * 32, x ? 1u : acc);
          mma_commit(&sh.pvdone[g]);
          mma_commit(&sh.vfree[vs]);
        }
        __syncwarp();
        if (++vs == C::SV) vs = 0, vpar ^= 1;
        if (++g == NG) g = 0, ppar ^= 1;
      }
      if (elect()) {
        mma_commit(&sh.ended[1]);
        wait(&sh.ended[1], 0, c.status);
      }
      __syncwarp();
    }
  } else if (u1 > u0) {  // ------------------------------------------------------------------- softmax, a key a thread
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::RSOFT));
    const int grp = warp >> 2, tid = threadIdx.x & 127, wq = warp & 3;
    const uint32_t lane_base = (uint32_t)(32 * wq) << 16;
    const uint32_t st = tmem + lane_base + grp * C::SCOL;
    float* grow = sh.grow[grp];
    uint8_t* pd = pbuf + grp * C::P + tid * 16;
    bool dead = false;
    bool last = false;
    uint32_t turn = 0;  // tiles of this group so far
    for (int p = 0; !last; ++p) {
      const PairMeta<N>& pm = sh.pair[p % C::QB];
      if (!wait(&sh.qfull[p % C::QB], (uint32_t)(p / C::QB) & 1u, c.status)) dead = true;
      if (any_of(grp, dead)) break;
      const int R = pm.R, i0 = pm.i0, i1 = pm.i1, set = p % C::OB;
      if (i1 == 0) break;
      last = pm.last;
      float* ref = sh.ref[set][grp];
      const uint32_t ot = otm + lane_base + set * C::OSET + grp * (C::MB * C::OCOL);
      float l[N];
#pragma unroll
      for (int r = 0; r < N; ++r) l[r] = 0.0f;
      const int mine = i0 + (grp - i0 % NG + NG) % NG;  // this group's first tile of the pair, if it has one
      for (int i = mine; i < i1; i += NG) {
        const bool first = i == mine;
        const TileMeta& tm = sh.tile[i % C::METAS];
        if (!wait(&sh.sfull[grp], turn & 1, c.status)) dead = true;
        tc_fence_after();
        // the key's scores: both terms of every row
        float x[N];
#pragma unroll
        for (int r = 0; r < N; r += 16) {
          if (r < R) {
            uint32_t u[16], v[16];
            tmem_ld16(st + r, u);
            tmem_ld16(st + N + r, v);
            tmem_ld_wait();
            tmem_arrived(u);
            tmem_arrived(v);
#pragma unroll
            for (int e = 0; e < 16; ++e) x[r + e] = fmaf(__uint_as_float(v[e]), 0x1p-5f, __uint_as_float(u[e]));
          }
        }
        tc_fence_before();
        warp_arrive(&sh.sfree[grp]);
        const float ks = tm.ks[tid >> 4], vs = tm.vs[tid >> 4];
        const float lvs = lg2(vs), ivs = ks == 0.0f ? 0.0f : rcp(vs);
        const int flags = tm.flags, tok = tm.tok0 + tid, most = tm.len;
        // the group's references and outputs are free once the pair that had them before has been joined
        if (first && p >= C::OB && !wait(&sh.joined[set], (uint32_t)(p / C::OB - 1) & 1u, c.status)) dead = true;
        bool over = first;
#pragma unroll
        for (int r = 0; r < N; r += 4) {
          if (r < R) {
            const float4 rc = *reinterpret_cast<const float4*>(&pm.rc[r]);
            const float4 rf = *reinterpret_cast<const float4*>(&ref[r]);
            const float rcs[4] = {rc.x, rc.y, rc.z, rc.w}, rfs[4] = {rf.x, rf.y, rf.z, rf.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              x[r + e] = fmaf(x[r + e], rcs[e] * ks, lvs);
              over |= x[r + e] - rfs[e] > kHead;
            }
          }
        }
        if ((flags & 2) || ks == 0.0f) {  // masks; a page of key scale 0 may lie in any tile
          if (ks == 0.0f && tok <= pm.pos[0] && tok > pm.pos[R - 1] - a.window &&
              !drop_values<D, N>(vring, sh.vfull, i, tid, c.status))
            dead = true;
          const bool hidden = ks == 0.0f || tok >= most;
          over = first;
#pragma unroll
          for (int r = 0; r < N; ++r) {
            if (r < R) {
              const int pos = pm.pos[r];
              if (hidden || tok > pos || tok <= pos - a.window) x[r] = -INFINITY;
              over |= x[r] - ref[r] > kHead;
            }
          }
        }
        if (first || any_of(grp, over || dead)) {
          // some key passes its row's reference, or there is none yet: new references, and what was summed up
          // moves to them (16 x 4 rows of 256: 45.4 us, 49.4 with all rows' outputs multiplied each time)
#pragma unroll
          for (int r = 0; r < N; ++r) {
            if (r < R) {
              const float top = warp_max(x[r]);
              if (lane == 0) sh.red[grp][wq][r] = top;
            }
          }
          if (any_of(grp, dead)) break;
          if (tid >= R && tid < N) ref[tid] = INFINITY;  // not a row: nothing passes it
          if (tid < 32) {
            float moved = 1.0f;
            if (tid < R) {
              const float* red = sh.red[grp][0];
              const float top = fmaxf(fmaxf(red[tid], red[N + tid]), fmaxf(red[2 * N + tid], red[3 * N + tid]));
              const float old = first ? -INFINITY : ref[tid];
              const float now = fmaxf(fmaxf(top, old), kNone);
              ref[tid] = now;
              if (now != old) moved = ex2(old - now);
              grow[tid] = moved;
            }
            const uint32_t rows = __ballot_sync(0xFFFFFFFFu, moved != 1.0f);
            if (tid == 0) sh.moved[grp] = rows;
          }
          any_of(grp, false);
          if (!first) {
            if (!wait(&sh.pvdone[grp], (turn - 1) & 1, c.status)) dead = true;
            if (any_of(grp, dead)) break;
            tc_fence_after();
            const uint32_t rows = sh.moved[grp];
#pragma unroll
            for (int r = 0; r < N; ++r)
              if (r < R) l[r] *= grow[r];
#pragma unroll 1
            for (int r = 0; r < R; r += 4) {  // four rows' outputs at a time, where one of them moves
              if (!(rows >> r & 15)) continue;
              uint32_t u[3 * C::MB][4];
#pragma unroll
              for (int e = 0; e < 3 * C::MB; ++e) tmem_ld4(ot + e * N + r, u[e]);
              const float4 w = *reinterpret_cast<const float4*>(&grow[r]);
              const float ws[4] = {w.x, w.y, w.z, w.w};
              tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 3 * C::MB; ++e) {
                tmem_arrived(u[e]);
#pragma unroll
                for (int z = 0; z < 4; ++z) u[e][z] = __float_as_uint(__uint_as_float(u[e][z]) * (r + z < R ? ws[z] : 0.0f));
                tmem_st4(ot + e * N + r, u[e]);
              }
            }
            tmem_st_wait();
            tc_fence_before();
          }
        }
        // P, its sums and its terms; the buffer is free once the group's tile before has been multiplied
        if (turn && !wait(&sh.pvdone[grp], (turn - 1) & 1, c.status)) dead = true;
#pragma unroll
        for (int r = 0; r < N; r += 16) {
          uint32_t t0[4] = {0, 0, 0, 0}, t1[4] = {0, 0, 0, 0}, t2[4] = {0, 0, 0, 0};
#pragma unroll
          for (int q = 0; q < 16; q += 4) {
            if (r + q < R) {
              const float4 rf = *reinterpret_cast<const float4*>(&ref[r + q]);
              const float rfs[4] = {rf.x, rf.y, rf.z, rf.w};
              float pr[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                pr[e] = r + q + e >= R ? 0.0f : ex2(x[r + q + e] - rfs[e] + kBias);
                l[r + q + e] = fmaf(pr[e], ivs, l[r + q + e]);
              }
#pragma unroll
              for (int z = 0; z < 2; ++z) {
                const uint32_t h = f16x2(pr[2 * z], pr[2 * z + 1]);
                const uint16_t c0 = e4m3x2(h);
                const uint32_t r1 = rest<16>(h, codes_f16x2(c0));  // 256 at most, as half of 448's last place is 16
                const uint16_t c1 = e4m3x2(r1);
                const uint16_t c2 = e4m3x2(rest<32>(r1, codes_f16x2(c1)));  // 256 at most
                t0[q / 4] |= (uint32_t)c0 << (16 * z);
                t1[q / 4] |= (uint32_t)c1 << (16 * z);
                t2[q / 4] |= (uint32_t)c2 << (16 * z);
              }
            }
          }
          // N-contiguous groups of 16 columns, a key's 16 bytes after the other's
          *reinterpret_cast<uint4*>(pd + (r / 16) * (kTile * 16)) = make_uint4(t0[0], t0[1], t0[2], t0[3]);
          *reinterpret_cast<uint4*>(pd + ((N + r) / 16) * (kTile * 16)) = make_uint4(t1[0], t1[1], t1[2], t1[3]);
          *reinterpret_cast<uint4*>(pd + ((2 * N + r) / 16) * (kTile * 16)) = make_uint4(t2[0], t2[1], t2[2], t2[3]);
        }
        fence_proxy_async_smem();
        tc_fence_before();
        warp_arrive(&sh.pfull[grp]);
        ++turn;
      }
      // the pair's end here: the group's sums, then all groups' outputs by the one that had the last tile
      const bool took = mine < i1;
      if (took) {
        if (!wait(&sh.pvdone[grp], (turn - 1) & 1, c.status)) dead = true;
        // rows' sums over the group's threads, by way of P's buffer, which nothing reads any more
        float* lp = reinterpret_cast<float*>(pbuf + grp * C::P);
#pragma unroll
        for (int r = 0; r < N; ++r) {
          if (r < R) {
            const float v = l[r] + __shfl_xor_sync(0xFFFFFFFFu, l[r], 16);
            if (lane < 16) lp[r * 64 + wq * 16 + lane] = v;
          }
        }
        if (any_of(grp, dead)) break;
#pragma unroll 1
        for (int r = wq; r < R; r += 4) {
          float v = lp[r * 64 + lane] + lp[r * 64 + 32 + lane];
#pragma unroll
          for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
          if (lane == 0) {
            sh.sum[set][grp][r] = v;
            if (v != v) ref[r] = INFINITY;  // a NaN outweighs the other groups and parts
          }
        }
        any_of(grp, false);
      }
      // A group without a tile of this pair waits for that join all the same: nobody is OB pairs
      // ahead of a join, so no phase of the two barriers below is missed or arrived at twice.
      if (!took) {
        if (p >= C::OB && !wait(&sh.joined[set], (uint32_t)(p / C::OB - 1) & 1u, c.status)) dead = true;
        if (any_of(grp, dead)) break;
      }
      const bool join = (i1 - 1) % NG == grp;
      if (tid == 0) mbar_arrive(&sh.summed[set]);
      if (join) {
        if (!wait(&sh.summed[set], (uint32_t)(p / C::OB) & 1u, c.status)) dead = true;
        if (any_of(grp, dead)) break;
        tc_fence_after();
        const int first_tile = pm.first;
        const int64_t base = pm.base;
        const int n_tiles = pm.n_tiles, parts_here = min(NG, i1 - i0);
        const bool whole = pm.skipped == 0 && i1 - i0 == n_tiles;
        const int slot = 2 * cta + (i0 == 0 ? 0 : 1);
        // row's factors of the groups (below 0 without a tile of this pair), and its reference and sum
        if (tid < R) {
          float top = -INFINITY, sum = 0.0f, m[NG];
#pragma unroll
          for (int gq = 0; gq < NG; ++gq) {
            const int q = gq - i0 % NG;
            m[gq] = (q < 0 ? q + NG : q) < parts_here ? sh.ref[set][gq][tid] : -INFINITY;
            top = fmaxf(top, m[gq]);
          }
#pragma unroll
          for (int gq = 0; gq < NG; ++gq) {
            const bool none = m[gq] == -INFINITY;
            const float f = none ? -1.0f : ex2(m[gq] - top);
            if (!none && f != 0.0f) sum = fmaf(sh.sum[set][gq][tid], f, sum);
            sh.factor[gq][tid] = f;
          }
          if (whole)
            sh.inv[tid] = sum == 0.0f ? 0.0f : 1.0f / sum;
          else
            da.part_ml[slot * N + tid] = make_float2(top, sum);
        }
        any_of(grp, false);
#pragma unroll 1
        for (int e = 0; e < C::MB * ((R + 3) / 4); ++e) {  // blocks of 128 dims x 4 rows
          const int mb = C::MB == 1 ? 0 : e & 1, r = C::MB == 1 ? 4 * e : (e >> 1) * 4, d = mb * 128 + tid;
          uint32_t v[NG][3][4];
#pragma unroll
          for (int gq = 0; gq < NG; ++gq)
#pragma unroll
            for (int t = 0; t < 3; ++t) tmem_ld4(otm + lane_base + set * C::OSET + (gq * C::MB + mb) * C::OCOL + t * N + r, v[gq][t]);
          tmem_ld_wait();
#pragma unroll
          for (int gq = 0; gq < NG; ++gq)
#pragma unroll
            for (int t = 0; t < 3; ++t) tmem_arrived(v[gq][t]);
          float o[4] = {0, 0, 0, 0};
#pragma unroll
          for (int gq = 0; gq < NG; ++gq) {
            const float4 f4 = *reinterpret_cast<const float4*>(&sh.factor[gq][r]);
            const float f[4] = {f4.x, f4.y, f4.z, f4.w};
#pragma unroll
            for (int z = 0; z < 4; ++z) {
              const float y = fmaf(__uint_as_float(v[gq][2][z]), 0x1p-9f,
                                   fmaf(__uint_as_float(v[gq][1][z]), 0x1p-4f, __uint_as_float(v[gq][0][z])));
              if (!(f[z] < 0.0f)) o[z] = fmaf(y, f[z], o[z]);  // a group without a tile of this pair holds anything
            }
          }
          if (d < D) {
            if (sh.poison) {
              const int last = pm.pos[R - 1], all0 = last - a.window + 1;
#pragma unroll
              for (int z = 0; z < 4; ++z)
                if (r + z < R && nan_dims(c, pm.pages, pm.head, D, d & ~15, pm.pos[r + z], a.window, all0, pm.pos[0]) >> (d & 15) & 1)
                  o[z] = __int_as_float(0x7FFFFFFF);
            }
#pragma unroll
            for (int z = 0; z < 4; ++z) {
              if (r + z < R) {
                if (whole) {
                  const __nv_bfloat16 y = __float2bfloat16_rn(o[z] * sh.inv[r + z]);
                  a.out[base + pm.off[r + z] + d] = *reinterpret_cast<const uint16_t*>(&y);
                } else {
                  da.part_o[((int64_t)slot * N + r + z) * D + d] = o[z];
                }
              }
            }
          }
        }
        tc_fence_before();
        any_of(grp, false);
        // the other groups may go on with the next pair, and the query buffer is free
        if (tid == 0) {
          mbar_arrive(&sh.qfree[p % C::QB]);
          mbar_arrive(&sh.joined[set]);
        }
        if (!whole) {
          // the CTA whose ticket completes the pair joins its parts, when all its own work is done
          any_of(grp, false);
          const int c0 = share.owner(first_tile), parts = share.owner(first_tile + n_tiles - 1) - c0 + 1;
          if (tid == 0 && ticket_add(da.counters + c0, 1) == parts - 1) {
            da.counters[c0] = 0;
            const int at = atomicAdd(&sh.joins, 1);
            sh.join[at][0] = R, sh.join[at][1] = c0, sh.join[at][2] = parts;
            sh.join[at][3] = first_tile - share.begin(c0) <= kPairCost;
            sh.join_base[at] = base;
          }
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMma) tmem_dealloc(tmem, 512);
  uint32_t phase = 0;
  for (int j = 0; j < sh.joins && warp < kMma; ++j)
    join_parts<D, N>(da, sh.join[j][0], G, sh.join_base[j], sh.join[j][1], sh.join[j][2], sh.join[j][3], ring, &sh.joinbar, &phase);
}

template <int D, int N>
int launch(const DecodeArgs& da, const CUtensorMap& km, const CUtensorMap& vm, int grid, cudaStream_t s) {
  using C = Cfg<D, N>;
  static std::atomic<unsigned long long> configured{0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return QG_ERR_CUDA;
  const unsigned long long bit = 1ull << (dev & 63);
  if (!(configured.load() & bit)) {
    if (cudaFuncSetAttribute((const void*)attn_decode_kernel<D, N>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             C::SMEM) != cudaSuccess)
      return QG_ERR_CUDA;
    configured.fetch_or(bit);
  }
  return launch_pdl(attn_decode_kernel<D, N>, dim3(grid), dim3(C::THREADS), C::SMEM, s, km, vm, da) == cudaSuccess
             ? QG_OK
             : QG_ERR_CUDA;
}

template <int D>
int launch_rows(int rows, const DecodeArgs& da, const CUtensorMap& km, const CUtensorMap& vm, int grid, cudaStream_t s) {
  if (rows == 16) return launch<D, 16>(da, km, vm, grid, s);
  return launch<D, 32>(da, km, vm, grid, s);
}

}  // namespace

int decode_rows(int64_t rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : 0; }

size_t decode_workspace(int64_t rows, int head_dim, const DeviceInfo& dev) {
  const size_t r = (size_t)decode_rows(rows), slots = 2 * (size_t)dev.sms;
  return kWsHeader + kAttnCounterBytes + slots * r * sizeof(float2) + slots * r * head_dim * sizeof(float);
}

int launch_attn_decode(const AttnArgs& a, int head_dim, int64_t rows, const DeviceInfo& dev, void* ws, void* stream) {
  if (dev.sms * sizeof(int) > kAttnCounterBytes) return QG_ERR_UNSUPPORTED;
  const int page = 1 << a.c.page_log2, box = std::min(page, kTile);
  CUtensorMap km, vm;
  if (!encode_pages(&km, a.c.k, head_dim, page, a.c.n_pages * a.c.hkv, box) ||
      !encode_pages(&vm, a.c.v, head_dim, page, a.c.n_pages * a.c.hkv, box))
    return QG_ERR_CUDA;
  const int r = decode_rows(rows);
  DecodeArgs da;
  da.a = a;
  uint8_t* w = static_cast<uint8_t*>(ws) + kWsHeader;
  da.counters = reinterpret_cast<int*>(w);
  w += kAttnCounterBytes;
  da.part_ml = reinterpret_cast<float2*>(w);
  da.part_o = reinterpret_cast<float*>(w + 2 * (size_t)dev.sms * r * sizeof(float2));
  // no more CTAs than tiles that there can be
  const int64_t pairs = (int64_t)a.c.n_seqs * a.c.hkv, most = pairs * ((a.c.max_len + kTile - 1) / kTile);
  if (most + kPairCost * pairs > 0x7FFFFFFF) return QG_ERR_UNSUPPORTED;  // the line's places are 32-bit
  const int grid = (int)std::min<int64_t>(std::min(dev.sms, kMostCtas), most);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  switch (head_dim) {
    case 64: return launch_rows<64>(r, da, km, vm, grid, s);
    case 128: return launch_rows<128>(r, da, km, vm, grid, s);
    case 256: return launch_rows<256>(r, da, km, vm, grid, s);
  }
  return QG_ERR_UNSUPPORTED;
}

}  // namespace qg
