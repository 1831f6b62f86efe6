// Attention of a few rows a KV head over the 8-bit paged cache (decode, speculative
// verification): the R = new * G query rows of one (sequence, KV head) pair, at most 64, against
// all its keys.
//
// The mathematics.  With codes k, v, page scales ks, vs and s_j = scale * ks_j * (q . k_j) * log2(e), each
// row keeps t_j = s_j + log2(vs_j), a reference m near their maximum and P_j = 2^(t_j - m + 2):
//   out = sum_j P_j v_j / sum_j P_j / vs_j.
// The value scale sits in the exponent, so P is rounded relative to the largest contribution
// whatever the scales' spread.  m need not be the maximum: it moves only when some t_j passes it by
// 6.5, so no tile but the first few reduces anything over its keys.
//
// Bound by HBM: each key and value code is used for R rows only.  So nothing converts them: both
// products run on the E4M3 tensor cores with the codes as they lie in the cache, and the 16-bit side
// is split into E4M3 terms instead, which is little work for few rows:
//   scores   S^T[key][row]  = K[128 keys x D]   * Q^T      (A: the key tile, B: the rows, N = 2 terms x rows)
//   outputs  O^T[dim][row] += V^T[D x 128 keys] * P^T      (A: the value tile read transposed, N = 3 terms x rows)
// A query row over a power of two is the sum of two E4M3 terms (bf16 has 8 significant bits, a term 4
// and a sign; exact but for elements 2^-9 below the row's largest, off by 2^-18 of it at most).  P, rounded to
// fp16's 11 bits, is the sum of three, the second and third scaled up by 2^4 and 2^8; each term has its own
// accumulator columns, so the scaling comes out at the end.  Keys as the M dimension fill it whatever R
// is.  Accumulation and statistics are fp32.
//
//   * The pairs' keys, in tiles of 128, lie on one line, which the CTAs (one an SM) share out evenly
//     whatever the lengths; a pair cut between CTAs leaves partial (m, l, O) rows in the workspace, and the
//     CTA that finishes last adds them in order.  One launch.
//   * warp 5 copies tiles into a ring by TMA, warps 6-7 bring a pair's query rows, warp 4 issues the MMAs, and
//     warps 0-3 turn S into P, a key a thread: its column of R scores comes from tensor memory, its terms
//     go to shared memory as 16-byte rows.  The sums of P stay per thread until the pair ends.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>

#include "qg_attn.h"
#include "qg_sync.cuh"
#include "qg_tc.cuh"

namespace qg {
namespace {

constexpr int kThreads = 256;
constexpr int kTile = 128;           // keys a tile
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kBias = 2.0f;        // P of a key at the reference is 2^2 ...
constexpr float kHead = 6.5f;        // ... and at most 2^8.5, below E4M3's 448

// D: head dimension; N: rows it is built for (16, 32, 64).
template <int D, int N>
struct Cfg {
  static constexpr int PW = D < 128 ? D : 128;       // bytes of a panel row (a TMA box row)
  static constexpr int NP = D / PW;                  // panels
  static constexpr int PANEL = kTile * PW;
  static constexpr int KV = kTile * D;               // bytes of a key (or value) tile
  static constexpr int Q = 2 * N * D;                // both terms of the query rows
  static constexpr int QPANEL = 2 * N * PW;
  static constexpr int P = 3 * N * kTile;
  static constexpr bool BIG = D == 256 && N == 64;   // tensor and shared memory for one buffer of S, Q and P
  static constexpr int B = BIG ? 1 : 2;
  static constexpr int MB = NP;                      // M blocks of O (128 dims; D = 64 fills half of one)
  static constexpr int SCOL = 2 * N, OCOL = 3 * N;   // TMEM columns of an S buffer and of a block of O
  static constexpr int STAGE = 2 * KV;
  static constexpr int FIXED = 1024 + B * (Q + P) + 8192;
  static constexpr int S0 = (232448 - FIXED) / STAGE;
  static constexpr int S = S0 > 8 ? 8 : S0;
  static constexpr int SMEM = FIXED + S * STAGE;
  static_assert(S >= 2 && B * SCOL + MB * OCOL <= 512, "shared and tensor memory");
};

// What a stage holds.
struct TileMeta {
  int first, last;      // of its pair in this CTA
  int tok0, len;
  int cut, pad[3];      // cut: some of its rows hold no key
  float ks[8], vs[8];   // scales of its groups of 16 keys; 0: the group holds no key
};
// What a query buffer holds besides the rows.
struct PairMeta {
  int R, len, h, start;
  int n_tiles, low, high, pad;  // low, high: least and largest position of its rows
  int64_t first;                // the pair's first tile on the line
  int64_t pad2;
  float rc[64];                 // the row's power of two * scale * log2(e)
  int pos[64];
};
template <int D, int N>
struct Shared {
  using C = Cfg<D, N>;
  TileMeta tile[C::S];
  PairMeta pair[C::B];
  alignas(16) float ref[64];
  float grow[64];
  float red[4][64];
  uint64_t kfull[C::S], vfull[C::S], empty[C::S];
  uint64_t qfull[C::B], qfree[C::B], sfull[C::B], sfree[C::B], pfull[C::B], pvdone[C::B], ended;
  uint32_t tmem;
  int ticket;
};

struct DecodeArgs {
  AttnArgs a;
  int* counters;   // one a CTA: the parts of the pair that begins in it and ends in another
  float2* part_ml; // [2 * grid][N]
  float* part_o;   // [2 * grid][N][D]
};

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
// 16 * (h - c) of two fp16 pairs: exact where c is h rounded to fewer bits
__device__ __forceinline__ uint32_t rest16(uint32_t h, uint32_t c) {
  uint32_t d, r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(h), "r"(c));
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(d), "r"(0x4C004C00u));
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

// Shared-memory matrix descriptor (version 1): start, leading and stride byte offsets, swizzle
// (0 none, 2 128 bytes, 4 64 bytes).
__device__ __forceinline__ uint64_t mat_desc(uint32_t addr, uint32_t lbo, uint32_t sbo, uint32_t swizzle) {
  return (uint64_t)((addr & 0x3FFFFu) >> 4) | (uint64_t)(lbo >> 4) << 16 | (uint64_t)(sbo >> 4) << 32 |
         (uint64_t)1 << 46 | (uint64_t)swizzle << 61;
}
// kind::f8f6f4, E4M3 x E4M3 -> fp32, M = 128; ta, tb: A, B lie M- or N-contiguous.
__host__ __device__ constexpr uint32_t idesc_e4m3(int n, int ta, int tb) {
  return (1u << 4) | ((uint32_t)ta << 15) | ((uint32_t)tb << 16) | ((uint32_t)(n >> 3) << 17) | (8u << 24);
}
__device__ __forceinline__ void mma_e4m3(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc),
      "r"((uint32_t)acc)
      : "memory");
}
// Barrier of the four softmax warps that returns whether any thread's v is set.
__device__ __forceinline__ bool any_of_128(bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\tbarrier.cta.red.or.pred q, 1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)v)
      : "memory");
  return r != 0;
}

// First key that any row of the sequence sees, rounded down to a page; tiles of a pair (one at least where
// there are rows, so that rows without a key are written).
__device__ __forceinline__ int first_key(const Seq& s, const AttnArgs& a) {
  const int64_t p = (int64_t)s.len - s.rows + 1 - a.window;
  return a.window && p > 0 ? ((int)min(p, (int64_t)s.len) >> a.c.page_log2) << a.c.page_log2 : 0;
}
__device__ __forceinline__ int tiles_of(const Seq& s, const AttnArgs& a) {
  return s.rows > 0 ? max(1, (s.len - first_key(s, a) + kTile - 1) / kTile) : 0;
}

// A place on the line: tile k of head h of sequence b, whose pairs have n tiles.  A whole warp walks.
struct Walk {
  int b, h, k, n, lo;
  Seq sq;

  __device__ __forceinline__ void find(const AttnArgs& a, int64_t unit, int lane) {
    const KvArgs& c = a.c;
    int64_t left = unit;
    bool ignore = false;
    b = 0, n = 1;
    sq = {0, 0, 0};
    for (int base = 0; base < c.n_seqs; base += 32) {
      Seq t = {0, 0, 0};
      if (base + lane < c.n_seqs) t = seq_of(c, base + lane, &ignore);
      const int un = tiles_of(t, a);
      int64_t sum = (int64_t)un * c.hkv;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xFFFFFFFFu, sum, o);
        if (lane >= o) sum += v;
      }
      const int64_t all = __shfl_sync(0xFFFFFFFFu, sum, 31);
      if (left < all) {
        const int who = __ffs(__ballot_sync(0xFFFFFFFFu, sum > left)) - 1;
        b = base + who;
        n = __shfl_sync(0xFFFFFFFFu, un, who);
        left -= __shfl_sync(0xFFFFFFFFu, sum, who) - (int64_t)n * c.hkv;
        sq.start = __shfl_sync(0xFFFFFFFFu, t.start, who);
        sq.rows = __shfl_sync(0xFFFFFFFFu, t.rows, who);
        sq.len = __shfl_sync(0xFFFFFFFFu, t.len, who);
        break;
      }
      left -= all;
    }
    h = (int)(left / n);
    k = (int)(left - (int64_t)h * n);
    lo = first_key(sq, a);
  }
  // the next pair; there is one
  __device__ __forceinline__ void next_pair(const AttnArgs& a) {
    k = 0;
    if (++h == a.c.hkv) {
      bool ignore = false;
      h = 0;
      do {
        ++b;
        sq = seq_of(a.c, b, &ignore);
        n = tiles_of(sq, a);
      } while (n == 0);
      lo = first_key(sq, a);
    }
  }
};

template <int D, int N>
__global__ void __launch_bounds__(kThreads, 1)
    attn_decode_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                       const DecodeArgs da) {
  using C = Cfg<D, N>;
  static_assert(sizeof(Shared<D, N>) <= 8192, "shared memory");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* qbuf = ring + C::S * C::STAGE;
  uint8_t* pbuf = qbuf + C::B * C::Q;
  Shared<D, N>& sh = *reinterpret_cast<Shared<D, N>*>(pbuf + C::B * C::P);
  const AttnArgs& a = da.a;
  const KvArgs& c = a.c;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = a.hq / c.hkv;

  if (tid == 0) {
    for (int s = 0; s < C::S; ++s) {
      mbar_init(&sh.kfull[s], 16);
      mbar_init(&sh.vfull[s], 8);
      mbar_init(&sh.empty[s], 1);
    }
    for (int i = 0; i < C::B; ++i) {
      mbar_init(&sh.qfull[i], 64);
      mbar_init(&sh.qfree[i], 1);
      mbar_init(&sh.sfull[i], 1);
      mbar_init(&sh.sfree[i], 128);
      mbar_init(&sh.pfull[i], 128);
      mbar_init(&sh.pvdone[i], 1);
    }
    mbar_init(&sh.ended, 1);
    fence_mbar_init();
  }
  if (warp == 4) {
    tmem_alloc(&sh.tmem, 512);
    tmem_relinquish();
  }
  pdl_wait();
  // the line: tiles of all sequences, each counted once (all its KV heads have as many)
  int64_t total = 0;
  bool bad = false;
  for (int base = 0; base < c.n_seqs; base += 32) {
    int n = 0;
    if (base + lane < c.n_seqs) n = tiles_of(seq_of(c, base + lane, &bad), a);
    total += __reduce_add_sync(0xFFFFFFFFu, n);
  }
  if (bad && warp == 0 && blockIdx.x == 0) atomicExch(c.status, kStatusInvalid);
  total *= c.hkv;
  // with no more CTAs than tiles, each has one at least
  const int64_t grid = min((int64_t)gridDim.x, total), cta = blockIdx.x;
  const int64_t u0 = cta < grid ? cta * total / grid : 0, u1 = cta < grid ? (cta + 1) * total / grid : 0;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  const int n = (int)(u1 - u0);
  const uint32_t otm = tmem + C::B * C::SCOL;

  if (n > 0 && warp == 5) {  // ------------------------------------------------------------ key and value tiles
    Walk w;
    w.find(a, u0, lane);
    const int P = 1 << c.page_log2, box = min(P, kTile);
    // this lane's group of 16 keys: its page id (-1: no such keys)
    auto page_of = [&]() {
      const int64_t tok = (int64_t)w.lo + (int64_t)w.k * kTile + 16 * lane;
      return lane < 8 && tok < w.sq.len ? c.pages[(int64_t)w.b * c.page_stride + (tok >> c.page_log2)] : -1;
    };
    int id = page_of();
    bool dead = false;
    int s = 0;
    uint32_t lap = 0;
    int i = 0;
    for (; i < n; ++i) {
      // this tile's data, and the next one's page id on its way
      const int tok0 = w.lo + w.k * kTile, head = w.h, cid = id, len = w.sq.len;
      const bool first = w.k == 0 || i == 0, last = w.k == w.n - 1 || i == n - 1;
      if (i + 1 < n) {
        if (++w.k == w.n) w.next_pair(a);
        id = page_of();
      }
      if (lap && !mbar_wait_bounded(&sh.empty[s], (lap - 1) & 1, c.status)) dead = true;
      if (__any_sync(0xFFFFFFFFu, dead)) break;
      TileMeta& m = sh.tile[s];
      const int tok = tok0 + 16 * lane;
      bool ok = lane < 8 && tok < len;
      if (ok && (cid < 0 || cid >= c.n_pages)) {
        ok = false;
        atomicExch(c.status, kStatusInvalid);
      }
      const bool cut = __any_sync(0xFFFFFFFFu, lane < 8 && (!ok || tok + 16 > len));
      if (lane == 0) {
        m.first = first, m.last = last, m.tok0 = tok0, m.len = len, m.cut = cut;
      }
      if (lane < 8) {
        uint8_t* kd = ring + s * C::STAGE + 16 * lane * C::PW;
        const int64_t tile = (int64_t)cid * c.hkv + head;
        const bool lead = ok && (16 * lane) % box == 0;
        if (ok) {
          cp_async4(&m.ks[lane], c.ks + tile);
          cp_async4(&m.vs[lane], c.vs + tile);
        } else {
          m.ks[lane] = 0.0f;
          m.vs[lane] = 0.0f;
        }
        if (lead) {
          mbar_arrive_expect_tx(&sh.kfull[s], box * D);
          mbar_arrive_expect_tx(&sh.vfull[s], box * D);
#pragma unroll
          for (int x = 0; x < C::NP; ++x)
            tma_load_3d(kd + x * C::PANEL, &kmap, x * 128, tok & (P - 1), (int)tile, &sh.kfull[s]);
#pragma unroll
          for (int x = 0; x < C::NP; ++x)
            tma_load_3d(kd + C::KV + x * C::PANEL, &vmap, x * 128, tok & (P - 1), (int)tile, &sh.vfull[s]);
        } else {
          mbar_arrive(&sh.kfull[s]);
          mbar_arrive(&sh.vfull[s]);
        }
        cp_async_arrive_noinc(&sh.kfull[s]);
      }
      __syncwarp();
      if (++s == C::S) s = 0, ++lap;
    }
    // no copy is left in flight into this CTA's shared memory when it ends: the last stages filled
    for (int j = max(0, i - C::S); j < i; ++j) {
      mbar_wait_bounded(&sh.kfull[j % C::S], (uint32_t)(j / C::S) & 1u, c.status);
      mbar_wait_bounded(&sh.vfull[j % C::S], (uint32_t)(j / C::S) & 1u, c.status);
    }
  } else if (n > 0 && warp >= 6) {  // ------------------------------------------------------ query rows
    // 64 threads: D / 16 of them a row, 16 elements each
    constexpr int TPR = D / 16, RPP = 64 / TPR;
    const int t = tid - 192, part = t % TPR;
    Walk w;
    w.find(a, u0, lane);
    int64_t u = u0;
    bool dead = false;
    for (int p = 0; u < u1; ++p) {
      const int qb = p % C::B;
      if (p >= C::B && !mbar_wait_bounded(&sh.qfree[qb], (uint32_t)(p / C::B - 1) & 1u, c.status)) dead = true;
      if (__any_sync(0xFFFFFFFFu, dead)) break;
      PairMeta& m = sh.pair[qb];
      const int R = min(w.sq.rows * G, N), first_pos = w.sq.len - w.sq.rows;
      if (t == 0) {
        m.R = R, m.len = w.sq.len, m.h = w.h, m.start = w.sq.start, m.n_tiles = w.n;
        m.low = first_pos, m.high = w.sq.len - 1, m.first = u - w.k;
      }
      uint8_t* qd = qbuf + qb * C::Q;
      for (int r0 = 0; r0 < N; r0 += RPP) {
        const int row = r0 + t / TPR;
        const bool in = row < R;
        const int i = in ? row / G : 0, g = in ? row - i * G : 0;
        uint4 x[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
        if (in) {
          const uint4* qp = reinterpret_cast<const uint4*>(a.q + (int64_t)(w.sq.start + i) * a.ldq +
                                                           (int64_t)(w.h * G + g) * a.hsq + 16 * part);
          x[0] = qp[0];
          x[1] = qp[1];
        }
        const uint32_t v[8] = {x[0].x, x[0].y, x[0].z, x[0].w, x[1].x, x[1].y, x[1].z, x[1].w};
        float amax = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e)
          amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(v[e] << 16)), fabsf(__uint_as_float(v[e] & 0xFFFF0000u))));
#pragma unroll
        for (int o = TPR / 2; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
        // a power of two that brings the row's largest element to [128, 256)
        const int e2 = min(max((__float_as_int(amax) >> 23) - 127 - 7, -125), 125);
        const float down = __int_as_float((127 - e2) << 23);
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint16_t hh[2], ll[2];
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            const uint32_t y = v[2 * e + z];
            // bf16's bits fit fp16 at this size but for the smallest elements
            const uint32_t h16 = f16x2(__uint_as_float(y << 16) * down, __uint_as_float(y & 0xFFFF0000u) * down);
            hh[z] = e4m3x2(h16);
            uint32_t d16;
            asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d16) : "r"(h16), "r"(codes_f16x2(hh[z])));
            ll[z] = e4m3x2(d16);
          }
          hi[e] = hh[0] | (uint32_t)hh[1] << 16;
          lo[e] = ll[0] | (uint32_t)ll[1] << 16;
        }
        // rows of PW bytes in the swizzle of the key tiles: term, then row
        const int panel = part / (C::PW / 16), chunk = part % (C::PW / 16);
        const int rh = row, rl = N + row;
        const int ch = D == 64 ? chunk ^ ((rh >> 1) & 3) : chunk ^ (rh & 7);
        const int cl = D == 64 ? chunk ^ ((rl >> 1) & 3) : chunk ^ (rl & 7);
        if (row < N) {
          *reinterpret_cast<uint4*>(qd + panel * C::QPANEL + rh * C::PW + ch * 16) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          *reinterpret_cast<uint4*>(qd + panel * C::QPANEL + rl * C::PW + cl * 16) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
          if (part == 0) {
            m.rc[row] = __int_as_float((127 + e2) << 23) * (a.scale * kLog2e);
            m.pos[row] = in ? first_pos + i : -1;
          }
        }
      }
      fence_proxy_async_smem();
      mbar_arrive(&sh.qfull[qb]);
      u += w.n - w.k;
      if (u < u1) w.next_pair(a);
    }
  } else if (n > 0 && warp == 4) {  // ------------------------------------------------------ MMAs
    constexpr uint32_t kSwz = D == 64 ? 4 : 2;
    constexpr uint32_t kSbo = 8 * C::PW;
    constexpr uint32_t kQk = idesc_e4m3(2 * N, 0, 0), kPv = idesc_e4m3(3 * N, 1, 1);
    int p = -1;  // pairs begun by the score MMAs
    auto scores = [&](int i) {
      const int s = i % C::S, sb = i % C::B;
      if (!mbar_wait_bounded(&sh.kfull[s], (uint32_t)(i / C::S) & 1u, c.status)) return false;
      if (sh.tile[s].first) {
        ++p;
        if (!mbar_wait_bounded(&sh.qfull[p % C::B], (uint32_t)(p / C::B) & 1u, c.status)) return false;
      }
      if (i >= C::B && !mbar_wait_bounded(&sh.sfree[sb], (uint32_t)(i / C::B - 1) & 1u, c.status)) return false;
      tc_fence_after();
      if (lane == 0) {
        const uint32_t ka = smem_u32(ring + s * C::STAGE), qa = smem_u32(qbuf + (p % C::B) * C::Q);
#pragma unroll
        for (int x = 0; x < D / 32; ++x) {
          const uint32_t panel = x * 32 / C::PW, off = x * 32 % C::PW;
          mma_e4m3(tmem + sb * C::SCOL, mat_desc(ka + panel * C::PANEL + off, 16, kSbo, kSwz),
                   mat_desc(qa + panel * C::QPANEL + off, 16, kSbo, kSwz), kQk, x > 0);
        }
        mma_commit(&sh.sfull[sb]);
      }
      __syncwarp();
      return true;
    };
    auto outputs = [&](int i) {
      const int s = i % C::S, pb = i % C::B;
      if (!mbar_wait_bounded(&sh.vfull[s], (uint32_t)(i / C::S) & 1u, c.status)) return false;
      const TileMeta& m = sh.tile[s];
      uint8_t* vt = ring + s * C::STAGE + C::KV;
      if (m.cut) {  // rows without a key hold anything, NaN codes too: they must be numbers for P = 0
        for (int r = lane; r < kTile; r += 32) {
          if (m.tok0 + r >= m.len || m.ks[r >> 4] == 0.0f) {
#pragma unroll 1
            for (int x = 0; x < C::NP; ++x)
#pragma unroll
              for (int b = 0; b < C::PW; b += 16)
                *reinterpret_cast<uint4*>(vt + x * C::PANEL + r * C::PW + b) = make_uint4(0, 0, 0, 0);
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
      }
      if (!mbar_wait_bounded(&sh.pfull[pb], (uint32_t)(i / C::B) & 1u, c.status)) return false;
      tc_fence_after();
      if (lane == 0) {
        const uint32_t va = smem_u32(vt), pa = smem_u32(pbuf + pb * C::P);
        const bool first = m.first;
#pragma unroll
        for (int mb = 0; mb < C::MB; ++mb)
#pragma unroll
          for (int x = 0; x < kTile / 32; ++x) {
            // A: V^T, dims contiguous: groups of 8 keys 8 * PW bytes apart; for D = 64 the upper 64 of the
            // 128 rows are the next 8 KB (in the ring or right behind it): lanes that nobody reads.
            // B: P^T, rows contiguous in groups of 16, no swizzle: groups of 8 keys 128 bytes apart
            mma_e4m3(otm + mb * C::OCOL, mat_desc(va + mb * C::PANEL + x * 32 * C::PW, C::PANEL, kSbo, kSwz),
                     mat_desc(pa + x * 32 * 16, 128, kTile * 16, 0), kPv, !(first && x == 0));
          }
        mma_commit(&sh.pvdone[pb]);
        mma_commit(&sh.empty[s]);
      }
      __syncwarp();
      return true;
    };
    bool go = scores(0);
    for (int i = 0; i < n && go; ++i) go = (i + 1 == n || scores(i + 1)) && outputs(i);
    // every MMA has ended before the CTA's memory goes
    if (lane == 0) {
      mma_commit(&sh.ended);
      mbar_wait_bounded(&sh.ended, 0, c.status);
    }
    __syncwarp();
  } else if (n > 0 && warp < 4) {  // ------------------------------------------------------- softmax, a key a thread
    const uint32_t lane_base = (uint32_t)(32 * warp) << 16;
    float l[N];
    int p = -1;
    bool dead = false;
    for (int i = 0; i < n; ++i) {
      const int s = i % C::S, sb = i % C::B;
      if (!mbar_wait_bounded(&sh.kfull[s], (uint32_t)(i / C::S) & 1u, c.status)) dead = true;
      const TileMeta& tm = sh.tile[s];
      const bool first = tm.first, last = tm.last;
      if (first && !dead) {
        ++p;
        if (!mbar_wait_bounded(&sh.qfull[p % C::B], (uint32_t)(p / C::B) & 1u, c.status)) dead = true;
#pragma unroll
        for (int r = 0; r < N; ++r) l[r] = 0.0f;
      }
      const PairMeta& pm = sh.pair[max(p, 0) % C::B];
      const int R = pm.R;
      if (!dead && !mbar_wait_bounded(&sh.sfull[sb], (uint32_t)(i / C::B) & 1u, c.status)) dead = true;
      tc_fence_after();
      // the key's scores: both terms of every row
      float x[N];
#pragma unroll
      for (int r = 0; r < N; r += 16) {
        if (r < R) {
          uint32_t u[16], v[16];
          tmem_ld16(tmem + lane_base + sb * C::SCOL + r, u);
          tmem_ld16(tmem + lane_base + sb * C::SCOL + N + r, v);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 16; ++e) x[r + e] = __uint_as_float(u[e]) + __uint_as_float(v[e]);
        }
      }
      tc_fence_before();
      mbar_arrive(&sh.sfree[sb]);
      const int tok = tm.tok0 + tid;
      const float ks = tm.ks[tid >> 4], vs = tm.vs[tid >> 4];
      const float lvs = __log2f(vs), ivs = ks == 0.0f ? 0.0f : __frcp_rn(vs);
      const bool edge = tm.cut || tm.tok0 + kTile - 1 > pm.low || (a.window && tm.tok0 <= (int64_t)pm.high - a.window);
      const bool hidden = ks == 0.0f || tok >= pm.len;
      bool over = false;
#pragma unroll
      for (int r = 0; r < N; r += 4) {
        if (r < R) {
          const float4 rc = *reinterpret_cast<const float4*>(&pm.rc[r]);
          const float4 rf = *reinterpret_cast<const float4*>(&sh.ref[r]);
          const float rcs[4] = {rc.x, rc.y, rc.z, rc.w}, rfs[4] = {rf.x, rf.y, rf.z, rf.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float t = fmaf(x[r + e], rcs[e] * ks, lvs);
            if (edge) {
              const int pos = pm.pos[r + e];
              if (hidden || tok > pos || (a.window && tok <= (int64_t)pos - a.window)) t = -INFINITY;
            }
            x[r + e] = t;
            over |= t > (first ? -INFINITY : rfs[e] + kHead);
          }
        }
      }
      if (any_of_128(over || dead)) {
        // some key passes its row's reference: new references, and what was summed up moves to them
        if (any_of_128(dead)) break;
#pragma unroll
        for (int r = 0; r < N; ++r) {
          if (r < R) {
            float top = x[r];
#pragma unroll
            for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
            if (lane == 0) sh.red[warp][r] = top;
          }
        }
        any_of_128(false);
        if (tid >= R && tid < N) sh.ref[tid] = INFINITY;  // not a row: nothing passes it
        if (tid < R) {
          const float top = fmaxf(fmaxf(sh.red[0][tid], sh.red[1][tid]), fmaxf(sh.red[2][tid], sh.red[3][tid]));
          const float old = first ? -INFINITY : sh.ref[tid];
          const float now = fmaxf(top, old);
          sh.ref[tid] = now;
          sh.grow[tid] = now == old ? 1.0f : ex2(old - now);
        }
        any_of_128(false);
        if (!first) {
          if (!mbar_wait_bounded(&sh.pvdone[(i - 1) % C::B], (uint32_t)((i - 1) / C::B) & 1u, c.status)) dead = true;
          if (any_of_128(dead)) break;
          tc_fence_after();
#pragma unroll
          for (int r = 0; r < N; ++r)
            if (r < R) l[r] *= sh.grow[r];
#pragma unroll 1
          for (int col = 0; col < C::MB * C::OCOL; col += 16) {
            const int r = col % N;
            if (r < R) {
              uint32_t u[16];
              tmem_ld16(otm + lane_base + col, u);
              tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 16; ++e) u[e] = __float_as_uint(__uint_as_float(u[e]) * (r + e < R ? sh.grow[r + e] : 0.0f));
              tmem_st16(otm + lane_base + col, u);
            }
          }
          tmem_st_wait();
          tc_fence_before();
        }
      } else if (first) {  // no row sees a key of the pair's first tile
        if (tid < N) sh.ref[tid] = tid < R ? -INFINITY : INFINITY;
        any_of_128(false);
      }
      // P, its sums and its terms; the buffer is free once the tile before last has been multiplied
      if (i >= C::B && !mbar_wait_bounded(&sh.pvdone[sb], (uint32_t)(i / C::B - 1) & 1u, c.status)) dead = true;
      uint8_t* pd = pbuf + sb * C::P + tid * 16;
#pragma unroll
      for (int r = 0; r < N; r += 16) {
        uint32_t t0[4] = {0, 0, 0, 0}, t1[4] = {0, 0, 0, 0}, t2[4] = {0, 0, 0, 0};
#pragma unroll
        for (int q = 0; q < 16; q += 4) {
          if (r + q < R) {
            const float4 rf = *reinterpret_cast<const float4*>(&sh.ref[r + q]);
            const float rfs[4] = {rf.x, rf.y, rf.z, rf.w};
            float pr[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float m = rfs[e] == -INFINITY ? 0.0f : rfs[e];
              pr[e] = r + q + e < R ? ex2(x[r + q + e] - m + kBias) : 0.0f;
              l[r + q + e] = fmaf(pr[e], ivs, l[r + q + e]);
            }
#pragma unroll
            for (int z = 0; z < 2; ++z) {
              const uint32_t h = f16x2(pr[2 * z], pr[2 * z + 1]);
              const uint16_t c0 = e4m3x2(h);
              const uint32_t r1 = rest16(h, codes_f16x2(c0));
              const uint16_t c1 = e4m3x2(r1);
              const uint16_t c2 = e4m3x2(rest16(r1, codes_f16x2(c1)));
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
      mbar_arrive(&sh.pfull[sb]);

      if (last) {  // the pair's last tile here
#pragma unroll
        for (int r = 0; r < N; ++r) {
          if (r < R) {
            float v = l[r];
#pragma unroll
            for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
            if (lane == 0) sh.red[warp][r] = v;
          }
        }
        if (!mbar_wait_bounded(&sh.pvdone[sb], (uint32_t)(i / C::B) & 1u, c.status)) dead = true;
        if (any_of_128(dead)) break;
        tc_fence_after();
        const int64_t first_tile = pm.first;
        const int n_tiles = pm.n_tiles, start = pm.start, h = pm.h;
        const bool whole = first_tile >= u0 && first_tile + n_tiles <= u1;
        const int64_t slot = 2 * cta + (first_tile <= u0 ? 0 : 1);
#pragma unroll 1
        for (int mb = 0; mb < C::MB; ++mb) {
          const int d = mb * 128 + tid;
#pragma unroll 1
          for (int r = 0; r < R; r += 8) {
            uint32_t v0[8], v1[8], v2[8];
            const uint32_t at = otm + lane_base + mb * C::OCOL + r;
            tmem_ld8(at, v0);
            tmem_ld8(at + N, v1);
            tmem_ld8(at + 2 * N, v2);
            tmem_ld_wait();
            if (d < D) {
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const int row = r + e;
                if (row < R) {
                  const float sum = (sh.red[0][row] + sh.red[1][row]) + (sh.red[2][row] + sh.red[3][row]);
                  const float o = fmaf(__uint_as_float(v2[e]), 0x1p-8f, fmaf(__uint_as_float(v1[e]), 0x1p-4f, __uint_as_float(v0[e])));
                  if (whole) {
                    const int t = row / G, g = row - t * G;
                    const __nv_bfloat16 y = __float2bfloat16_rn(sum == 0.0f ? 0.0f : o / sum);
                    a.out[(int64_t)(start + t) * a.ldo + (int64_t)(h * G + g) * a.hso + d] =
                        *reinterpret_cast<const uint16_t*>(&y);
                  } else {
                    da.part_o[(slot * N + row) * D + d] = o;
                    if (d == 0) da.part_ml[slot * N + row] = make_float2(sh.ref[row], sum);
                  }
                }
              }
            }
          }
        }
        tc_fence_before();
        if (!whole) {
          // the CTA whose ticket completes the pair joins the parts, in their order on the line
          auto owner = [&](int64_t unit) { return ((unit + 1) * grid - 1) / total; };
          const int64_t c0 = owner(first_tile), c1 = owner(first_tile + n_tiles - 1);
          const int parts = (int)(c1 - c0 + 1);
          any_of_128(false);
          if (tid == 0) sh.ticket = ticket_add(da.counters + c0, 1);
          any_of_128(false);
          if (sh.ticket == parts - 1) {
            const bool at_start = c0 * total / grid == first_tile;  // the first part is its CTA's first pair
            for (int e = tid; e < R * (D / 4); e += 128) {
              const int row = e / (D / 4), d = (e % (D / 4)) * 4;
              float4 v = make_float4(0, 0, 0, 0);
              float top = -INFINITY, sum = 0.0f;
              for (int q = 0; q < parts; ++q) {
                const int64_t sl = 2 * (c0 + q) + (q == 0 && !at_start ? 1 : 0);
                top = fmaxf(top, __ldcg(&da.part_ml[sl * N + row]).x);
              }
              for (int q = 0; q < parts; ++q) {
                const int64_t sl = 2 * (c0 + q) + (q == 0 && !at_start ? 1 : 0);
                const float2 z = __ldcg(&da.part_ml[sl * N + row]);
                const float4 y = __ldcg(reinterpret_cast<const float4*>(da.part_o + (sl * N + row) * D + d));
                const float f = z.x == -INFINITY ? 0.0f : ex2(z.x - top);
                v.x = fmaf(y.x, f, v.x), v.y = fmaf(y.y, f, v.y), v.z = fmaf(y.z, f, v.z), v.w = fmaf(y.w, f, v.w);
                sum = fmaf(z.y, f, sum);
              }
              const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
              const int t = row / G, g = row - t * G;
              const __nv_bfloat162 y0 = __floats2bfloat162_rn(v.x * inv, v.y * inv), y1 = __floats2bfloat162_rn(v.z * inv, v.w * inv);
              *reinterpret_cast<uint2*>(a.out + (int64_t)(start + t) * a.ldo + (int64_t)(h * G + g) * a.hso + d) =
                  make_uint2(*reinterpret_cast<const uint32_t*>(&y0), *reinterpret_cast<const uint32_t*>(&y1));
            }
            if (tid == 0) da.counters[c0] = 0;
          }
        }
        any_of_128(false);  // everyone is done with this pair's rows, sums and references
        if (tid == 0) mbar_arrive(&sh.qfree[p % C::B]);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 4) tmem_dealloc(tmem, 512);
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
  return launch_pdl(attn_decode_kernel<D, N>, dim3(grid), dim3(kThreads), C::SMEM, s, km, vm, da) == cudaSuccess
             ? QG_OK
             : QG_ERR_CUDA;
}

template <int D>
int launch_rows(int rows, const DecodeArgs& da, const CUtensorMap& km, const CUtensorMap& vm, int grid, cudaStream_t s) {
  if (rows == 16) return launch<D, 16>(da, km, vm, grid, s);
  if (rows == 32) return launch<D, 32>(da, km, vm, grid, s);
  return launch<D, 64>(da, km, vm, grid, s);
}

constexpr size_t kCounterBytes = 4096;  // counters of up to 1024 CTAs, at the same place whatever the call

}  // namespace

int decode_rows(int64_t rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 ? 64 : 0; }

size_t decode_workspace(int64_t rows, int head_dim, const DeviceInfo& dev) {
  const size_t r = (size_t)decode_rows(rows), slots = 2 * (size_t)dev.sms;
  return kWsHeader + kCounterBytes + slots * r * sizeof(float2) + slots * r * head_dim * sizeof(float);
}

int launch_attn_decode(const AttnArgs& a, int head_dim, int64_t rows, const DeviceInfo& dev, void* ws, void* stream) {
  if (dev.sms > 1024) return QG_ERR_UNSUPPORTED;
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
  w += kCounterBytes;
  da.part_ml = reinterpret_cast<float2*>(w);
  da.part_o = reinterpret_cast<float*>(w + 2 * (size_t)dev.sms * r * sizeof(float2));
  // no more CTAs than tiles that there can be
  const int64_t most = (int64_t)a.c.n_seqs * a.c.hkv * ((a.c.max_len + kTile - 1) / kTile);
  const int grid = (int)std::min<int64_t>(dev.sms, most);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  switch (head_dim) {
    case 64: return launch_rows<64>(r, da, km, vm, grid, s);
    case 128: return launch_rows<128>(r, da, km, vm, grid, s);
    case 256: return launch_rows<256>(r, da, km, vm, grid, s);
  }
  return QG_ERR_UNSUPPORTED;
}

}  // namespace qg
