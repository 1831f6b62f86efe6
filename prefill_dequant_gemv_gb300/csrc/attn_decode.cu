// Attention of a few rows a KV head over the 8-bit paged cache (decode, speculative
// verification): the new tokens' query heads of one (sequence, KV head) pair, R = new * G rows,
// against all its keys.
//
// The mathematics.  With codes k, v, page scales ks, vs and s_j = scale * ks_j * (q . k_j) * log2(e), each
// row keeps t_j = s_j + log2(vs_j), a running maximum m of them and P_j = 2^(t_j - m):
//   out = sum_j P_j v_j / sum_j P_j / vs_j.
// The value scale sits in the exponent, so P is rounded to fp16 relative to the largest
// contribution whatever the scales' spread, and one multiply a key and row (in the denominator's FMA) is
// all they cost.  E4M3 codes are exact in fp16; a query row is divided by a power of two to
// fit fp16 (exactly, but for elements 2^-14 below its largest).  Sums and statistics are fp32.
//
// Bound by HBM: each key and value code is used for R rows only.
//   * The pairs' keys, in units of UT tokens, lie on one line, which the CTAs (one an SM) share
//     out evenly whatever the lengths; a pair cut between CTAs leaves partial (m, l, O) rows in the
//     workspace, and the CTA that finishes last adds them in order.  One launch.
//   * A producer warp copies units into a ring in shared memory by TMA: slices of 16 tokens (a
//     page holds whole slices), whose 128-byte swizzle makes every read below free of bank conflicts.
//   * Each of the eight consumer warps takes a 16-token slice of a unit from the codes to its own (m, l, O)
//     in registers; the warps meet once a pair.  Both products are warp-level MMAs m16n8k16 whose rows are the
//     query rows.  A contraction may be taken in any order, so a lane's
//     16-byte read of a key row is four k-steps of the B operand as it stands, and the token order of the
//     score columns is chosen so that a lane's own four tokens are the rows it reads of
//     V, where two byte permutes a word pair up the tokens.  Codes go from shared memory to operands
//     without another copy.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>

#include "qg_attn.h"
#include "qg_sync.cuh"

namespace qg {
namespace {

constexpr int kConsumers = 8;
// Two warpgroups of consumers and one for the producer warp, so that registers can move: 384 threads
// launch with 168 each, the consumers take 232 and the producer's group keeps 40.
constexpr int kThreads = 384;
constexpr int kConsumerRegs = 232, kProducerRegs = 40;
static_assert(256 * kConsumerRegs + 128 * kProducerRegs <= kThreads * 168, "registers");
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLazy = 8.0f;  // a row is rescaled once its maximum has grown by 2^8: P stays below 2^8

// D: head dimension; RT: row tiles of 16 a warp; GW: warps that share a slice (each its own rows).
template <int D, int RT, int GW>
struct Cfg {
  static constexpr int BOX = D < 128 ? D : 128;       // bytes of a TMA row
  static constexpr int NBOX = D / BOX;
  static constexpr int SLICE = 16 * D;                // bytes of a slice of keys (or values)
  static constexpr int NS = kConsumers / GW;          // slices a unit
  static constexpr int UT = 16 * NS;                  // tokens a unit
  static constexpr int UNIT = 2 * NS * SLICE;
  static constexpr int ROWS = 16 * RT * GW;
  static constexpr int CW = BOX / 8;                  // columns of O a lane column holds in a box
  static constexpr int NT = D / 8;                    // 8-wide column tiles of O
  static constexpr int MC = D == 256 ? 32 : 64;       // columns of O merged at a time
  static constexpr int MERGE = kConsumers * 16 * MC * 4;
  static constexpr int META = 128;
  static constexpr int FIXED = 1024 + MERGE + kConsumers * 16 * RT * 8 + 64;
  static constexpr int S0 = (232448 - FIXED) / (UNIT + META + 16);
  static constexpr int S = S0 > 8 ? 8 : S0;
  static constexpr int SMEM = FIXED + S * (UNIT + META + 16);
  static_assert(S >= 2 && SMEM <= 232448, "shared memory");
};

// What a stage holds (128 bytes of shared memory).
struct Meta {
  int flags;          // 1: first unit of a pair in this CTA, 2: last one
  int h, tok0, n_units;
  int start, rows, len, pad0;
  int64_t pair_first;  // the pair's first unit on the line
  int pad1[6];
  float ks[8], vs[8];  // the slices' scales; 0: the slice holds no key
};
static_assert(sizeof(Meta) == 128, "meta");

struct DecodeArgs {
  AttnArgs a;
  int* counters;   // one a CTA: the parts of the pair that begins in it and ends in another
  float2* part_ml; // [2 * grid][ROWS]
  float* part_o;   // [2 * grid][ROWS][D]
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Two E4M3 codes (the low or high 16 bits of w) -> two fp16 values.
__device__ __forceinline__ uint32_t codes_lo(uint32_t w) {
  uint32_t r;
  asm("{.reg .b16 l, h; mov.b32 {l, h}, %1; cvt.rn.f16x2.e4m3x2 %0, l;}" : "=r"(r) : "r"(w));
  return r;
}
__device__ __forceinline__ uint32_t codes_hi(uint32_t w) {
  uint32_t r;
  asm("{.reg .b16 l, h; mov.b32 {l, h}, %1; cvt.rn.f16x2.e4m3x2 %0, h;}" : "=r"(r) : "r"(w));
  return r;
}
__device__ __forceinline__ uint32_t f16x2(float a, float b) {  // a in the low half
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}
__device__ __forceinline__ uint32_t bf16x2(float a, float b) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
  return v;
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
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// First key that any row of the sequence sees, rounded down to a slice; units of a pair (one at least where
// there are rows, so that rows without a key are written).
__device__ __forceinline__ int first_key(const Seq& s, int64_t window) {
  const int64_t p = (int64_t)s.len - s.rows + 1 - window;
  return window && p > 0 ? (int)(min(p, (int64_t)s.len) & ~int64_t(15)) : 0;
}
template <int UT>
__device__ __forceinline__ int units_of(const Seq& s, int64_t window) {
  return s.rows > 0 ? max(1, (s.len - first_key(s, window) + UT - 1) / UT) : 0;
}

template <int D, int RT, int GW>
__global__ void __launch_bounds__(kThreads, 1)
    attn_decode_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                       const DecodeArgs da) {
  using C = Cfg<D, RT, GW>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* merge = reinterpret_cast<float*>(smem + C::S * C::UNIT);
  float2* ml = reinterpret_cast<float2*>(merge + C::MERGE / 4);  // [warp][16 * RT]
  Meta* meta = reinterpret_cast<Meta*>(ml + kConsumers * 16 * RT);
  uint64_t* full = reinterpret_cast<uint64_t*>(meta + C::S);
  uint64_t* empty = full + C::S;
  uint64_t* cbar = empty + C::S;                 // the consumers' own barrier
  int* shared = reinterpret_cast<int*>(cbar + 1);
  const AttnArgs& a = da.a;
  const KvArgs& c = a.c;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = a.hq / c.hkv;

  if (tid == 0) {
    for (int s = 0; s < C::S; ++s) {
      mbar_init(&full[s], 2 * C::NS);
      mbar_init(&empty[s], kConsumers);
    }
    mbar_init(cbar, kConsumers);
    fence_mbar_init();
  }
  pdl_wait();

  // the line: units of all sequences, each counted once (all its KV heads have as many)
  int64_t total = 0;
  bool bad = false;
  for (int base = 0; base < c.n_seqs; base += 32) {
    int n = 0;
    if (base + lane < c.n_seqs) n = units_of<C::UT>(seq_of(c, base + lane, &bad), a.window);
    total += __reduce_add_sync(0xFFFFFFFFu, n);
  }
  if (bad && warp == 0 && blockIdx.x == 0) atomicExch(c.status, kStatusInvalid);
  total *= c.hkv;
  // with no more CTAs than units, each has one at least
  const int64_t grid = min((int64_t)gridDim.x, total), cta = blockIdx.x;
  __syncthreads();
  if (cta >= grid) return;
  const int64_t u0 = cta * total / grid, u1 = (cta + 1) * total / grid;

  if (warp >= kConsumers) {  // ---------------------------------------------------------------- producer
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kProducerRegs));
    if (warp > kConsumers) return;
    // the pair of unit u0
    int b = 0, h = 0;
    int64_t k = 0, left = u0;
    Seq sq = {0, 0, 0};
    bool ignore = false;
    int n = 0;
    for (int base = 0; base < c.n_seqs; base += 32) {
      Seq t = {0, 0, 0};
      if (base + lane < c.n_seqs) t = seq_of(c, base + lane, &ignore);
      const int un = units_of<C::UT>(t, a.window);
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
    k = left - (int64_t)h * n;
    int64_t pair_first = u0 - k;
    int lo = first_key(sq, a.window);
    const int smask = (1 << c.page_log2) - 1;
    // this lane's slice of the unit: its token and page id (-1: no such tokens)
    auto page_of = [&](int64_t kk) {
      const int64_t tok = lo + kk * C::UT + 16 * lane;
      return lane < C::NS && tok < sq.len ? c.pages[(int64_t)b * c.page_stride + (tok >> c.page_log2)] : -1;
    };
    int id = page_of(k);
    bool dead = false;
    int64_t issued = 0;
    for (int64_t u = u0; u < u1; ++u) {
      const int s = (int)(issued % C::S);
      // this unit's data before the state moves on to the next
      const int tok0 = (int)(lo + k * C::UT), ch = h, cn = n, cid = id;
      const Seq cs = sq;
      const int64_t cfirst = pair_first;
      const bool first = k == 0 || u == u0, last = k == n - 1 || u == u1 - 1;
      if (u + 1 < u1) {
        if (++k == n) {
          k = 0;
          pair_first += n;
          if (++h == c.hkv) {
            h = 0;
            do {
              ++b;
              sq = seq_of(c, b, &ignore);
              n = units_of<C::UT>(sq, a.window);
            } while (n == 0);
            lo = first_key(sq, a.window);
          }
        }
        id = page_of(k);
      }
      if (issued >= C::S && !dead && !mbar_wait_bounded(&empty[s], (uint32_t)((issued / C::S) & 1) ^ 1u, c.status))
        dead = true;
      if (dead) break;
      Meta* m = &meta[s];
      if (lane == 0) {
        m->flags = (first ? 1 : 0) | (last ? 2 : 0);
        m->h = ch, m->tok0 = tok0, m->n_units = cn;
        m->start = cs.start, m->rows = cs.rows, m->len = cs.len;
        m->pair_first = cfirst;
      }
      if (lane < C::NS) {
        const int tok = tok0 + 16 * lane;
        bool ok = tok < cs.len;
        if (ok && (cid < 0 || cid >= c.n_pages)) {
          ok = false;
          atomicExch(c.status, kStatusInvalid);
        }
        uint8_t* kd = smem + s * C::UNIT + lane * C::SLICE;
        uint8_t* vd = kd + C::NS * C::SLICE;
        if (ok) {
          const int64_t tile = (int64_t)cid * c.hkv + ch;
          mbar_arrive_expect_tx(&full[s], 2 * C::SLICE);
#pragma unroll
          for (int x = 0; x < C::NBOX; ++x) tma_load_3d(kd + x * 2048, &kmap, x * 128, tok & smask, (int)tile, &full[s]);
#pragma unroll
          for (int x = 0; x < C::NBOX; ++x) tma_load_3d(vd + x * 2048, &vmap, x * 128, tok & smask, (int)tile, &full[s]);
          cp_async4(&m->ks[lane], c.ks + tile);
          cp_async4(&m->vs[lane], c.vs + tile);
        } else {
          m->ks[lane] = 0.0f;  // a hidden slice: no scale is 0
          m->vs[lane] = 0.0f;
          mbar_arrive(&full[s]);
        }
        cp_async_arrive(&full[s]);
      }
      __syncwarp();
      ++issued;
    }
    // no copy is left in flight into this CTA's shared memory when it ends
    for (int64_t j = issued > C::S ? issued - C::S : 0; j < issued; ++j)
      mbar_wait_bounded(&full[j % C::S], (uint32_t)(j / C::S) & 1u, c.status);
    return;
  }

  // ------------------------------------------------------------------------------------ consumers
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kConsumerRegs));
  const int n4 = lane >> 2, j4 = lane & 3;  // column (or row) and quad lane of the MMA fragments
  const int slice = warp / GW, rbase = (warp % GW) * (16 * RT);
  // token of score column col in tile x: 8x + g, g = ((j ^ 2p) << 1) | p for col = 2j + p
  const int kr = (((n4 >> 1) ^ (2 * (n4 & 1))) << 1) | (n4 & 1);
  const int g0 = j4 << 1, g1 = ((j4 ^ 2) << 1) | 1;
  const uint32_t base_k = smem_u32(smem) + slice * C::SLICE, base_v = base_k + C::NS * C::SLICE;
  uint32_t qf[RT][D / 16][4];
  float o[RT][C::NT][4];
  float m_[RT][2], l_[RT][2], rc[RT][2];
  int pos[RT][2];
  bool dead = false;
  uint32_t phase = 0;
  // all consumer warps meet; a warp that gave up leaves the others to their own limit
  auto meet = [&]() {
    __syncwarp();
    if (lane == 0) mbar_arrive(cbar);
    if (!dead && !mbar_wait_bounded(cbar, phase, c.status)) dead = true;
    dead = __any_sync(0xFFFFFFFFu, dead);
    phase ^= 1;
  };

  for (int64_t u = u0; u < u1; ++u) {
    const int64_t it = u - u0;
    const int s = (int)(it % C::S);
    if (!dead && !mbar_wait_bounded(&full[s], (uint32_t)(it / C::S) & 1u, c.status)) dead = true;
    dead = __any_sync(0xFFFFFFFFu, dead);
    const Meta& m = meta[s];
    const int flags = m.flags, R = min(m.rows * G, C::ROWS), len = m.len, t0 = m.tok0 + 16 * slice;
    const int sh = m.h, sstart = m.start, srows = m.rows, n_units = m.n_units;
    const int64_t pair_first = m.pair_first;
    if (dead) break;
    if (flags & 1) {  // a new pair: its query rows
#pragma unroll
      for (int r = 0; r < RT; ++r) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int row = rbase + 16 * r + 8 * half + n4;
          const bool in = row < R;
          const int i = in ? row / G : 0, g = in ? row - i * G : 0;
          const uint16_t* qp = a.q + (int64_t)(sstart + i) * a.ldq + (int64_t)(sh * G + g) * a.hsq;
          pos[r][half] = in ? len - srows + i : -1;
          uint4 w[D / 32];
          float amax = 0.0f;
#pragma unroll
          for (int x = 0; x < D / 64; ++x) {
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              uint4 v = make_uint4(0, 0, 0, 0);
              if (in) v = *reinterpret_cast<const uint4*>(qp + (4 * x + j4) * 16 + 8 * y);
              w[2 * x + y] = v;
              const uint32_t e[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
              for (int z = 0; z < 4; ++z)
                amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(e[z] << 16)), fabsf(__uint_as_float(e[z] & 0xFFFF0000u))));
            }
          }
          amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
          amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
          // a power of two that brings the row's largest element to [1, 2)
          const int e = min(max((__float_as_int(amax) >> 23) - 127, -125), 125);
          const float down = __int_as_float((127 - e) << 23);
          rc[r][half] = __int_as_float((127 + e) << 23) * (a.scale * kLog2e);
          m_[r][half] = -INFINITY;
          l_[r][half] = 0.0f;
#pragma unroll
          for (int x = 0; x < D / 32; ++x) {  // 8 elements: two k-steps' halves
            const uint32_t v[4] = {w[x].x, w[x].y, w[x].z, w[x].w};
#pragma unroll
            for (int z = 0; z < 4; ++z)
              qf[r][2 * x + (z >> 1)][half + 2 * (z & 1)] =
                  f16x2(__uint_as_float(v[z] << 16) * down, __uint_as_float(v[z] & 0xFFFF0000u) * down);
          }
        }
#pragma unroll
        for (int t = 0; t < C::NT; ++t) o[r][t][0] = o[r][t][1] = o[r][t][2] = o[r][t][3] = 0.0f;
      }
    }
    const float ks = m.ks[slice], vs = m.vs[slice];
    if (t0 < len && ks != 0.0f) {
      // scores
      float sc[RT][2][4];
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int x = 0; x < 2; ++x) sc[r][x][0] = sc[r][x][1] = sc[r][x][2] = sc[r][x][3] = 0.0f;
      const uint32_t kb = base_k + s * C::UNIT, vb = base_v + s * C::UNIT;
#pragma unroll
      for (int x = 0; x < D / 64; ++x) {
        const uint32_t at = D == 64 ? kb + kr * 64 + ((j4 ^ ((kr >> 1) & 3)) << 4)
                                    : kb + (x >> 1) * 2048 + kr * 128 + ((((x & 1) * 4 + j4) ^ kr) << 4);
        const uint4 ka = lds128(at), kc = lds128(at + 8 * C::BOX);
        const uint32_t wa[4] = {ka.x, ka.y, ka.z, ka.w}, wc[4] = {kc.x, kc.y, kc.z, kc.w};
#pragma unroll
        for (int z = 0; z < 4; ++z) {
          const uint32_t a0 = codes_lo(wa[z]), a1 = codes_hi(wa[z]), c0 = codes_lo(wc[z]), c1 = codes_hi(wc[z]);
#pragma unroll
          for (int r = 0; r < RT; ++r) {
            const uint32_t* f = qf[r][4 * x + z];
            mma(sc[r][0], f[0], f[1], f[2], f[3], a0, a1);
            mma(sc[r][1], f[0], f[1], f[2], f[3], c0, c1);
          }
        }
      }
      const float lvs = __log2f(vs), ivs = __frcp_rn(vs);
      const int tok[4] = {t0 + g0, t0 + g1, t0 + 8 + g0, t0 + 8 + g1};
      uint32_t pf[RT][4];
#pragma unroll
      for (int r = 0; r < RT; ++r) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          float* s0 = &sc[r][0][2 * half];
          float* s1 = &sc[r][1][2 * half];
          const float f = rc[r][half] * ks;
          float t[4] = {fmaf(s0[0], f, lvs), fmaf(s0[1], f, lvs), fmaf(s1[0], f, lvs), fmaf(s1[1], f, lvs)};
          const int p = pos[r][half];
          if (t0 + 15 > p || (a.window && (int64_t)t0 <= (int64_t)p - a.window)) {
            const int64_t from = a.window ? (int64_t)p - a.window : -1;
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (tok[e] > p || tok[e] <= from) t[e] = -INFINITY;
          }
          float top = fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3]));
          top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
          top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
          const float old = m_[r][half];
          const bool grow = top > old + kLazy || old == -INFINITY;
          const float now = grow ? fmaxf(top, old) : old;
          const float w = now == -INFINITY ? 1.0f : ex2(old - now);
          if (__any_sync(0xFFFFFFFFu, w != 1.0f)) {
            l_[r][half] *= w;
#pragma unroll
            for (int y = 0; y < C::NT; ++y) {
              o[r][y][2 * half] *= w;
              o[r][y][2 * half + 1] *= w;
            }
          }
          m_[r][half] = now;
          const float ref = now == -INFINITY ? 0.0f : now;
          float sum = 0.0f;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            t[e] = ex2(t[e] - ref);
            sum += t[e];
          }
          l_[r][half] = fmaf(sum, ivs, l_[r][half]);
          pf[r][half] = f16x2(t[0], t[1]);
          pf[r][2 + half] = f16x2(t[2], t[3]);
        }
      }
      // values: rows of this lane's four tokens; what lies beyond the sequence is cleared
      const bool cut = t0 + 16 > len;
#pragma unroll
      for (int x = 0; x < C::NBOX; ++x) {
        uint4 v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int row = (i & 1) ? g1 : g0;
          if (D == 64) {
            const uint2 w = lds64(vb + (i >> 1) * 512 + row * 64 + (((n4 >> 1) ^ ((row >> 1) & 3)) << 4) + (n4 & 1) * 8);
            v[i] = make_uint4(w.x, w.y, 0, 0);
          } else {
            v[i] = lds128(vb + x * 2048 + (i >> 1) * 1024 + row * 128 + ((n4 ^ row) << 4));
          }
          if (cut && tok[i] >= len) v[i] = make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int y = 0; y < C::CW / 4; ++y) {
          const uint32_t w[4] = {y == 0 ? v[0].x : y == 1 ? v[0].y : y == 2 ? v[0].z : v[0].w,
                                 y == 0 ? v[1].x : y == 1 ? v[1].y : y == 2 ? v[1].z : v[1].w,
                                 y == 0 ? v[2].x : y == 1 ? v[2].y : y == 2 ? v[2].z : v[2].w,
                                 y == 0 ? v[3].x : y == 1 ? v[3].y : y == 2 ? v[3].z : v[3].w};
          const uint32_t p0 = __byte_perm(w[0], w[1], 0x5140), p1 = __byte_perm(w[0], w[1], 0x7362);
          const uint32_t q0 = __byte_perm(w[2], w[3], 0x5140), q1 = __byte_perm(w[2], w[3], 0x7362);
          const uint32_t b0[4] = {codes_lo(p0), codes_hi(p0), codes_lo(p1), codes_hi(p1)};
          const uint32_t b1[4] = {codes_lo(q0), codes_hi(q0), codes_lo(q1), codes_hi(q1)};
#pragma unroll
          for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int r = 0; r < RT; ++r)
              mma(o[r][x * C::CW + 4 * y + e], pf[r][0], pf[r][1], pf[r][2], pf[r][3], b0[e], b1[e]);
        }
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&empty[s]);

    if (flags & 2) {  // the pair's last unit here: merge the warps' rows
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          float l = l_[r][half];
          l += __shfl_xor_sync(0xFFFFFFFFu, l, 1);
          l += __shfl_xor_sync(0xFFFFFFFFu, l, 2);
          if (j4 == 0) ml[warp * 16 * RT + 16 * r + 8 * half + n4] = make_float2(m_[r][half], l);
        }
      meet();
      const bool whole = u - pair_first == n_units - 1 && pair_first >= u0;
      const int64_t slot = 2 * cta + (pair_first <= u0 ? 0 : 1);
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        float f[2];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          float top = -INFINITY;
#pragma unroll
          for (int w = 0; w < C::NS; ++w)
            top = fmaxf(top, ml[(w * GW + warp % GW) * 16 * RT + 16 * r + 8 * half + n4].x);
          f[half] = m_[r][half] == -INFINITY ? 0.0f : ex2(m_[r][half] - top);
        }
#pragma unroll
        for (int x = 0; x < C::NBOX; ++x) {
#pragma unroll
          for (int pass = 0; pass < C::CW * 8 / C::MC; ++pass) {
            constexpr int TP = C::MC / 8;
            // this warp's 16 rows x MC columns: column n * TP + t
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              if (rbase + 16 * r + 8 * half + n4 < R) {
                float* dst = merge + (warp * 16 + 8 * half + n4) * C::MC + 2 * j4 * TP;
#pragma unroll
                for (int p = 0; p < 2; ++p)
#pragma unroll
                  for (int t = 0; t < TP; t += 4) {
                    float4 v;
                    v.x = o[r][x * C::CW + pass * TP + t][2 * half + p] * f[half];
                    v.y = o[r][x * C::CW + pass * TP + t + 1][2 * half + p] * f[half];
                    v.z = o[r][x * C::CW + pass * TP + t + 2][2 * half + p] * f[half];
                    v.w = o[r][x * C::CW + pass * TP + t + 3][2 * half + p] * f[half];
                    *reinterpret_cast<float4*>(dst + p * TP + t) = v;
                  }
              }
            }
            meet();
            // rows of every warp group, four columns a thread
            for (int e = tid; e < GW * 16 * (C::MC / 4); e += 32 * kConsumers) {
              const int col = (e % (C::MC / 4)) * 4, row16 = (e / (C::MC / 4)) % 16, gw = e / (C::MC * 4);
              const int row = gw * 16 * RT + 16 * r + row16;
              if (row < R) {
                float4 v = make_float4(0, 0, 0, 0);
                float top = -INFINITY, l = 0.0f;
#pragma unroll
                for (int w = 0; w < C::NS; ++w) {
                  const float4 z = *reinterpret_cast<const float4*>(merge + ((w * GW + gw) * 16 + row16) * C::MC + col);
                  v.x += z.x, v.y += z.y, v.z += z.z, v.w += z.w;
                  top = fmaxf(top, ml[(w * GW + gw) * 16 * RT + 16 * r + row16].x);
                }
#pragma unroll
                for (int w = 0; w < C::NS; ++w) {
                  const float2 z = ml[(w * GW + gw) * 16 * RT + 16 * r + row16];
                  if (z.x != -INFINITY) l = fmaf(z.y, ex2(z.x - top), l);
                }
                const int d = x * 128 + (col / TP) * C::CW + pass * TP + col % TP;
                if (whole) {
                  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
                  const int i = row / G, g = row - i * G;
                  *reinterpret_cast<uint2*>(a.out + (int64_t)(sstart + i) * a.ldo + (int64_t)(sh * G + g) * a.hso + d) =
                      make_uint2(bf16x2(v.x * inv, v.y * inv), bf16x2(v.z * inv, v.w * inv));
                } else {
                  *reinterpret_cast<float4*>(da.part_o + (slot * C::ROWS + row) * D + d) = v;
                  if (d == 0) da.part_ml[slot * C::ROWS + row] = make_float2(top, l);
                }
              }
            }
            meet();
          }
        }
      }
      if (!whole) {
        // the CTA whose ticket completes the pair joins the parts, in their order on the line
        auto owner = [&](int64_t unit) { return ((unit + 1) * grid - 1) / total; };
        const int64_t c0 = owner(pair_first), c1 = owner(pair_first + n_units - 1);
        const int parts = (int)(c1 - c0 + 1);
        if (dead) break;
        if (tid == 0) shared[0] = ticket_add(da.counters + c0, 1);
        meet();
        if (shared[0] == parts - 1) {
          const bool at_start = c0 * total / grid == pair_first;  // the first part is its CTA's first pair
          for (int e = tid; e < R * (D / 4); e += 32 * kConsumers) {
            const int row = e / (D / 4), d = (e % (D / 4)) * 4;
            float4 v = make_float4(0, 0, 0, 0);
            float top = -INFINITY, l = 0.0f;
            for (int p = 0; p < parts; ++p) {
              const int64_t sl = 2 * (c0 + p) + (p == 0 && !at_start ? 1 : 0);
              top = fmaxf(top, __ldcg(&da.part_ml[sl * C::ROWS + row]).x);
            }
            for (int p = 0; p < parts; ++p) {
              const int64_t sl = 2 * (c0 + p) + (p == 0 && !at_start ? 1 : 0);
              const float2 z = __ldcg(&da.part_ml[sl * C::ROWS + row]);
              const float4 y = __ldcg(reinterpret_cast<const float4*>(da.part_o + (sl * C::ROWS + row) * D + d));
              const float f = z.x == -INFINITY ? 0.0f : ex2(z.x - top);
              v.x = fmaf(y.x, f, v.x), v.y = fmaf(y.y, f, v.y), v.z = fmaf(y.z, f, v.z), v.w = fmaf(y.w, f, v.w);
              l = fmaf(z.y, f, l);
            }
            const float inv = l == 0.0f ? 0.0f : 1.0f / l;
            const int i = row / G, g = row - i * G;
            *reinterpret_cast<uint2*>(a.out + (int64_t)(sstart + i) * a.ldo + (int64_t)(sh * G + g) * a.hso + d) =
                make_uint2(bf16x2(v.x * inv, v.y * inv), bf16x2(v.z * inv, v.w * inv));
          }
          if (tid == 0) da.counters[c0] = 0;
        }
        meet();
      }
    }
  }
}

template <int D, int RT, int GW>
int launch(const DecodeArgs& da, const CUtensorMap& km, const CUtensorMap& vm, int grid, cudaStream_t s) {
  using C = Cfg<D, RT, GW>;
  static std::atomic<unsigned long long> configured{0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return QG_ERR_CUDA;
  const unsigned long long bit = 1ull << (dev & 63);
  if (!(configured.load() & bit)) {
    if (cudaFuncSetAttribute((const void*)attn_decode_kernel<D, RT, GW>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             C::SMEM) != cudaSuccess)
      return QG_ERR_CUDA;
    configured.fetch_or(bit);
  }
  return launch_pdl(attn_decode_kernel<D, RT, GW>, dim3(grid), dim3(kThreads), C::SMEM, s, km, vm, da) == cudaSuccess
             ? QG_OK
             : QG_ERR_CUDA;
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
  CUtensorMap km, vm;
  if (!encode_pages(&km, a.c.k, head_dim, 1 << a.c.page_log2, a.c.n_pages * a.c.hkv, 16) ||
      !encode_pages(&vm, a.c.v, head_dim, 1 << a.c.page_log2, a.c.n_pages * a.c.hkv, 16))
    return QG_ERR_CUDA;
  const int r = decode_rows(rows);
  DecodeArgs da;
  da.a = a;
  uint8_t* w = static_cast<uint8_t*>(ws) + kWsHeader;
  da.counters = reinterpret_cast<int*>(w);
  w += kCounterBytes;
  da.part_ml = reinterpret_cast<float2*>(w);
  da.part_o = reinterpret_cast<float*>(w + 2 * (size_t)dev.sms * r * sizeof(float2));
  // no more CTAs than units of 64 tokens that there can be
  const int64_t most = (int64_t)a.c.n_seqs * a.c.hkv * ((a.c.max_len + 63) / 64);
  const int grid = (int)std::min<int64_t>(dev.sms, most);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (head_dim == 64) {
    if (r == 16) return launch<64, 1, 1>(da, km, vm, grid, s);
    if (r == 32) return launch<64, 2, 1>(da, km, vm, grid, s);
    return launch<64, 4, 1>(da, km, vm, grid, s);
  }
  if (head_dim == 128) {
    if (r == 16) return launch<128, 1, 1>(da, km, vm, grid, s);
    if (r == 32) return launch<128, 2, 1>(da, km, vm, grid, s);
    return launch<128, 2, 2>(da, km, vm, grid, s);
  }
  if (r == 16) return launch<256, 1, 1>(da, km, vm, grid, s);
  if (r == 32) return launch<256, 1, 2>(da, km, vm, grid, s);
  return launch<256, 1, 4>(da, km, vm, grid, s);
}

}  // namespace qg
