// Attention of many rows a KV head over the 8-bit paged cache (prompts and chunks of prompts): a CTA
// takes MT tiles of 128 query rows of one (sequence, KV head) -- row = token * G + query head, so the G
// heads share what is loaded -- through the keys that they see, BN at a time, with an online softmax.
//
// The mathematics is the few-row kernel's: t_j = scale * ks_j * (q . k_j) * log2(e) + log2(vs_j), P_j = 2^(t_j - m + 7),
//   out = sum P_j v_j / sum (P_j / vs_j),   m moving only when a row's maximum has grown by 2^8 (conditional rescaling, a
//   published refinement of the online softmax).
//
// Bound by the tensor cores and, about as much, by the softmax's exponentials and conversions, so:
//   * scores run on the 8-bit tensor cores, the key codes as they come from the cache and a query row as
//     the sum of an E4M3 and an E5M2 term (bf16's 8 significant bits; the second's exponents keep what is left of small
//     elements: exact but for those below 2^-13 of the row's largest, off by 2^-21 of it at most), which costs what one
//     fp16 product of converted keys would, without the conversion and at half its shared-memory traffic;
//   * P is rounded to fp16 (11 bits of it, or 2^-32 of the row's largest weight) and stays in tensor memory, over the scores it came from, as the A operand
//     of the second product; splitting it into E4M3 terms would cost three conversions an element where
//     this needs one, and the value codes are converted once for all rows instead, by a
//     warpgroup of their own, into the fp16 tile that the second product reads transposed;
//   * a row belongs to two threads, each with half of a step's keys and of the outputs: with one thread a row
//     a prompt of 2048 tokens took 88 us where two took 84;
//   * two row tiles of 128 take turns: one's products run during the other's softmax (heads of 256 have room in tensor
//     memory for one tile and two buffers of scores).
// Few tiles are split over the keys (parts of a row join in order in the CTA that finishes last).
//
// Measured (GB300): a prompt of 8192 tokens, 40/8 heads of 128: 631 us, 1090 TFLOP/s of the 4 D a query and key; 2048 tokens:
// 68 us; 512 tokens on 32768, 24/4 heads of 256: 394 us, 1050 TFLOP/s; 6 prompts of up to 2777 tokens under a
// window of 1024, 32/4 heads of 64: 187 us, 407 TFLOP/s.  A step of 256 rows x 128 keys takes 4020 cycles (heads of 128) or
// 3370 (64), 128 x 64 at 256 takes 2060; the tensor cores' share at 128 is 2350, as the scores' two terms cost what the
// outputs do.  The rest is the chain of one row tile, 2300 cycles from scores to weights and 300 until the
// products start, which two tiles overlap in part.  A CTA's start and end take 20000 cycles, the work of five steps.  The
// forms of 80 registers (heads of 64 and 128) spill 28 and 48 bytes.
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

constexpr float kLazy = 8.0f;           // a row's reference moves when its maximum has grown by this
// P of a key at the reference is 2^7 and below 2^15 then, what fp16 holds: 11 bits down to 2^-21 of the reference's
// weight, and off by 2^-32 of it below.  The sums take P * 2^-7, so that they have the room of plain weights.
constexpr float kBias = 7.0f, kUnbias = 0x1p-7f;

template <int D>
struct Cfg {
  static constexpr int MT = D == 256 ? 1 : 2;         // row tiles of 128
  // keys a step (two row tiles with two buffers of 64 keys each: 843 us where one of 128 took 703, 8192 tokens, heads of
  // 128: an MMA of 64 keys takes as long as one of 128)
  static constexpr int BN = D == 256 ? 64 : 128;
  static constexpr int ROWS = 128 * MT;
  static constexpr int SOFT = 256 * MT;               // softmax threads: two a row
  static constexpr int THREADS = SOFT + 256;
  // registers a thread: what the launch gives, what softmax threads take, what the other two warpgroups keep
  static constexpr int REGS = MT == 2 ? 80 : 128, RSOFT = MT == 2 ? 96 : 144, RREST = MT == 2 ? 48 : 112;
  static_assert(SOFT * RSOFT + 256 * RREST <= THREADS * REGS && THREADS * REGS <= 65536, "registers");
  static constexpr int PW = D < 128 ? D : 128;        // bytes of a row of a code panel
  static constexpr int NP = D / PW;
  static constexpr int KV = BN * D;                   // bytes of a tile of key (or value) codes
  static constexpr int Q = 2 * 128 * D;               // both terms of a row tile
  static constexpr int VF = 2 * KV;                   // values in fp16
  static constexpr int VPANEL = BN * 128;             // 64 dims of all keys
  static constexpr int KS = D == 64 ? 4 : 3, VS = 2, FS = 2;
  static constexpr int SB = MT == 1 ? 2 : 1;          // score buffers a row tile
  static constexpr int OCOL = MT * SB * BN;           // TMEM column of the outputs
  static constexpr int SMEM = 1024 + MT * Q + KS * KV + VS * KV + FS * VF + 8192;
  static_assert(SMEM <= 232448 && OCOL + MT * D <= 512, "shared and tensor memory");
};

struct StepMeta {
  float ks[8], lvs[8], ivs[8];  // scale, log2 and reciprocal (times kUnbias) of the value scale of each 16 keys; ks 0: hidden
  int cut, pad[7];              // some of its keys are hidden
};
// What the CTA works on.  It stays in shared memory: registers are for scores.
struct Block {
  int run, seq;                 // whether there is work; the sequence
  int tok0, rem0;               // the first row's token among the call's, and its query head
  float inv_g;                  // 1 / G
  int R, tiles;                 // rows of the block, row tiles in use
  int pos0, pos1;               // of its first and last row
  int n, first_key, key1;       // steps, the first one's first key; the end of the block's keys
};
// A row's token from the block's first one on: (rem0 + row) / G.  The quotient of numbers below 2^9 and the half
// is 2^-8 at least away from a whole number, so its rounding does no harm.
__device__ __forceinline__ int token_of(const Block& b, int row) { return (int)(((float)(b.rem0 + row) + 0.5f) * b.inv_g); }
template <int D>
struct Shared {
  using C = Cfg<D>;
  StepMeta step[8];
  uint64_t kfull[C::KS], kfree[C::KS], cfull[C::VS], cfree[C::VS], vfull[C::FS], vfree[C::FS];
  float other[2][C::MT][2][128];  // what the two threads of a row tell each other
  float rc[C::ROWS];              // a row's power of two * scale * log2(e)
  uint64_t qfull, sfull[C::MT * C::SB], pfull[C::MT * C::SB], odone[C::MT], ended;
  uint32_t tmem;
  Block b;
  int pos[C::ROWS];    // a row's position
  int2 edge[C::ROWS / 32];  // of 32 rows: the last key that all see, the last one that some do not see any more
  int ticket, poison;  // poison: a NaN value code was dropped
};

struct PrefillArgs {
  AttnArgs a;
  int splits;
  int* counters;    // [blocks * hkv]
  float2* part_ml;  // [blocks * hkv * splits][ROWS]
  float* part_o;    // [blocks * hkv * splits][ROWS][D]
};

constexpr uint32_t idesc_f16(int n) {  // f16 x f16 -> fp32, M = 128, B N-contiguous
  return (1u << 4) | (1u << 16) | ((uint32_t)(n >> 3) << 17) | (8u << 24);
}
template <uint32_t BHI, uint32_t IDESC>
__device__ __forceinline__ void mma_f16_ts(uint32_t d, uint32_t a, uint32_t blo, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 db;\n\tsetp.ne.b32 p, %5, 0;\n\tmov.b64 db, {%2, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %4, p;\n\t}" ::"r"(d), "r"(a), "r"(blo), "n"(BHI), "n"(IDESC),
      "r"(acc)
      : "memory");
}

// Barrier of the 256 softmax threads of a row tile that returns whether any thread's v is set.
__device__ __forceinline__ bool any_of_pair(int tile, bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %2, 0;\n\tbarrier.cta.red.or.pred q, %1, 256, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(1 + tile), "r"((uint32_t)v)
      : "memory");
  return r != 0;
}

template <int D>
__global__ void __launch_bounds__(Cfg<D>::THREADS, 1)
    attn_prefill_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                        const PrefillArgs pa) {
  using C = Cfg<D>;
  constexpr int MT = C::MT, BN = C::BN;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* qbuf = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* kring = qbuf + MT * C::Q;
  uint8_t* cring = kring + C::KS * C::KV;
  uint8_t* vring = cring + C::VS * C::KV;
  Shared<D>& sh = *reinterpret_cast<Shared<D>*>(vring + C::FS * C::VF);
  static_assert(sizeof(Shared<D>) <= 8192, "shared memory");
  const AttnArgs& a = pa.a;
  const KvArgs& c = a.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tid = threadIdx.x & 127;
  const int G = a.hq / c.hkv;
  constexpr int kConv = 8 * MT, kMma = kConv + 4;  // first warps of the converters' and the last warpgroup

  // all heads and splits of a row block before the next block
  const int wide = c.hkv * pa.splits, block = blockIdx.x / wide, head = blockIdx.x % wide / pa.splits;
  const int split = blockIdx.x % pa.splits;

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::KS; ++i) mbar_init(&sh.kfull[i], 9), mbar_init(&sh.kfree[i], 1);
    for (int i = 0; i < C::VS; ++i) mbar_init(&sh.cfull[i], 8), mbar_init(&sh.cfree[i], 4);
    for (int i = 0; i < C::FS; ++i) mbar_init(&sh.vfull[i], 4), mbar_init(&sh.vfree[i], 1);
    for (int i = 0; i < MT * C::SB; ++i) mbar_init(&sh.sfull[i], 2), mbar_init(&sh.pfull[i], 8);
    for (int i = 0; i < MT; ++i) mbar_init(&sh.odone[i], 1);
    mbar_init(&sh.qfull, C::SOFT / 32);
    mbar_init(&sh.ended, 1);
    sh.poison = 0;
    fence_mbar_init();
  }
  if (warp == kMma) {
    tmem_alloc(&sh.tmem, 512);
    tmem_relinquish();
  }
  pdl_launch_dependents();
  pdl_wait();
  // this CTA's row block: the blocks of all sequences in a row, the last ones (with the most keys) first
  if (warp == 0) {
    bool bad = false;
    int total = 0;
    Seq s = {0, 0, 0};
    auto blocks_of = [&](const Seq& s) { return (int)(((int64_t)s.rows * G + C::ROWS - 1) / C::ROWS); };
    for (int base = 0; base < c.n_seqs; base += 32) {
      s = {0, 0, 0};
      if (base + lane < c.n_seqs) s = seq_of(c, base + lane, &bad);
      total += __reduce_add_sync(0xFFFFFFFFu, blocks_of(s));
    }
    if (bad && blockIdx.x == 0) atomicMax(c.status, kStatusInvalid);
    int left = total - 1 - block;
    int ok = left >= 0;
    for (int base = 0; ok && base < c.n_seqs; base += 32) {
      bool ignore = false;
      if (c.n_seqs > 32) {  // (up to 32 are here already)
        s = {0, 0, 0};
        if (base + lane < c.n_seqs) s = seq_of(c, base + lane, &ignore);
      }
      const int nb = blocks_of(s);
      int sum = nb;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xFFFFFFFFu, sum, o);
        if (lane >= o) sum += v;
      }
      const int all = __shfl_sync(0xFFFFFFFFu, sum, 31);
      if (left < all) {
        const int who = __ffs(__ballot_sync(0xFFFFFFFFu, sum > left)) - 1;
        if (lane == who) {
          Block& b = sh.b;
          const int64_t row0 = (int64_t)(left - (sum - nb)) * C::ROWS;
          const int first = row0 >> 32 ? (int)(row0 / G) : (int)((uint32_t)row0 / (uint32_t)G);  // (64-bit division is long)
          b.seq = base + who;
          b.R = (int)min((int64_t)C::ROWS, (int64_t)s.rows * G - row0);
          b.tiles = MT == 2 && b.R <= 128 ? 1 : MT;
          b.tok0 = s.start + first;
          b.rem0 = (int)(row0 - (int64_t)first * G);
          b.inv_g = 1.0f / (float)G;
          // its keys: from the first one that its first row sees (a whole page) to its last row's own
          b.pos0 = s.len - s.rows + first;
          b.pos1 = b.pos0 + (b.rem0 + b.R - 1) / G;
          const int key0 = b.pos0 >= a.window ? (b.pos0 - a.window + 1) >> c.page_log2 << c.page_log2 : 0;
          b.key1 = max(b.pos1 + 1, 0);
          const int steps = b.key1 > key0 ? (b.key1 - key0 + BN - 1) / BN : 0;
          const int s0 = steps * split / pa.splits, s1 = steps * (split + 1) / pa.splits;  // (below 2^25 steps, 32 splits)
          b.n = s1 - s0;
          b.first_key = key0 + s0 * BN;
        }
        break;
      }
      left -= all;
    }
    if (lane == 0) {
      sh.b.run = ok;
      if (!ok) sh.b.n = 0;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  const Block& b = sh.b;
  const bool run = b.run != 0;
  const int n = b.n;

  if (warp >= kConv) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::RREST));
    if (run && warp == kMma + 1) {  // --------------------------------------------------------- tiles of codes
      // Lane g looks after keys 16g .. of a step (g < BN / 16); page ids come two steps ahead, scales one.
      constexpr int NG = BN / 16;
      const int P = 1 << c.page_log2, box = min(P, BN), seq = b.seq, first_key = b.first_key, key1 = b.key1;
      auto page_of = [&](int i) {
        const int64_t tok = (int64_t)first_key + (int64_t)i * BN + 16 * lane;
        return i < n && lane < NG && tok < key1 ? c.pages[(int64_t)seq * c.page_stride + (tok >> c.page_log2)] : -1;
      };
      int id = page_of(0), id1 = page_of(1);
      bool dead = false;
      int ks = 0, vs = 0, klap = 0, vlap = 0;
      int i = 0;
      for (; i < n; ++i) {
        const int tok = first_key + i * BN + 16 * lane, id2 = page_of(i + 2);
        bool ok = lane < NG && tok < key1;
        if (ok && (id < 0 || id >= c.n_pages)) {
          ok = false;
          atomicMax(c.status, kStatusInvalid);
        }
        const int64_t tile = (int64_t)id * c.hkv + head;
        float sk = 0.0f, sv = 0.0f;
        if (ok) {
          sk = c.ks[tile];
          sv = c.vs[tile];
        }
        const bool lead = ok && (16 * lane) % box == 0;
        if (klap && !wait(&sh.kfree[ks], (klap - 1) & 1, c.status)) dead = true;
        if (__any_sync(0xFFFFFFFFu, dead)) break;
        if (lane < NG || lane < 8) {
          if (lead) {
            mbar_arrive_expect_tx(&sh.kfull[ks], box * D);
#pragma unroll
            for (int x = 0; x < C::NP; ++x)
              tma_load_3d(kring + ks * C::KV + x * BN * C::PW + 16 * lane * C::PW, &kmap, x * 128, tok & (P - 1), (int)tile,
                          &sh.kfull[ks]);
          } else if (lane < 8) {
            mbar_arrive(&sh.kfull[ks]);
          }
        }
        if (vlap && !wait(&sh.cfree[vs], (vlap - 1) & 1, c.status)) dead = true;
        if (__any_sync(0xFFFFFFFFu, dead)) {
          ++i;  // this step's keys are on their way
          break;
        }
        // the step's description goes with the value codes' barrier to the converters, and with the keys' to the rest
        StepMeta& m = sh.step[i & 7];
        const bool seen = ok && sk != 0.0f;
        const bool cut = __any_sync(0xFFFFFFFFu, lane < NG && (!seen || tok + 16 > key1));
        if (lane < NG) {
          m.ks[lane] = sk;
          m.lvs[lane] = seen ? lg2(sv) : 0.0f;
          m.ivs[lane] = seen ? rcp(sv) * kUnbias : 0.0f;
        }
        if (lane == 0) m.cut = cut;
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.kfull[ks]);
        if (lead) {
          mbar_arrive_expect_tx(&sh.cfull[vs], box * D);
#pragma unroll
          for (int x = 0; x < C::NP; ++x)
            tma_load_3d(cring + vs * C::KV + x * BN * C::PW + 16 * lane * C::PW, &vmap, x * 128, tok & (P - 1), (int)tile,
                        &sh.cfull[vs]);
        } else if (lane < 8) {
          mbar_arrive(&sh.cfull[vs]);
        }
        __syncwarp();
        id = id1;
        id1 = id2;
        if (++ks == C::KS) ks = 0, ++klap;
        if (++vs == C::VS) vs = 0, ++vlap;
      }
      // no copy is left in flight into this CTA's shared memory when it ends
      if (!dead) {
        for (int j = max(0, i - C::KS); j < i; ++j) wait(&sh.kfull[j % C::KS], (uint32_t)(j / C::KS) & 1u, c.status);
        for (int j = max(0, i - C::VS); j < i; ++j) wait(&sh.cfull[j % C::VS], (uint32_t)(j / C::VS) & 1u, c.status);
      } else {
        const unsigned long long t0 = global_ns();  // a pipeline that gave up: any copy has landed long before
        while (global_ns() - t0 < 1000000ull) {
        }
      }
    } else if (run && warp == kMma) {  // ------------------------------------------------------ MMAs
      constexpr uint32_t kSwz = D == 64 ? 4 : 2, kHi = desc_hi(8 * C::PW, kSwz), kVHi = desc_hi(1024, 2);
      constexpr uint32_t kQk = idesc_e4m3(BN, 0, 0), kQl = idesc_e4m3(BN, 0, 0, true), kPv = idesc_f16(D);
      const uint32_t q0 = desc_lo(smem_u32(qbuf), 16), k0 = desc_lo(smem_u32(kring), 16);
      const uint32_t v0 = desc_lo(smem_u32(vring), C::VPANEL);
      const int tiles = b.tiles;
      int ks = 0, fs = 0;
      uint32_t kpar = 0, vpar = 0;
      auto scores = [&](int m, int sb) {
        if (elect()) {
          const uint32_t d = tmem + (m * C::SB + sb) * BN;
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int x = 0; x < D / 32; ++x) {
              const uint32_t panel = x * 32 / C::PW, off = x * 32 % C::PW;
              const uint32_t qa = q0 + (m * C::Q + t * 128 * D + panel * 128 * C::PW + off) / 16;
              const uint32_t ka = k0 + (ks * C::KV + panel * BN * C::PW + off) / 16;
              if (t == 0)
                mma_e4m3<kHi, kHi, kQk>(d, qa, ka, x > 0);
              else
                mma_e4m3<kHi, kHi, kQl>(d, qa, ka, 1);
            }
          mma_commit(&sh.sfull[m * C::SB + sb]);
          mbar_arrive(&sh.sfull[m * C::SB + sb]);  // passes the step's description on
          if (m == tiles - 1) mma_commit(&sh.kfree[ks]);
        }
        __syncwarp();
      };
      auto outputs = [&](int m, int sb, int i) {
        if (elect()) {
          const uint32_t p = tmem + (m * C::SB + sb) * BN, d = tmem + C::OCOL + m * D;
#pragma unroll
          for (int x = 0; x < BN / 16; ++x)
            mma_f16_ts<kVHi, kPv>(d, p + (x < BN / 32 ? 8 * x : BN / 2 + 8 * (x - BN / 32)), 
                                  v0 + (fs * C::VF + x * 16 * 128) / 16, (i > 0) | (x > 0));
          if (m == tiles - 1) mma_commit(&sh.vfree[fs]);
          if (i == n - 1) mma_commit(&sh.odone[m]);
        }
        __syncwarp();
      };
      bool ok = __all_sync(0xFFFFFFFFu, n == 0 || wait(&sh.qfull, 0, c.status));
      // Step i's outputs and step i + 1's scores; in a turn before the first, only scores (of one tile, a copy of the loop's
      // code would have to be fetched anew).
      for (int i = -1; i < n && ok; ++i) {
        const bool more = i + 1 < n;
        if (more) ok = wait(&sh.kfull[ks], kpar, c.status);
        if (MT == 1) {  // the next scores go to the other buffer, whose P has been multiplied by then
          ok = __all_sync(0xFFFFFFFFu, ok);
          if (!ok) break;
          tc_fence_after();
          if (more) scores(0, (i + 1) & 1);
        }
        if (i >= 0 && ok) ok = wait(&sh.vfull[fs], vpar, c.status);
        // of two tiles, P lies over the scores: multiply it, then the tile's next scores; the other tile's softmax meanwhile
        for (int m = 0; m < tiles; ++m) {
          const int sb = MT == 1 ? i & 1 : 0;
          if (i >= 0 && ok) ok = wait(&sh.pfull[m * C::SB + sb], (uint32_t)(MT == 1 ? i >> 1 : i) & 1u, c.status);
          ok = __all_sync(0xFFFFFFFFu, ok);
          if (!ok) break;
          tc_fence_after();
          if (i >= 0) outputs(m, sb, i);
          if (MT > 1 && more) scores(m, 0);
        }
        if (more && ++ks == C::KS) ks = 0, kpar ^= 1;
        if (i >= 0 && ++fs == C::FS) fs = 0, vpar ^= 1;
      }
      // every MMA has ended before the CTA's memory goes
      if (elect()) {
        mma_commit(&sh.ended);
        wait(&sh.ended, 0, c.status);
      }
      __syncwarp();
    } else if (run && warp >= kConv && warp < kMma) {  // ------------------------------------ value codes -> fp16
      // a key a thread (two threads a key where there are 64)
      constexpr int TPK = 128 / BN, CH = D / 16 / TPK;  // chunks of 16 codes a thread
      const int key = tid % BN, part = tid / BN;
      const int first_key = b.first_key, key1 = b.key1;
      const int all0 = max(b.pos1, -1) - a.window + 1, all1 = b.pos0;  // all rows see all0 .. all1
      bool dead = false;
      int vs = 0, fs = 0;
      uint32_t cpar = 0, fpar = 1;
      if (n > 0 && !wait(&sh.qfull, 0, c.status)) dead = true;  // the queries have been read from the ring
      for (int i = 0; i < n; ++i) {
        if (!wait(&sh.cfull[vs], cpar, c.status)) dead = true;
        if (i >= C::FS && !dead && !wait(&sh.vfree[fs], fpar, c.status)) dead = true;
        if (__any_sync(0xFFFFFFFFu, dead)) break;
        const uint8_t* src = cring + vs * C::KV;
        uint8_t* dst = vring + fs * C::VF;
        // keys that nobody may see hold anything, NaN codes too: they must be numbers for P = 0
        const int t = first_key + i * BN + key;
        const bool real = t < key1 && sh.step[i & 7].ks[key >> 4] != 0.0f;
        if (__any_sync(0xFFFFFFFFu, t > all1 || t < all0)) {  // keys that not all rows see
          bool found = false;
#pragma unroll 1
          for (int ch = part * CH; ch < (part + 1) * CH; ++ch) {
            uint4* at = reinterpret_cast<uint4*>(cring + vs * C::KV + ch / (C::PW / 16) * BN * C::PW + key * C::PW +
                                                 (D == 64 ? ch % 4 ^ ((key >> 1) & 3) : ch % 8 ^ (key & 7)) * 16);
            if (t > all1 || t < all0) *at = drop_nans(*at, &found);
          }
          if (found) sh.poison = 1;
          fence_proxy_async_smem();  // the next copy into this place comes after these writes
        }
#pragma unroll
        for (int x = 0; x < CH; ++x) {
          const int ch = part * CH + x, panel = ch / (C::PW / 16), cc = ch % (C::PW / 16);
          const int sw = D == 64 ? cc ^ ((key >> 1) & 3) : cc ^ (key & 7);
          uint4 w = *reinterpret_cast<const uint4*>(src + panel * BN * C::PW + key * C::PW + sw * 16);
          if (!real) w = make_uint4(0, 0, 0, 0);
          // 16 values: two 16-byte chunks of the 64-dim panel ch / 4
          uint8_t* row = dst + (ch / 4) * C::VPANEL + key * 128;
          const int c0 = (ch % 4) * 2;
          *reinterpret_cast<uint4*>(row + ((c0 ^ (key & 7)) << 4)) =
              make_uint4(codes_lo(w.x), codes_hi(w.x), codes_lo(w.y), codes_hi(w.y));
          *reinterpret_cast<uint4*>(row + (((c0 + 1) ^ (key & 7)) << 4)) =
              make_uint4(codes_lo(w.z), codes_hi(w.z), codes_lo(w.w), codes_hi(w.w));
        }
        fence_proxy_async_smem();
        warp_arrive(&sh.cfree[vs]);
        warp_arrive(&sh.vfull[fs]);
        if (++vs == C::VS) vs = 0, cpar ^= 1;
        if (++fs == C::FS) fs = 0, fpar ^= 1;
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::RSOFT));
    if (run) {  // -------------------------------------------------------------------------- softmax, two threads a row
      const int mt = warp >> 3, half = warp >> 2 & 1, wq = warp & 3;
      const int row = mt * 128 + tid;  // in the block
      const uint32_t lane_base = (uint32_t)(32 * wq) << 16;
      if (n > 0) {  // the query rows as two 8-bit terms: D / 16 lanes a row
        // They come by way of the converted values' ring, which nobody needs yet, all at once, and their terms are made in a
        // loop that is not unrolled: what runs once runs as fast as its instructions arrive.
        constexpr int TPR = D / 16, RPP = C::SOFT / TPR, PASSES = C::ROWS / RPP;
        static_assert(C::ROWS * D * 2 <= C::FS * C::VF, "queries fit");
        const int part = threadIdx.x % TPR;
        uint8_t* raw = vring + threadIdx.x * 32;
#pragma unroll 1
        for (int y = 0; y < PASSES; ++y) {
          const int qr = y * RPP + threadIdx.x / TPR, qt = token_of(b, qr), qg = b.rem0 + qr - qt * G;
          const bool in = qr < b.R;
          const uint16_t* qp = a.q + (in ? (int64_t)(b.tok0 + qt) * a.ldq + (int64_t)(head * G + qg) * a.hsq + 16 * part : 0);
          cp_async16(raw + y * C::SOFT * 32, qp, in ? 16 : 0);
          cp_async16(raw + y * C::SOFT * 32 + 16, qp + (in ? 8 : 0), in ? 16 : 0);
        }
        if (half == 0) {
          const int pos = max(row < b.R ? b.pos0 + token_of(b, row) : b.pos1, -1);
          sh.pos[row] = pos;
          // rows ascend, so the warp's first row sees the fewest keys, its last row's window begins last
          const int see = __shfl_sync(0xFFFFFFFFu, pos, 0), skip = __reduce_max_sync(0xFFFFFFFFu, pos) - a.window;
          if (lane == 0) sh.edge[4 * mt + wq] = make_int2(see, skip);
        }
        cp_async_wait_all();  // (a thread reads what it has copied itself)
#pragma unroll 1
        for (int y = 0; y < PASSES; ++y) {
          const int qr = y * RPP + threadIdx.x / TPR;
          const uint4* src = reinterpret_cast<const uint4*>(raw + y * C::SOFT * 32);
          const uint4 v[2] = {src[0], src[1]};
          float amax = query_max(v);
#pragma unroll
          for (int o = TPR / 2; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
          // a power of two that brings the row's largest element to [128, 256)
          const int e2 = min(max((__float_as_int(amax) >> 23) - 127 - 7, -125), 125);
          uint4 hi, lo;
          split_query<true>(v, query_down(amax, e2), &hi, &lo);
          const int panel = part / (C::PW / 16), cc = part % (C::PW / 16);
          const int sw = D == 64 ? cc ^ ((qr >> 1) & 3) : cc ^ (qr & 7);
          uint8_t* at = qbuf + qr / 128 * C::Q + panel * 128 * C::PW + qr % 128 * C::PW + sw * 16;
          *reinterpret_cast<uint4*>(at) = hi;
          *reinterpret_cast<uint4*>(at + 128 * D) = lo;
          if (part == 0) sh.rc[qr] = __int_as_float((127 + e2) << 23) * (a.scale * kLog2e);
        }
        fence_proxy_async_smem();
        warp_arrive(&sh.qfull);
      }
      float m = -INFINITY, l = 0.0f;
      bool dead = false;
      constexpr int GH = BN / 32;  // groups of 16 keys of this thread's half
      const uint32_t ot = tmem + lane_base + C::OCOL + mt * D + half * (D / 2);
      const int mine = mt < b.tiles ? n : 0;
      for (int i = 0; i < mine; ++i) {
        const int sb = MT == 1 ? i & 1 : 0, buf = mt * C::SB + sb;
        if (!wait(&sh.sfull[buf], (MT == 1 ? i >> 1 : i) & 1, c.status)) dead = true;
        tc_fence_after();
        const StepMeta& sm = sh.step[i & 7];
        const uint32_t st = tmem + lane_base + buf * BN + half * (BN / 2);
        const int t0 = b.first_key + i * BN + half * (BN / 2), g0 = half * GH;
        const int2 edge = sh.edge[4 * mt + wq];
        const bool masked = sm.cut || t0 + BN / 2 - 1 > edge.x || t0 <= edge.y;
        const float rc = sh.rc[row];
        // this thread's scores, read once; masked ones are -inf
        uint32_t s[16 * GH];
        tmem_ld_now(st, s);
        if (masked) {
          asm volatile("" ::: "memory");  // a branch: as predicates the masks took a third of every step's time
          const int pos = sh.pos[row], last = pos - t0, first = max(pos - a.window + 1, 0) - t0;  // of this half, seen
#pragma unroll
          for (int w = 0; w < GH / 2; ++w) {  // 32 keys, a bit each
            const int u = last - 32 * w, v = first - 32 * w;
            uint32_t keep = (u < 0 ? 0u : u > 30 ? ~0u : (2u << u) - 1u) & (v > 31 ? 0u : ~0u << max(v, 0));
            if (sm.ks[g0 + 2 * w] == 0.0f) keep &= 0xFFFF0000u;
            if (sm.ks[g0 + 2 * w + 1] == 0.0f) keep &= 0xFFFFu;
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (!(keep >> e & 1)) s[32 * w + e] = 0xFF800000u;
          }
        }
        // the row's largest t
        float top = -INFINITY;
#pragma unroll
        for (int gr = 0; gr < GH; ++gr) {
          auto at = [&](int e) { return __uint_as_float(s[16 * gr + e]); };
          float m0 = max3(at(0), at(1), at(2)), m1 = max3(at(3), at(4), at(5));
          m0 = max3(m0, at(6), at(7));
          m1 = max3(m1, at(8), at(9));
          m0 = max3(m0, at(10), at(11));
          m1 = max3(m1, at(12), at(13));
          // (a factor above 0, so that a masked score stays -inf)
          top = fmaxf(top, fmaf(fmaxf(max3(m0, at(14), at(15)), m1), fmaxf(rc * sm.ks[g0 + gr], 0x1p-126f), sm.lvs[g0 + gr]));
        }
        float(&other)[2][128] = sh.other[i & 1][mt];
        other[half][tid] = top;
        dead = any_of_pair(mt, dead);
        if (dead) break;
        top = fmaxf(top, other[half ^ 1][tid]);
        const bool grow = top > m + kLazy || (m == -INFINITY && top != -INFINITY);
        if (__any_sync(0xFFFFFFFFu, grow)) {
          const float w = grow ? ex2(m - top) : 1.0f;
          if (grow) m = top;
          l *= w;
          if (i > 0) {
            // (heads of 256: the product before may still run)
            if (MT == 1 && !wait(&sh.vfree[(i - 1) % C::FS], (uint32_t)((i - 1) / C::FS) & 1u, c.status)) dead = true;
            tc_fence_after();
#pragma unroll 1
            for (int x = 0; x < D / 2; x += 16) {
              uint32_t o[16];
              tmem_ld16(ot + x, o);
              tmem_ld_wait16(o);
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * w);
              tmem_st16(ot + x, o);
            }
            tmem_st_wait();
          }
        }
        const float ref = (m == -INFINITY ? 0.0f : m) - kBias;
        // two groups at a time
#pragma unroll
        for (int gr = 0; gr < GH; gr += 2) {
          uint64_t t[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const int x = gr + e / 8;
            const float off = sm.lvs[g0 + x] - ref, f = fmaxf(rc * sm.ks[g0 + x], 0x1p-126f);
            const uint64_t y = pack2(__uint_as_float(s[16 * gr + 2 * e]), __uint_as_float(s[16 * gr + 2 * e + 1]));
            t[e] = fma2(y, pack2(f, f), pack2(off, off));
          }
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            float t0, t1;
            unpack2(t[e], &t0, &t1);
            t[e] = pack2(ex2(t0), ex2(t1));
          }
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            uint32_t p[8];
            float p0, p1;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              unpack2(t[8 * x + e], &p0, &p1);
              p[e] = f16x2(p0, p1);
            }
            tmem_st8(st + 8 * (gr + x), p);  // over the scores of this half
#pragma unroll
            for (int w = 4; w; w >>= 1)
#pragma unroll
              for (int e = 0; e < w; ++e) t[8 * x + e] = add2(t[8 * x + e], t[8 * x + e + w]);
            unpack2(t[8 * x], &p0, &p1);
            l = fmaf(p0 + p1, sm.ivs[g0 + gr + x], l);
          }
        }
        tmem_st_wait();
        tc_fence_before();
        warp_arrive(&sh.pfull[buf]);
      }
      if (mine > 0 && !dead && !wait(&sh.odone[mt], 0, c.status)) dead = true;
      if (mt < b.tiles) {
        float(&other)[2][128] = sh.other[n & 1][mt];
        other[half][tid] = l;
        dead = any_of_pair(mt, dead);
        l += other[half ^ 1][tid];
        tc_fence_after();
      }
      if (!dead && mt < b.tiles) {
        // A warp's rows go by way of shared memory (the queries are done with), so that lanes side by side write one row: a
        // 16-byte piece of a row from each lane took 9300 cycles from here to the CTA's end, this 6000 (heads of 128).
        const bool in = row < b.R, parts = pa.splits > 1;
        const int tok = token_of(b, row), g = b.rem0 + row - tok * G;
        const float inv = parts ? 1.0f : l == 0.0f ? 0.0f : kUnbias / l;
        const int64_t part = blockIdx.x;  // of (block, head), split by split
        const bool poison = sh.poison;
        const int64_t at = parts ? ((part * C::ROWS + row) * D + half * (D / 2)) * 4
                                 : ((int64_t)(b.tok0 + tok) * a.ldo + (int64_t)(head * G + g) * a.hso + half * (D / 2)) * 2;
        uint8_t* base = parts ? reinterpret_cast<uint8_t*>(pa.part_o) : reinterpret_cast<uint8_t*>(a.out);
        constexpr int CPR = D / 16;  // pieces of a row in a warp's D * 32 bytes
        uint8_t* stage = qbuf + mt * C::Q + (warp & 7) * (C::Q / 8);
        auto piece = [&](int r, int k) {
          return reinterpret_cast<uint4*>(stage + r * D + ((k ^ (D == 64 ? r >> 1 & 3 : r & 7)) << 4));
        };
        const int dims = parts ? D / 4 : D / 2;  // in a warp's bytes at a time
#pragma unroll 1
        for (int x0 = 0; x0 < D / 2; x0 += dims) {
#pragma unroll 1
          for (int x = x0; x < x0 + dims; x += 16) {
            uint32_t o[16];
            if (n > 0) {
              tmem_ld16(ot + x, o);
              tmem_ld_wait16(o);
            } else {
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = 0u;
            }
            if (poison && in) {
              const uint32_t nans = nan_dims(c, c.pages + (int64_t)b.seq * c.page_stride, head, D, half * (D / 2) + x,
                                             sh.pos[row], a.window, max(b.pos1, -1) - a.window + 1, b.pos0);
#pragma unroll
              for (int e = 0; e < 16; ++e)
                if (nans >> e & 1) o[e] = 0x7FFFFFFFu;
            }
            if (parts) {
#pragma unroll
              for (int e = 0; e < 4; ++e)
                *piece(lane, (x - x0) / 4 + e) = make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
            } else {
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                uint32_t y[4];
#pragma unroll
                for (int z = 0; z < 4; ++z)
                  y[z] = bf16x2(__uint_as_float(o[8 * e + 2 * z]) * inv, __uint_as_float(o[8 * e + 2 * z + 1]) * inv);
                *piece(lane, x / 8 + e) = make_uint4(y[0], y[1], y[2], y[3]);
              }
            }
          }
          __syncwarp();
          const int xb = x0 * 4;  // (0 where the outputs go out at once)
#pragma unroll 2
          for (int e = 0; e < CPR; ++e) {
            const int r = e * (32 / CPR) + lane / CPR, k = lane % CPR;
            const int64_t to = __shfl_sync(0xFFFFFFFFu, at, r) + xb + 16 * k;
            const uint4 v = *piece(r, k);
            if (mt * 128 + wq * 32 + r < b.R) *reinterpret_cast<uint4*>(base + to) = v;
          }
          __syncwarp();
        }
        if (in && half == 0 && pa.splits > 1) pa.part_ml[part * C::ROWS + row] = make_float2(m, l);
      }
      tc_fence_before();
    }
  }
  __syncthreads();
  if (warp == kMma) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (!run || pa.splits == 1) return;
  // the CTA whose ticket completes the block joins its parts, in order
  int* counter = pa.counters + blockIdx.x / pa.splits;
  if (threadIdx.x == 0) sh.ticket = ticket_add(counter, 1);
  __syncthreads();
  if (sh.ticket != pa.splits - 1) return;
  const int64_t part0 = blockIdx.x / pa.splits * pa.splits;
  const int R = b.R, tok0 = b.tok0;
  for (int e = threadIdx.x; e < R * (D / 8); e += C::THREADS) {
    const int row = e / (D / 8), d = e % (D / 8) * 8;
    float top = -INFINITY, l = 0.0f, o[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    for (int s = 0; s < pa.splits; ++s) top = fmaxf(top, __ldcg(&pa.part_ml[(part0 + s) * C::ROWS + row]).x);
#pragma unroll 2
    for (int s = 0; s < pa.splits; ++s) {
      const float2 z = __ldcg(&pa.part_ml[(part0 + s) * C::ROWS + row]);
      const float4* src = reinterpret_cast<const float4*>(pa.part_o + ((part0 + s) * C::ROWS + row) * D + d);
      const float4 y0 = __ldcg(src), y1 = __ldcg(src + 1);
      const float f = z.x == -INFINITY ? 0.0f : ex2(z.x - top);
      const float y[8] = {y0.x, y0.y, y0.z, y0.w, y1.x, y1.y, y1.z, y1.w};
#pragma unroll
      for (int k = 0; k < 8; ++k) o[k] = fmaf(y[k], f, o[k]);
      l = fmaf(z.y, f, l);
    }
    const float inv = l == 0.0f ? 0.0f : kUnbias / l;
    const int tok = token_of(b, row), g = b.rem0 + row - tok * G;
    *reinterpret_cast<uint4*>(a.out + (int64_t)(tok0 + tok) * a.ldo + (int64_t)(head * G + g) * a.hso + d) =
        make_uint4(bf16x2(o[0] * inv, o[1] * inv), bf16x2(o[2] * inv, o[3] * inv), bf16x2(o[4] * inv, o[5] * inv),
                   bf16x2(o[6] * inv, o[7] * inv));
  }
  if (threadIdx.x == 0) *counter = 0;
}

// Parts along the keys of each of `items` blocks of some `keys` keys.  The CTAs come in waves of one an SM; a CTA takes
// its keys' time and that of 640 more for its start and end, of 800 where it writes a part, and each part of a block
// costs 160 in the join: the number with the shortest sum is taken.  (Measured: 96 items of 33280 keys 531 us whole, 394
// in three parts, 436 in six; 152 of 8192 138 whole, 164 in two; 48 of 16384 111 in three, 125 in six; 40 of 4096 36 in
// three, 48 in four or more; 8 of 2048 38 in two, 34 in four, 42 in eight; 20 of 2000 45 whole, 38 in three, 46 in seven.)
int choose_splits(int64_t items, int64_t keys, int sms) {
  if (items > (int64_t)(kAttnCounterBytes / sizeof(int))) return 1;
  int best = 1;
  int64_t least = INT64_MAX;
  for (int s = 1; s <= 32 && (s == 1 || keys / s >= 256); ++s) {
    const int64_t cost = (items * s + sms - 1) / sms * (keys / s + (s > 1 ? 800 : 640)) + (s > 1 ? 160 * s : 0);
    if (cost < least) best = s, least = cost;
  }
  return best;
}

template <int D>
int launch(const AttnArgs& a, const PrefillPlan& p, void* ws, cudaStream_t s) {
  using C = Cfg<D>;
  static std::atomic<unsigned long long> configured{0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return QG_ERR_CUDA;
  const unsigned long long bit = 1ull << (dev & 63);
  if (!(configured.load() & bit)) {
    if (cudaFuncSetAttribute((const void*)attn_prefill_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM) !=
        cudaSuccess)
      return QG_ERR_CUDA;
    configured.fetch_or(bit);
  }
  const int page = 1 << a.c.page_log2, box = std::min(page, C::BN);
  CUtensorMap km, vm;
  if (!encode_pages(&km, a.c.k, D, page, a.c.n_pages * a.c.hkv, box) ||
      !encode_pages(&vm, a.c.v, D, page, a.c.n_pages * a.c.hkv, box))
    return QG_ERR_CUDA;
  // a window leaves a block fewer keys than the plan, which does not know it, has counted on
  DeviceInfo info;
  if (!current_device_info(&info)) return QG_ERR_CUDA;
  const int64_t keys = std::min<int64_t>(a.c.max_len, (int64_t)a.window + C::ROWS / (a.hq / a.c.hkv) + page);
  const int splits = std::min(p.splits, choose_splits(p.blocks * a.c.hkv, keys, info.sms));
  PrefillArgs pa;
  pa.a = a;
  pa.splits = splits;
  uint8_t* w = static_cast<uint8_t*>(ws);
  pa.counters = reinterpret_cast<int*>(w + kWsHeader);
  pa.part_ml = reinterpret_cast<float2*>(w + p.off_ml);
  pa.part_o = reinterpret_cast<float*>(w + p.off_o);
  return launch_pdl(attn_prefill_kernel<D>, dim3((unsigned)(p.blocks * a.c.hkv * splits)), dim3(C::THREADS),
                    C::SMEM, s, km, vm, pa) == cudaSuccess
             ? QG_OK
             : QG_ERR_CUDA;
}

}  // namespace

bool plan_prefill(const qg_kv_cache* cache, const qg_kv_batch* batch, int64_t n_tokens, int hq, const DeviceInfo& dev,
                  PrefillPlan* p) {
  const int64_t G = hq / cache->n_kv_heads, rows = cache->head_dim == 256 ? 128 : 256;
  const int64_t each = (batch->max_new * G + rows - 1) / rows;
  // a sequence of t tokens has at most t * G / rows + 1 blocks
  p->blocks = std::min<int64_t>(each * batch->n_seqs, n_tokens * G / rows + batch->n_seqs);
  const int64_t items = p->blocks * cache->n_kv_heads;
  if (items > 0x7FFFFFFF / 32) return false;
  const int s = choose_splits(items, batch->max_len, dev.sms);
  p->splits = s;
  p->off_ml = kWsHeader + kAttnCounterBytes;
  p->off_o = p->off_ml;
  p->ws_bytes = p->off_ml;
  if (s > 1) {
    p->off_o = p->off_ml + (size_t)(items * s * rows) * sizeof(float2);
    p->ws_bytes = p->off_o + (size_t)(items * s * rows) * cache->head_dim * sizeof(float);
  }
  return true;
}

int launch_attn_prefill(const AttnArgs& a, int head_dim, const PrefillPlan& p, void* ws, void* stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  switch (head_dim) {
    case 64: return launch<64>(a, p, ws, s);
    case 128: return launch<128>(a, p, ws, s);
    case 256: return launch<256>(a, p, ws, s);
  }
  return QG_ERR_UNSUPPORTED;
}

}  // namespace qg
