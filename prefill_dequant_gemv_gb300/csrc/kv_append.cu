// Norm, rotate and append: what runs between a QKV projection and the attention (TurboEXL3
// article §4.3: QK-norm and partial rotary fused behind the projection).  One launch:
//   queries: y = x * r * (w + offset), r = 1/sqrt(mean(x^2) + eps), rotated, rounded to bf16;
//   keys:    the same, then E4M3 codes under the scale of their (page, KV head);
//   values:  E4M3 codes under theirs.
//
// A head of D elements lies across D/8 lanes, eight elements each in two runs of four that hold both
// elements of a rotation's pairs: 4l .. and R/2 + 4l .. (pairs R/2 apart), or 8l .. (neighbours).  So the norm's
// sum is the only thing that crosses lanes, and a lane needs four angles.
//
// Keys and values are worked on by unit = (page, KV head, K or V): the page's scale depends on all
// its new tokens, so one group of threads owns them, holds the normed values in registers
// while it reduces their largest magnitude, and stores the codes; a page's scale has one
// writer and no atomics.  A group is one warp for up to four new tokens a sequence (decode:
// eight units a block, no block barrier) and a whole block for prompts.
// The scale is a power of two: dividing by it is exact, so each code is its value rounded once,
// and a later, larger scale moves the codes' exponents only.
//
// Bound by HBM: bf16 in, bf16 and bytes out.  Measured (GB300): 4096 tokens of 40/8 heads of 128: 28 us, 4.0 TB/s; seven
// prompts of up to 1201 tokens, 24/4 heads of 256, pages of 16: 34 us, 3.9 TB/s; one token 7.1 us, 64 sequences of one 7.5 us,
// which is the host's call, the launch and three dependent loads.  The long calls are about half issue (57% of the slots: the
// norms' and codes' arithmetic, 17 M warp instructions) and half waiting for their one round of loads: a unit's values are held
// in registers until its scale is known, so its block has no next loads to send meanwhile.  The queries, 77% of the bytes
// at 40/8 heads, need no scale; their blocks could, and do not.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "qg_attn.h"
#include "qg_sync.cuh"

namespace qg {
namespace {

constexpr int kAppendThreads = 256;
constexpr int kQHeads = 4;       // heads of one token a query lane group takes: one position, one set of angles
constexpr int kWarpRows = 4;     // new tokens a sequence up to which a warp owns a unit

// Two floats -> two E4M3 codes (a in the low byte), nearest even, saturating; NaN stays NaN.
__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}
__device__ __forceinline__ float e4m3_value(uint32_t code) {
  __nv_fp8_e4m3 v;
  v.__x = (uint8_t)code;
  return static_cast<float>(v);
}

// Two fp32 numbers in a register pair, worked on by one instruction.
struct F2 {
  float x, y;
};
__device__ __forceinline__ uint64_t pair(F2 v) { return (uint64_t)__float_as_uint(v.y) << 32 | __float_as_uint(v.x); }
__device__ __forceinline__ F2 unpair(uint64_t v) {
  return {__uint_as_float((uint32_t)v), __uint_as_float((uint32_t)(v >> 32))};
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(pair(a)), "l"(pair(b)));
  return unpair(d);
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(pair(a)), "l"(pair(b)), "l"(pair(c)));
  return unpair(d);
}
__device__ __forceinline__ void unpack8(uint2 v, uint2 w, F2 (&f)[4]) {
  const uint32_t u[4] = {v.x, v.y, w.x, w.y};
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = {__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xFFFF0000u)};
}
__device__ __forceinline__ uint32_t bf16x2(F2 v) {
  const __nv_bfloat162 r = __floats2bfloat162_rn(v.x, v.y);
  return *reinterpret_cast<const uint32_t*>(&r);
}

// The exponent x of the smallest power of two with amax <= 448 * 2^x (448 = 1.75 * 2^8),
// between -100 and 120, from amax's bits.
__device__ __forceinline__ int scale_exponent(float amax) {
  const int bits = __float_as_int(amax);
  const int x = (bits >> 23) - 127 - 8 + ((bits & 0x7FFFFF) > 0x600000 ? 1 : 0);
  return min(max(x, -100), 120);
}

// A lane's share of the norm and rotation of a head of LPH lanes: four elements from a on and four from b on.
template <int LPH>
struct NormRope {
  F2 w[4], c[2], s[2];
  float eps;
  int a, b;
  bool norm, inter, turn;  // turn: this lane's elements are rotated

  __device__ __forceinline__ void init(const uint16_t* weight, float off, float eps_, int rot, int interleaved, int l) {
    eps = eps_;
    inter = interleaved;
    turn = 8 * l < rot;
    a = turn && !inter ? 4 * l : 8 * l;
    b = turn && !inter ? rot / 2 + 4 * l : 8 * l + 4;
    norm = weight != nullptr;
    if (norm) {
      unpack8(__ldg(reinterpret_cast<const uint2*>(weight + a)), __ldg(reinterpret_cast<const uint2*>(weight + b)), w);
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i].x += off, w[i].y += off;
    }
  }
  __device__ __forceinline__ void angles(const float* cs, int rot, int64_t pos, int l) {
    if (turn) {
      const float4 x = __ldg(reinterpret_cast<const float4*>(cs + pos * rot + 4 * l));
      const float4 y = __ldg(reinterpret_cast<const float4*>(cs + pos * rot + rot / 2 + 4 * l));
      c[0] = {x.x, x.y}, c[1] = {x.z, x.w};
      s[0] = {y.x, y.y}, s[1] = {y.z, y.w};
    }
  }
  // every lane of the warp calls this
  __device__ __forceinline__ void apply(F2 (&y)[4]) const {
    if (norm) {
      F2 q = mul2(y[0], y[0]);
#pragma unroll
      for (int i = 1; i < 4; ++i) q = fma2(y[i], y[i], q);
      float ss = q.x + q.y;
#pragma unroll
      for (int o = LPH / 2; o; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
      const float r = rsqrtf(fmaf(ss, 1.0f / (8 * LPH), eps));
#pragma unroll
      for (int i = 0; i < 4; ++i) y[i] = mul2(mul2(y[i], {r, r}), w[i]);
    }
    if (!turn) return;
    if (inter) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float cc = i & 1 ? c[i / 2].y : c[i / 2].x, sn = i & 1 ? s[i / 2].y : s[i / 2].x;
        y[i] = {y[i].x * cc - y[i].y * sn, y[i].y * cc + y[i].x * sn};
      }
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const F2 u = y[i], v = y[2 + i];
        y[i] = fma2(v, {-s[i].x, -s[i].y}, mul2(u, c[i]));
        y[2 + i] = fma2(u, s[i], mul2(v, c[i]));
      }
    }
  }
};

// Sequence of row i: the last one that starts at or before it.
__device__ __forceinline__ int seq_of_row(const KvArgs& c, int64_t i) {
  int lo = 0, hi = c.n_seqs;  // q_start[lo] <= i
  while (hi - lo > 1) {
    const int m = (lo + hi) >> 1;
    if (c.q_start[m] <= i)
      lo = m;
    else
      hi = m;
  }
  return lo;
}

// The queries: a lane group takes kQHeads heads of one token, their loads issued together.
template <int LPH>
__device__ __forceinline__ void append_queries(const AppendArgs& a, uint32_t block) {
  constexpr int GROUPS = kAppendThreads / LPH;
  const int l = threadIdx.x % LPH;
  const uint32_t per = (uint32_t)(a.hq + kQHeads - 1) / kQHeads;
  const uint32_t item = block * GROUPS + threadIdx.x / LPH, row = item / per;
  const int h0 = (int)(item - row * per) * kQHeads;
  NormRope<LPH> nr;
  nr.init(a.qw, a.woff, a.eps, a.rot, a.interleaved, l);
  uint2 x[kQHeads][2];
  const bool in = row < a.c.n_tokens;
  const uint16_t* src = a.q + (int64_t)row * a.ldq + h0 * a.hsq;
#pragma unroll
  for (int p = 0; p < kQHeads; ++p, src += a.hsq) {
    x[p][0] = x[p][1] = make_uint2(0, 0);
    if (in && h0 + p < a.hq) {
      x[p][0] = *reinterpret_cast<const uint2*>(src + nr.a);
      x[p][1] = *reinterpret_cast<const uint2*>(src + nr.b);
    }
  }
  bool use = false;
  if (in) {
    bool bad = false;
    const Seq s = seq_of(a.c, seq_of_row(a.c, row), &bad);
    use = s.len >= s.rows && row >= (uint32_t)s.start && row < (uint32_t)(s.start + s.rows);
    if (use) nr.angles(a.cs, a.rot, (int64_t)s.len - s.rows + (int)(row - s.start), l);
  }
  uint16_t* dst = a.qo + (int64_t)row * a.ldo + h0 * a.hso;
#pragma unroll
  for (int p = 0; p < kQHeads; ++p, dst += a.hso) {
    F2 y[4];
    unpack8(x[p][0], x[p][1], y);
    nr.apply(y);
    if (use && h0 + p < a.hq) {
      *reinterpret_cast<uint2*>(dst + nr.a) = make_uint2(bf16x2(y[0]), bf16x2(y[1]));
      *reinterpret_cast<uint2*>(dst + nr.b) = make_uint2(bf16x2(y[2]), bf16x2(y[3]));
    }
  }
}

// Pages that hold new tokens of a sequence.
__device__ __forceinline__ int touched_pages(const Seq& s, int page_log2) {
  return s.rows > 0 && s.len >= s.rows ? ((s.len - 1) >> page_log2) - ((s.len - s.rows) >> page_log2) + 1 : 0;
}

// One unit: the new tokens of one page for one KV head, keys or values.
template <int LPH, int GT, int ITER>
__device__ __forceinline__ void append_unit(const AppendArgs& a, int64_t unit, int per_seq, bool scan, float* red) {
  constexpr int D = 8 * LPH, TPP = GT / LPH;  // tokens a pass
  const KvArgs& c = a.c;
  const int g = threadIdx.x % GT, l = g % LPH;
  const int64_t slot = unit / (2 * c.hkv);
  const int rest = (int)(unit - slot * (2 * c.hkv));
  const bool is_v = rest >= c.hkv;
  const int h = is_v ? rest - c.hkv : rest;

  // the slot's sequence and its page's place among the sequence's touched pages
  bool bad = false;
  Seq s = {0, 0, 0};
  int j = -1, b = 0;
  if (!scan) {
    b = (int)(slot / per_seq);
    if (b >= c.n_seqs) return;
    s = seq_of(c, b, &bad);
    j = (int)(slot - (int64_t)b * per_seq);
    if (s.len < s.rows) bad = true;
    if (j >= touched_pages(s, c.page_log2)) j = -1;
  } else {
    const int lane = threadIdx.x & 31;
    int64_t left = slot;
    for (int base = 0; base < c.n_seqs && j < 0; base += 32) {
      Seq t = {0, 0, 0};
      bool tb = false;
      if (base + lane < c.n_seqs) t = seq_of(c, base + lane, &tb);
      if (t.len < t.rows) tb = true;
      bad |= tb;
      const int n = touched_pages(t, c.page_log2);
      int sum = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xFFFFFFFFu, sum, o);
        if (lane >= o) sum += v;
      }
      const int total = __shfl_sync(0xFFFFFFFFu, sum, 31);
      if (left < total) {
        const int who = __ffs(__ballot_sync(0xFFFFFFFFu, sum > left)) - 1;
        b = base + who;
        j = (int)left - (__shfl_sync(0xFFFFFFFFu, sum, who) - __shfl_sync(0xFFFFFFFFu, n, who));
        s.start = __shfl_sync(0xFFFFFFFFu, t.start, who);
        s.rows = __shfl_sync(0xFFFFFFFFu, t.rows, who);
        s.len = __shfl_sync(0xFFFFFFFFu, t.len, who);
      } else {
        left -= total;
      }
    }
  }
  if (bad && c.status) atomicMax(c.status, kStatusInvalid);
  if (j < 0) return;
  const int P = 1 << c.page_log2, first = s.len - s.rows;
  const int pi = (first >> c.page_log2) + j;
  const int id = c.pages[(int64_t)b * c.page_stride + pi];
  if (id < 0 || id >= c.n_pages) {
    if (g == 0 && c.status) atomicMax(c.status, kStatusInvalid);
    return;
  }
  const int base = pi << c.page_log2;
  const int lo = max(first, base), hi = min(s.len, base + P), held = lo - base;
  float* scale_at = (is_v ? c.vs : c.ks) + (int64_t)id * c.hkv + h;
  uint8_t* tile = (is_v ? c.v : c.k) + (((int64_t)id * c.hkv + h) << c.page_log2) * D;
  const float old = held ? *scale_at : 0.0f;

  const uint16_t* src = is_v ? a.vin + (int64_t)h * a.hsv : a.kin + (int64_t)h * a.hsk;
  const int64_t ld = is_v ? a.ldv : a.ldk;
  NormRope<LPH> nr;
  nr.init(is_v ? nullptr : a.kw, a.woff, a.eps, is_v ? 0 : a.rot, a.interleaved, l);
  uint2 x[ITER][2];
#pragma unroll
  for (int i = 0; i < ITER; ++i) {
    const int t = lo + i * TPP + g / LPH;
    x[i][0] = x[i][1] = make_uint2(0, 0);
    if (t < hi) {
      const uint16_t* at = src + (int64_t)(s.start + (t - first)) * ld;
      x[i][0] = *reinterpret_cast<const uint2*>(at + nr.a);
      x[i][1] = *reinterpret_cast<const uint2*>(at + nr.b);
    }
  }
  F2 y[ITER][4];
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < ITER; ++i) {
    unpack8(x[i][0], x[i][1], y[i]);
    if (!is_v && lo + i * TPP < hi) {  // the same for the whole group
      nr.angles(a.cs, a.rot, min(lo + i * TPP + g / LPH, hi - 1), l);
      nr.apply(y[i]);
    }
    if (lo + i * TPP + g / LPH < hi) {
#pragma unroll
      for (int e = 0; e < 4; ++e) amax = fmaxf(amax, fmaxf(fabsf(y[i][e].x), fabsf(y[i][e].y)));  // NaN does not count
    }
  }
  if (amax == INFINITY) {  // nor do infinities
    amax = 0.0f;
#pragma unroll
    for (int i = 0; i < ITER; ++i)
      if (lo + i * TPP + g / LPH < hi)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float u = fabsf(y[i][e].x), v = fabsf(y[i][e].y);
          amax = fmaxf(amax, fmaxf(u < INFINITY ? u : 0.0f, v < INFINITY ? v : 0.0f));
        }
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
  if (GT > 32) {
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = amax;
    __syncthreads();
    amax = red[0];
#pragma unroll
    for (int i = 1; i < GT / 32; ++i) amax = fmaxf(amax, red[i]);
  }
  const float need = __int_as_float((scale_exponent(amax) + 127) << 23);
  const float scale = fmaxf(need, old);
  if (held && scale > old) {  // the page's older tokens move to the larger scale
    const float ratio = old / scale;
    for (int64_t o = (int64_t)g * 8; o < (int64_t)held * D; o += GT * 8) {
      uint2 w = *reinterpret_cast<const uint2*>(tile + o);
      uint32_t v[2] = {w.x, w.y};
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint32_t u = v[k];
        v[k] = e4m3x2(e4m3_value(u & 255) * ratio, e4m3_value((u >> 8) & 255) * ratio) |
               (e4m3x2(e4m3_value((u >> 16) & 255) * ratio, e4m3_value(u >> 24) * ratio) << 16);
      }
      *reinterpret_cast<uint2*>(tile + o) = make_uint2(v[0], v[1]);
    }
  }
  if (GT == 32) __syncwarp();     // every thread has read the old scale (a block: before its barrier)
  if (g == 0) *scale_at = scale;
  const bool exact = (__float_as_int(scale) & 0x7FFFFF) == 0 && scale >= 0x1p-100f && scale <= 0x1p120f;
  const float inv = exact ? 1.0f / scale : 0.0f;
#pragma unroll
  for (int i = 0; i < ITER; ++i) {
    const int t = lo + i * TPP + g / LPH;
    if (t >= hi) break;
    uint8_t* at = tile + (int64_t)(t - base) * D;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      F2 u = y[i][2 * k], v = y[i][2 * k + 1];
      if (exact)
        u = mul2(u, {inv, inv}), v = mul2(v, {inv, inv});
      else
        u = {u.x / scale, u.y / scale}, v = {v.x / scale, v.y / scale};
      *reinterpret_cast<uint32_t*>(at + (k ? nr.b : nr.a)) = e4m3x2(u.x, u.y) | (e4m3x2(v.x, v.y) << 16);
    }
  }
}

// Blocks 0 .. kv_blocks-1 take the units, the rest the queries.
template <int LPH, int GT, int ITER>
__global__ void __launch_bounds__(GT > kAppendThreads ? GT : kAppendThreads)
    append_kernel(const AppendArgs a, int64_t units, int64_t kv_blocks, int per_seq, int scan) {
  __shared__ float red[GT > 32 ? GT / 32 : 1];
  pdl_launch_dependents();
  pdl_wait();
  if ((int64_t)blockIdx.x < kv_blocks) {
    const int64_t unit = GT == 32 ? (int64_t)blockIdx.x * (kAppendThreads / 32) + (threadIdx.x >> 5) : blockIdx.x;
    if (unit < units) append_unit<LPH, GT, ITER>(a, unit, per_seq, scan != 0, red);
  } else if (threadIdx.x < kAppendThreads) {
    append_queries<LPH>(a, (uint32_t)(blockIdx.x - kv_blocks));
  }
}

template <int LPH, int GT, int ITER>
int launch(const AppendArgs& a, cudaStream_t s) {
  const KvArgs& c = a.c;
  const int64_t P = (int64_t)1 << c.page_log2;
  // a sequence of r new tokens touches at most (r + P - 2) / P + 1 <= r / P + 2 pages
  const int64_t per = ((int64_t)c.max_new + P - 2) / P + 1;
  const int64_t direct = (int64_t)c.n_seqs * per, bound = c.n_tokens / P + 2 * (int64_t)c.n_seqs;
  const bool scan = direct > 2 * bound;  // far fewer pages than slots: find each unit's sequence by a scan
  const int64_t units = (scan ? bound : direct) * 2 * c.hkv;
  const int64_t kv_blocks = GT == 32 ? (units + kAppendThreads / 32 - 1) / (kAppendThreads / 32) : units;
  const int64_t q_items = c.n_tokens * ((a.hq + kQHeads - 1) / kQHeads), groups = kAppendThreads / LPH;
  const int64_t q_blocks = (q_items + groups - 1) / groups;
  if (kv_blocks + q_blocks > 0x7FFFFFFF || q_items + groups > 0x7FFFFFFF) return QG_ERR_UNSUPPORTED;
  return launch_pdl(append_kernel<LPH, GT, ITER>, dim3((unsigned)(kv_blocks + q_blocks)), dim3(std::max(GT, kAppendThreads)), 0,
                    s, a, units, kv_blocks, (int)per, scan ? 1 : 0) == cudaSuccess
             ? QG_OK
             : QG_ERR_CUDA;
}

// Threads and passes so that a page's values fit the group's registers.
template <int LPH>
int launch_heads(const AppendArgs& a, cudaStream_t s) {
  if (a.c.max_new <= kWarpRows) return launch<LPH, 32, kWarpRows * LPH / 32>(a, s);
  const int passes = ((LPH << a.c.page_log2) + kAppendThreads - 1) / kAppendThreads;
  if (passes <= 1) return launch<LPH, 256, 1>(a, s);
  if (passes <= 2) return launch<LPH, 256, 2>(a, s);
  if (passes <= 4) return launch<LPH, 256, 4>(a, s);
  if (passes <= 8) return launch<LPH, 256, 8>(a, s);
  return launch<LPH, 512, 8>(a, s);
}

}  // namespace

int launch_append(const AppendArgs& a, int head_dim, void* stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  switch (head_dim) {
    case 64: return launch_heads<8>(a, s);
    case 128: return launch_heads<16>(a, s);
    case 256: return launch_heads<32>(a, s);
  }
  return QG_ERR_UNSUPPORTED;
}

}  // namespace qg
