// Attention over the 8-bit paged cache, in its simplest form: one block per (row, query head),
// its warps striding over the visible keys with an online softmax each, merged at the end.
//
// Where the scales go: with s_j = scale * q.k_j * log2(e), vs_j the value scale of key j's page
// and c_j its value codes, the warps keep t_j = s_j + log2(vs_j), m = max t_j, P_j = 2^(t_j - m):
//   out = sum P_j c_j / sum (P_j / vs_j).
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "qg_attn.h"
#include "qg_sync.cuh"

namespace qg {
namespace {

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float code_value(uint8_t x) {
  __nv_fp8_e4m3 v;
  v.__x = x;
  return static_cast<float>(v);
}

template <int D>
__global__ void __launch_bounds__(128) attn_simple_kernel(const AttnArgs a) {
  constexpr int E = D / 32;
  __shared__ float sm[4], sl[4], so[4][D];
  const KvArgs& c = a.c;
  const int64_t row = blockIdx.x;
  const int head = blockIdx.y, kvh = head / (a.hq / c.hkv), warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int lo = 0, hi = c.n_seqs;
  while (hi - lo > 1) {
    const int m = (lo + hi) >> 1;
    if (c.q_start[m] <= row) lo = m; else hi = m;
  }
  bool bad = false;
  const Seq s = seq_of(c, lo, &bad);
  if (bad && threadIdx.x == 0) atomicExch(c.status, kStatusInvalid);
  if (row < s.start || row >= (int64_t)s.start + s.rows) return;
  const int pos = s.len - s.rows + (int)(row - s.start);
  const int from = pos >= a.window ? pos + 1 - a.window : 0;  // a row before the sequence (pos < 0) sees nothing
  float q[E], o[E], m = -INFINITY, l = 0.0f;
  for (int e = 0; e < E; ++e) {
    q[e] = __uint_as_float((uint32_t)a.q[row * a.ldq + head * a.hsq + lane * E + e] << 16);
    o[e] = 0.0f;
  }
  for (int t = from + warp; pos >= 0 && t <= pos; t += 4) {
    const int id = c.pages[(int64_t)lo * c.page_stride + (t >> c.page_log2)];
    if (id < 0 || id >= c.n_pages) {
      if (lane == 0) atomicExch(c.status, kStatusInvalid);
      continue;
    }
    const int64_t at = ((int64_t)id * c.hkv + kvh), base = ((at << c.page_log2) + (t & ((1 << c.page_log2) - 1))) * D;
    float d = 0.0f;
    for (int e = 0; e < E; ++e) d += q[e] * code_value(c.k[base + lane * E + e]);
    for (int x = 16; x; x >>= 1) d += __shfl_xor_sync(0xFFFFFFFFu, d, x);
    const float vs = c.vs[at];
    const float tj = d * (c.ks[at] * a.scale * kLog2e) + log2f(vs);
    const float mn = fmaxf(m, tj), w = exp2f(m - mn), p = exp2f(tj - mn);
    l = l * w + p / vs;
    for (int e = 0; e < E; ++e) o[e] = o[e] * w + p * code_value(c.v[base + lane * E + e]);
    m = mn;
  }
  if (lane == 0) sm[warp] = m, sl[warp] = l;
  for (int e = 0; e < E; ++e) so[warp][lane * E + e] = o[e];
  __syncthreads();
  const float top = fmaxf(fmaxf(sm[0], sm[1]), fmaxf(sm[2], sm[3]));
  for (int d = threadIdx.x; d < D; d += 128) {
    float num = 0.0f, den = 0.0f;
    for (int w = 0; w < 4; ++w) {
      const float f = sm[w] == -INFINITY ? 0.0f : exp2f(sm[w] - top);
      num += f * so[w][d];
      den += f * sl[w];
    }
    const __nv_bfloat16 r = __float2bfloat16_rn(den == 0.0f ? 0.0f : num / den);
    a.out[row * a.ldo + head * a.hso + d] = *reinterpret_cast<const uint16_t*>(&r);
  }
}

}  // namespace

bool plan_attn(const qg_kv_cache* cache, const qg_kv_batch* batch, int64_t, int hq, const DeviceInfo& dev, AttnPlan* p) {
  const int64_t rows = (int64_t)batch->max_new * (hq / cache->n_kv_heads);
  p->decode = decode_rows(rows) != 0;
  p->ws_bytes = p->decode ? decode_workspace(rows, cache->head_dim, dev) : kWsHeader;
  return true;
}

int launch_attn(const AttnArgs& a, int head_dim, const AttnPlan& p, const DeviceInfo& dev, void* ws, void* stream) {
  if (p.decode) return launch_attn_decode(a, head_dim, (int64_t)a.c.max_new * (a.hq / a.c.hkv), dev, ws, stream);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const dim3 grid((unsigned)a.c.n_tokens, (unsigned)a.hq);
  switch (head_dim) {
    case 64: attn_simple_kernel<64><<<grid, 128, 0, s>>>(a); break;
    case 128: attn_simple_kernel<128><<<grid, 128, 0, s>>>(a); break;
    case 256: attn_simple_kernel<256><<<grid, 128, 0, s>>>(a); break;
    default: return QG_ERR_UNSUPPORTED;
  }
  return cudaGetLastError() == cudaSuccess ? QG_OK : QG_ERR_CUDA;
}

}  // namespace qg
