// C ABI entry points of the attention operators (qkv_append, qattn): argument validation on
// the host, then the kernel launchers.  No entry point allocates memory.
#include <cuda_runtime.h>

#include <cmath>

#include "qg_attn.h"
#include "qg_internal.h"

namespace qg {
namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Sizes of a cache, a batch and a call; no pointer is looked at.
int check_sizes(const qg_kv_cache* c, const qg_kv_batch* b, int64_t n_tokens) {
  if (!c || !b || n_tokens < 0) return QG_ERR_INVALID_ARG;
  if (c->fmt != QG_KV_E4M3 || c->n_kv_heads < 1 || c->n_pages < 1) return QG_ERR_INVALID_ARG;
  if (c->page_tokens != 16 && c->page_tokens != 32 && c->page_tokens != 64 && c->page_tokens != 128)
    return QG_ERR_UNSUPPORTED;
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return QG_ERR_UNSUPPORTED;
  if (c->n_kv_heads > 1024 || c->n_pages > 0x7FFFFFFF) return QG_ERR_UNSUPPORTED;
  if (b->n_seqs < 1 || b->max_new < 1 || b->max_len < 1 || b->page_stride < 1) return QG_ERR_INVALID_ARG;
  if (b->n_seqs > 65535 || b->max_len > 0x7FFFFF00 || n_tokens > 0x7FFFFF00) return QG_ERR_UNSUPPORTED;
  if ((b->max_len + c->page_tokens - 1) / c->page_tokens > b->page_stride) return QG_ERR_INVALID_ARG;
  return QG_OK;
}

int check_pointers(const qg_kv_cache* c, const qg_kv_batch* b) {
  if (!c->k_codes || !c->v_codes || !c->k_scales || !c->v_scales || !b->q_start || !b->lens || !b->pages)
    return QG_ERR_INVALID_ARG;
  if (!aligned16(c->k_codes) || !aligned16(c->v_codes) || !aligned16(c->k_scales) || !aligned16(c->v_scales))
    return QG_ERR_MISALIGNED;
  if (reinterpret_cast<uintptr_t>(b->q_start) % 4 || reinterpret_cast<uintptr_t>(b->lens) % 4 ||
      reinterpret_cast<uintptr_t>(b->pages) % 4)
    return QG_ERR_MISALIGNED;
  return QG_OK;
}

// A tensor [token][head][head_dim] of bf16.  A stride of 0 or below head_dim would make rows
// or heads overlap: refused where there is more than one of them.
int check_heads(const void* p, int64_t ld, int64_t hs, int64_t tokens, int heads, int d) {
  if (!p) return QG_ERR_INVALID_ARG;
  if ((tokens > 1 && ld < d) || (heads > 1 && hs < d)) return QG_ERR_INVALID_ARG;
  if (!aligned16(p) || ld % 8 || hs % 8) return QG_ERR_MISALIGNED;
  return QG_OK;
}

int log2i(int v) {
  int r = 0;
  while ((1 << r) < v) ++r;
  return r;
}

void fill(const qg_kv_cache* c, const qg_kv_batch* b, int64_t n_tokens, void* ws, KvArgs* a) {
  a->k = static_cast<uint8_t*>(c->k_codes);
  a->v = static_cast<uint8_t*>(c->v_codes);
  a->ks = c->k_scales;
  a->vs = c->v_scales;
  a->n_pages = c->n_pages;
  a->hkv = c->n_kv_heads;
  a->page_log2 = log2i(c->page_tokens);
  a->q_start = b->q_start;
  a->lens = b->lens;
  a->pages = b->pages;
  a->page_stride = b->page_stride;
  a->n_seqs = b->n_seqs;
  a->max_new = b->max_new;
  a->max_len = b->max_len;
  a->n_tokens = n_tokens;
  a->status = static_cast<int*>(ws);
}

}  // namespace
}  // namespace qg

using namespace qg;

extern "C" size_t qkv_append_workspace_size(void) { return kWsHeader; }

extern "C" qg_status qkv_append(const qg_kv_cache* cache, const qg_kv_batch* batch, const qg_norm_rope* norm_rope,
                                int64_t n_tokens, int n_q_heads, const void* q, int64_t ldq, int64_t hsq,
                                const void* k, int64_t ldk, int64_t hsk, const void* v, int64_t ldv, int64_t hsv,
                                void* q_out, int64_t ldqo, int64_t hsqo, void* workspace, size_t workspace_bytes,
                                void* stream) {
  int st = check_sizes(cache, batch, n_tokens);
  if (st != QG_OK) return (qg_status)st;
  if (n_q_heads < 0) return QG_ERR_INVALID_ARG;
  if (n_tokens > 0 && ((q == nullptr) != (n_q_heads == 0) || (q == nullptr) != (q_out == nullptr)))
    return QG_ERR_INVALID_ARG;
  if (n_q_heads > 16384) return QG_ERR_UNSUPPORTED;
  AppendArgs a = {};
  a.hq = n_q_heads;
  if (norm_rope) {
    const qg_norm_rope& r = *norm_rope;
    if (!(r.eps >= 0.0f) || !std::isfinite(r.eps) || !std::isfinite(r.weight_offset)) return QG_ERR_INVALID_ARG;
    if (r.rotary_dim < 0 || r.rotary_dim > cache->head_dim || (r.rotary_dim == 0) != (r.cos_sin == nullptr) ||
        (r.interleaved != 0 && r.interleaved != 1))
      return QG_ERR_INVALID_ARG;
    if (r.rotary_dim % 16) return QG_ERR_UNSUPPORTED;
    if (r.rotary_dim && r.n_positions < batch->max_len) return QG_ERR_INVALID_ARG;
    if ((r.q_weight && !aligned16(r.q_weight)) || (r.k_weight && !aligned16(r.k_weight)) ||
        (r.cos_sin && !aligned16(r.cos_sin)))
      return QG_ERR_MISALIGNED;
    a.qw = static_cast<const uint16_t*>(r.q_weight);
    a.kw = static_cast<const uint16_t*>(r.k_weight);
    a.cs = r.cos_sin;
    a.eps = r.eps;
    a.woff = r.weight_offset;
    a.rot = r.rotary_dim;
    a.interleaved = r.interleaved;
  }
  if (n_tokens == 0) return QG_OK;
  st = check_pointers(cache, batch);
  if (st != QG_OK) return (qg_status)st;
  const int d = cache->head_dim;
  if (q) {
    st = check_heads(q, ldq, hsq, n_tokens, n_q_heads, d);
    if (st == QG_OK) st = check_heads(q_out, ldqo, hsqo, n_tokens, n_q_heads, d);
    if (st != QG_OK) return (qg_status)st;
    if (q == q_out && (ldq != ldqo || hsq != hsqo)) return QG_ERR_INVALID_ARG;
  }
  st = check_heads(k, ldk, hsk, n_tokens, cache->n_kv_heads, d);
  if (st == QG_OK) st = check_heads(v, ldv, hsv, n_tokens, cache->n_kv_heads, d);
  if (st != QG_OK) return (qg_status)st;
  if (!workspace) return QG_ERR_INVALID_ARG;
  if (!aligned16(workspace)) return QG_ERR_MISALIGNED;
  if (workspace_bytes < kWsHeader) return QG_ERR_WORKSPACE_TOO_SMALL;
  fill(cache, batch, n_tokens, workspace, &a.c);
  a.q = static_cast<const uint16_t*>(q);
  a.kin = static_cast<const uint16_t*>(k);
  a.vin = static_cast<const uint16_t*>(v);
  a.qo = static_cast<uint16_t*>(q_out);
  a.ldq = ldq;
  a.hsq = hsq;
  a.ldk = ldk;
  a.hsk = hsk;
  a.ldv = ldv;
  a.hsv = hsv;
  a.ldo = ldqo;
  a.hso = hsqo;
  return (qg_status)launch_append(a, d, stream);
}

static int check_attn_sizes(const qg_kv_cache* cache, const qg_kv_batch* batch, int64_t n_tokens, int n_q_heads) {
  int st = check_sizes(cache, batch, n_tokens);
  if (st != QG_OK) return st;
  if (n_q_heads < 1 || n_q_heads % cache->n_kv_heads) return QG_ERR_INVALID_ARG;
  if (n_q_heads / cache->n_kv_heads > 128 || n_q_heads > 16384) return QG_ERR_UNSUPPORTED;
  return QG_OK;
}

extern "C" size_t qattn_workspace_size(const qg_kv_cache* cache, const qg_kv_batch* batch, int64_t n_tokens,
                                       int n_q_heads) {
  if (check_attn_sizes(cache, batch, n_tokens, n_q_heads) != QG_OK) return 0;
  DeviceInfo dev;
  AttnPlan p;
  if (!current_device_info(&dev) || !plan_attn(cache, batch, n_tokens, n_q_heads, dev, &p)) return 0;
  return p.ws_bytes;
}

extern "C" qg_status qattn(const qg_kv_cache* cache, const qg_kv_batch* batch, int64_t n_tokens, int n_q_heads,
                           const void* q, int64_t ldq, int64_t hsq, float scale, int64_t window, void* out,
                           int64_t ldo, int64_t hso, void* workspace, size_t workspace_bytes, void* stream) {
  int st = check_attn_sizes(cache, batch, n_tokens, n_q_heads);
  if (st != QG_OK) return (qg_status)st;
  if (!(scale > 0.0f) || !std::isfinite(scale) || window < 0) return QG_ERR_INVALID_ARG;
  if (n_tokens == 0) return QG_OK;
  st = check_pointers(cache, batch);
  if (st == QG_OK) st = check_heads(q, ldq, hsq, n_tokens, n_q_heads, cache->head_dim);
  if (st == QG_OK) st = check_heads(out, ldo, hso, n_tokens, n_q_heads, cache->head_dim);
  if (st != QG_OK) return (qg_status)st;
  if (q == out && (ldq != ldo || hsq != hso)) return QG_ERR_INVALID_ARG;
  if (!workspace) return QG_ERR_INVALID_ARG;
  if (!aligned16(workspace)) return QG_ERR_MISALIGNED;
  DeviceInfo dev;
  if (!current_device_info(&dev)) return QG_ERR_CUDA;
  AttnPlan p;
  if (!plan_attn(cache, batch, n_tokens, n_q_heads, dev, &p)) return QG_ERR_UNSUPPORTED;
  if (workspace_bytes < p.ws_bytes) return QG_ERR_WORKSPACE_TOO_SMALL;
  AttnArgs a = {};
  fill(cache, batch, n_tokens, workspace, &a.c);
  a.q = static_cast<const uint16_t*>(q);
  a.out = static_cast<uint16_t*>(out);
  a.ldq = ldq;
  a.hsq = hsq;
  a.ldo = ldo;
  a.hso = hso;
  a.scale = scale;
  a.window = window && window < 0x7FFFFFFF ? (int)window : 0x7FFFFFFF;
  a.hq = n_q_heads;
  return (qg_status)launch_attn(a, cache->head_dim, p, dev, workspace, stream);
}
