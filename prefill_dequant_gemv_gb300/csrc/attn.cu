// qattn's dispatch: few rows a KV head stream the cache, more take row blocks through it.
#include "qg_attn.h"

namespace qg {

bool plan_attn(const qg_kv_cache* cache, const qg_kv_batch* batch, int64_t n_tokens, int hq, const DeviceInfo& dev,
               AttnPlan* p) {
  const int64_t rows = (int64_t)batch->max_new * (hq / cache->n_kv_heads);
  p->decode = decode_rows(rows) != 0;
  if (p->decode) {
    p->ws_bytes = decode_workspace(rows, cache->head_dim, dev);
    return true;
  }
  if (!plan_prefill(cache, batch, n_tokens, hq, dev, &p->prefill)) return false;
  p->ws_bytes = p->prefill.ws_bytes;
  return true;
}

int launch_attn(const AttnArgs& a, int head_dim, const AttnPlan& p, const DeviceInfo& dev, void* ws, void* stream) {
  if (p.decode) return launch_attn_decode(a, head_dim, (int64_t)a.c.max_new * (a.hq / a.c.hkv), dev, ws, stream);
  return launch_attn_prefill(a, head_dim, p.prefill, ws, stream);
}

}  // namespace qg
