// qattn's dispatch: few rows a KV head stream the cache, more take row blocks through it.
//
// Up to 16 rows the streaming kernel is the faster one from one sequence of 1000 keys (16.8 us, row blocks 19.8;
// 5 rows, 8 KV heads of 128) to 16 of 8000 (62 against 122).  With 17 to 32 it needs some 2^18 keys over all pairs to
// win: 16 sequences of 2000, 8 heads of 128, 44 us against 39, of 4000 59 against 69, of 8000 85 against 122; 4 heads of
// 256, 16 of 4000 51 against 51, of 8000 69 against 82; one of 16000 59 against 46.  A form for 33 to 64 rows was
// slower everywhere (16 of 8000: 245 against 121).
#include "qg_attn.h"

namespace qg {

bool plan_attn(const qg_kv_cache* cache, const qg_kv_batch* batch, int64_t n_tokens, int hq, const DeviceInfo& dev,
               AttnPlan* p) {
  const int64_t rows = (int64_t)batch->max_new * (hq / cache->n_kv_heads);
  const int64_t keys = (int64_t)batch->n_seqs * cache->n_kv_heads * batch->max_len;
  p->decode = rows <= 16 || (decode_rows(rows) != 0 && keys >= 1 << 18);
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
