// qattn's dispatch: few rows a KV head stream the cache, more take row blocks through it.
//
// Up to 16 rows the streaming kernel is the faster one from one sequence of 1000 keys (19 us, row blocks 21;
// 5 rows, 8 KV heads of 128) to 16 of 8000 (66 against 123); at 15 rows only one of 1000 is not (22 against 21).  With 17
// to 32 it needs some 2^18 keys over all pairs to win: 16 sequences of 2000, 8 heads of 128, 49 us against 41, of 4000 68
// against 69, of 8000 98 against 123; 4 heads of 256, 16 of 4000 52 against 53, of 8000 71 against 84; one of 16000 53
// against 47; of 64, 16 of 4000 42 against 36, of 8000 56 against 58 (64 of 2000: 67 against 62).  A form for 33 to 64
// rows was slower everywhere (16 of 8000: 245 against 121).  The rule takes max_len for the keys and does not know the
// window, which the workspace's size does not depend on: with 17 to 32 rows under a window the row blocks would be
// faster (16 of 8000, window 128: 17 us against 22; 64 of 8000, window 1024: 102 against 106, heads of 64 44 against 53).
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
