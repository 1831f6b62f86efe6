// Shared by the cache append and the attention kernels: kernel arguments, the device-side
// reading of a batch's sequences, and E4M3 helpers.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "qg_internal.h"

namespace qg {

// What the kernels need of a cache and a batch.
struct KvArgs {
  uint8_t* k;
  uint8_t* v;
  float* ks;
  float* vs;
  int64_t n_pages;
  int hkv, page_log2;
  const int32_t* q_start;
  const int32_t* lens;
  const int32_t* pages;
  int64_t page_stride;
  int n_seqs, max_new;
  int64_t max_len, n_tokens;
  int* status;
};

struct AppendArgs {
  KvArgs c;
  const uint16_t* q;
  const uint16_t* kin;
  const uint16_t* vin;
  uint16_t* qo;
  int64_t ldq, hsq, ldk, hsk, ldv, hsv, ldo, hso;
  const uint16_t* qw;
  const uint16_t* kw;
  const float* cs;
  float eps, woff;
  int hq, rot, interleaved;
};

struct AttnArgs {
  KvArgs c;
  const uint16_t* q;
  uint16_t* out;
  int64_t ldq, hsq, ldo, hso;
  float scale;
  int window;  // keys a row sees at most; none: 2^31 - 1
  int hq;
};

// How qattn divides the work; a function of the sizes alone.
struct PrefillPlan {
  int64_t blocks;  // upper bound of the row blocks of a KV head
  int splits;      // parts of a block along the keys
  size_t off_ml, off_o, ws_bytes;
};
struct AttnPlan {
  size_t ws_bytes;
  bool decode;  // the streaming kernel
  PrefillPlan prefill;
};
// Counters of the joins, right behind the workspace's header whatever the call.
constexpr size_t kAttnCounterBytes = 4096;
bool plan_attn(const qg_kv_cache* cache, const qg_kv_batch* batch, int64_t n_tokens, int hq, const DeviceInfo& dev,
               AttnPlan* p);
int launch_attn(const AttnArgs& a, int head_dim, const AttnPlan& p, const DeviceInfo& dev, void* ws, void* stream);
// The streaming kernel of up to 32 rows (new tokens x query heads a KV head).
int decode_rows(int64_t rows);  // the row count it is built for: 16, 32; 0: too many
size_t decode_workspace(int64_t rows, int head_dim, const DeviceInfo& dev);
int launch_attn_decode(const AttnArgs& a, int head_dim, int64_t rows, const DeviceInfo& dev, void* ws, void* stream);
// The row-block kernel of more rows.
bool plan_prefill(const qg_kv_cache* cache, const qg_kv_batch* batch, int64_t n_tokens, int hq, const DeviceInfo& dev,
                  PrefillPlan* p);
int launch_attn_prefill(const AttnArgs& a, int head_dim, const PrefillPlan& p, void* ws, void* stream);
// Pages of codes as a 3-D TMA tensor (head_dim bytes x page_tokens x tiles, tile = page * n_kv_heads +
// head): box of min(head_dim, 128) bytes x box_tokens tokens, swizzled by its width.
bool encode_pages(CUtensorMap* map, const void* codes, int head_dim, int page_tokens, int64_t tiles, int box_tokens);
int launch_append(const AppendArgs& a, int head_dim, void* stream);

#ifdef __CUDACC__
// Sequence b's first row, number of rows and length.  A sequence outside the call's bounds
// has no rows.
struct Seq {
  int start, rows, len;
};
__device__ __forceinline__ Seq seq_of(const KvArgs& c, int b, bool* bad) {
  Seq s;
  const int s0 = c.q_start[b], s1 = c.q_start[b + 1];
  s.len = c.lens[b];
  s.start = s0;
  s.rows = s1 - s0;
  if (s0 < 0 || s1 < s0 || s1 > c.n_tokens || s1 - s0 > c.max_new || s.len < 0 || s.len > c.max_len) {
    s.start = 0;
    s.rows = 0;
    s.len = 0;
    *bad = true;
  }
  return s;
}
#endif

}  // namespace qg
