// C ABI entry points of the low-rank adapters (qlora): argument validation on the host, then the
// kernel launcher.
#include <cuda_runtime.h>

#include "qg_lora.h"

using namespace qg;

namespace {

bool misaligned(const void* p, int64_t ld) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0 || ld % 8; }

}  // namespace

extern "C" size_t qlora_workspace_size(const qg_lora* l, int64_t m) {
  if (!l || m < 0 || m >= (1 << 27) || l->n_adapters < 1 || l->n_adapters > kLoraMaxAdapters || l->max_rank < 1 ||
      l->max_rank > kLoraMaxRank || l->max_rank % 8 || l->n < 1 || l->n >= (1 << 24) || l->k < 1 || l->k >= (1 << 24))
    return 0;
  if (lora_few(m, l->n_adapters)) return kWsHeader;
  DeviceInfo dev;
  if (!current_device_info(&dev)) return 0;
  return kWsHeader + (dev.sms < kLoraMinSms ? 0 : lora_rows_bytes(l->n_adapters, l->max_rank, m, dev));
}

extern "C" qg_status qlora(const qg_lora* l, const int32_t* ids, int64_t m, const void* x, int64_t ldx, const void* y,
                           int64_t ldy, void* out, int64_t ldo, void* workspace, size_t workspace_bytes, void* stream) {
  if (!l || m < 0 || l->n_adapters < 1 || l->max_rank < 1 || l->n < 1 || l->k < 1) return QG_ERR_INVALID_ARG;
  if (l->n_adapters > kLoraMaxAdapters || l->max_rank > kLoraMaxRank || l->max_rank % 8 || m >= (1 << 27) ||
      l->n >= (1 << 24) || l->k >= (1 << 24))
    return QG_ERR_UNSUPPORTED;
  if (m == 0) return QG_OK;
  if (!l->a || !l->b || !l->scales || !ids || !x || !y || !out || !workspace) return QG_ERR_INVALID_ARG;
  if (l->lda < l->k || ldx < l->k || ldy < l->n || ldo < l->n) return QG_ERR_INVALID_ARG;
  if (l->lda > 0x7FFFFFFF || ldx > 0x7FFFFFFF || ldy > 0x7FFFFFFF || ldo > 0x7FFFFFFF) return QG_ERR_UNSUPPORTED;
  if (misaligned(l->a, l->lda) || misaligned(l->b, 0) || misaligned(x, ldx) || misaligned(y, ldy) || misaligned(out, ldo) ||
      misaligned(workspace, 0) || reinterpret_cast<uintptr_t>(ids) % 4 || reinterpret_cast<uintptr_t>(l->scales) % 4 ||
      reinterpret_cast<uintptr_t>(l->ranks) % 4)
    return QG_ERR_MISALIGNED;
  if ((out == y && ldo != ldy) || out == x) return QG_ERR_INVALID_ARG;
  if (workspace_bytes < kWsHeader) return QG_ERR_WORKSPACE_TOO_SMALL;
  DeviceInfo dev;
  if (!current_device_info(&dev)) return QG_ERR_CUDA;
  LoraArgs p = {};
  p.a = static_cast<const uint16_t*>(l->a);
  p.b = static_cast<const uint16_t*>(l->b);
  p.scales = l->scales;
  p.ranks = l->ranks;
  p.lda = (int)l->lda;
  p.n_adapters = l->n_adapters;
  p.max_rank = l->max_rank;
  p.n = (int)l->n;
  p.k = (int)l->k;
  p.ids = ids;
  p.m = (int)m;
  p.x = static_cast<const uint16_t*>(x);
  p.y = static_cast<const uint16_t*>(y);
  p.out = static_cast<uint16_t*>(out);
  p.ldx = (int)ldx;
  p.ldy = (int)ldy;
  p.ldo = (int)ldo;
  p.status = static_cast<int*>(workspace);
  if (lora_few(m, l->n_adapters)) return (qg_status)launch_lora(p, dev, stream);
  if (dev.sms < kLoraMinSms) return QG_ERR_UNSUPPORTED;
  if (workspace_bytes < kWsHeader + lora_rows_bytes(l->n_adapters, l->max_rank, m, dev)) return QG_ERR_WORKSPACE_TOO_SMALL;
  return (qg_status)launch_lora_rows(p, dev, static_cast<char*>(workspace) + kWsHeader, stream);
}
