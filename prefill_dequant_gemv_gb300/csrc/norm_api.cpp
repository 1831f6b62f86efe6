// C ABI entry point of the RMS norm (qg_rms_norm): argument validation on the host, then the
// kernel launcher.
#include <cuda_runtime.h>

#include <cmath>

#include "qg_norm.h"

namespace qg {
namespace {

bool misaligned(const void* p, int64_t ld) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0 || ld % 8; }

// An output may lie on an input only element by element.
bool crosses(const void* out, int64_t ldo, const void* in, int64_t ldi) { return out && out == in && ldo != ldi; }

}  // namespace
}  // namespace qg

using namespace qg;

extern "C" qg_status qg_rms_norm(const void* x, int64_t ldx, const void* residual, int64_t ldr, int64_t m, int64_t k,
                                 const void* weight, float eps, float weight_offset, const qg_norm_out* out,
                                 void* stream) {
  if (!out || m < 0 || k < 1 || !(eps >= 0.0f) || !std::isfinite(eps) || !std::isfinite(weight_offset))
    return QG_ERR_INVALID_ARG;
  const qg_norm_out& o = *out;
  if ((!o.y && !o.codes) || (o.codes == nullptr) != (o.scales == nullptr) || (o.sum && !residual))
    return m ? QG_ERR_INVALID_ARG : QG_OK;
  if (o.codes && o.group != 0 && o.group != 32 && o.group != 64 && o.group != 128)
    return o.group < 0 ? QG_ERR_INVALID_ARG : QG_ERR_UNSUPPORTED;
  if (k > kNormMaxCols || m > 0x7FFFFFFF) return QG_ERR_UNSUPPORTED;
  if (m == 0) return QG_OK;
  if (!x || !weight) return QG_ERR_INVALID_ARG;
  const int64_t groups = o.group ? (k + o.group - 1) / o.group : 1;
  if (ldx < k || (residual && ldr < k) || (o.sum && o.ldh < k) || (o.y && o.ldy < k) ||
      (o.codes && (o.ldc < k || o.lds < groups)))
    return QG_ERR_INVALID_ARG;
  if (misaligned(x, ldx) || misaligned(weight, 0) || (residual && misaligned(residual, ldr)) ||
      (o.sum && misaligned(o.sum, o.ldh)) || (o.y && misaligned(o.y, o.ldy)) || (o.codes && misaligned(o.codes, o.ldc)) ||
      reinterpret_cast<uintptr_t>(o.scales) % 4)
    return QG_ERR_MISALIGNED;
  if (crosses(o.sum, o.ldh, x, ldx) || crosses(o.sum, o.ldh, residual, ldr) || crosses(o.y, o.ldy, x, ldx) ||
      crosses(o.y, o.ldy, residual, ldr) || (o.sum && o.sum == o.y) || (o.codes && (o.codes == x || o.codes == residual)))
    return QG_ERR_INVALID_ARG;
  DeviceInfo dev;
  if (!current_device_info(&dev)) return QG_ERR_CUDA;
  NormArgs a = {};
  a.x = static_cast<const uint16_t*>(x);
  a.res = static_cast<const uint16_t*>(residual);
  a.w = static_cast<const uint16_t*>(weight);
  a.ldx = ldx;
  a.ldr = ldr;
  a.m = m;
  a.k = k;
  a.eps = eps;
  a.woff = weight_offset;
  a.sum = static_cast<uint16_t*>(o.sum);
  a.ldh = o.ldh;
  a.y = static_cast<uint16_t*>(o.y);
  a.ldy = o.ldy;
  a.codes = o.codes;
  a.scales = o.scales;
  a.ldc = o.ldc;
  a.lds = o.lds;
  a.group_lanes = o.codes ? (int)(o.group / 8) : 0;
  a.group_log2 = a.group_lanes == 4 ? 5 : a.group_lanes == 8 ? 6 : 7;
  return (qg_status)launch_rms_norm(a, dev, stream);
}
