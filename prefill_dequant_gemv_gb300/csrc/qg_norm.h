// Arguments of the RMS norm's launcher (validated by the caller).
#pragma once

#include <stdint.h>

#include "qg_internal.h"

namespace qg {

constexpr int64_t kNormMaxCols = 65536;  // a row of bf16 in shared memory

struct NormArgs {
  const uint16_t* x;
  const uint16_t* res;  // or null
  const uint16_t* w;
  int64_t ldx, ldr, m, k;
  float eps, woff;
  uint16_t* sum;  // or null
  uint16_t* y;    // or null (with codes)
  int64_t ldh, ldy;
  uint8_t* codes;  // or null
  float* scales;
  int64_t ldc, lds;
  int group_lanes;  // eighths of a group: 4, 8 or 16; 0: one scale a row
  int group_log2;
};
int launch_rms_norm(const NormArgs& a, const DeviceInfo& dev, void* stream);

}  // namespace qg
