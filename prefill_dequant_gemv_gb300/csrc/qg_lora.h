// Arguments of the low-rank adapters' launcher (validated by the caller).
#pragma once

#include <stdint.h>

#include "qg_internal.h"

namespace qg {

constexpr int kLoraMaxAdapters = 1024;
constexpr int kLoraMaxRank = 128;

struct LoraArgs {
  const uint16_t* a;  // [n_adapters][max_rank][lda]
  const uint16_t* b;  // [n_adapters][n][max_rank]
  const float* scales;
  const int32_t* ranks;  // or null: max_rank
  int64_t lda;
  int n_adapters, max_rank, n, k;
  const int32_t* ids;
  int m;
  const uint16_t* x;
  const uint16_t* y;
  uint16_t* out;  // y itself: rows without an adapter are not touched
  int64_t ldx, ldy, ldo;
  int* status;
};
int launch_lora(const LoraArgs& a, const DeviceInfo& dev, void* stream);

}  // namespace qg
