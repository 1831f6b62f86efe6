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
  int lda, n_adapters, max_rank, n, k;
  const int32_t* ids;
  int m;
  const uint16_t* x;
  const uint16_t* y;
  uint16_t* out;  // y itself: rows without an adapter are not touched
  int ldx, ldy, ldo;
  int* status;
};
constexpr int64_t kLoraFewRows = 256;       // in one launch of clusters (lora.cu)
constexpr int64_t kLoraRowsAtOnce = 16384;  // in one launch of many rows: what a CTA looks through itself
constexpr int kLoraMinSms = 96;             // of lora_rows.cu: fewer SMs' CTAs would have more tiles each than they list
// Whether a call goes to lora.cu, 256 rows a launch, or to lora_rows.cu.  There every adapter that is met has tiles of 128 rows,
// mostly empty where adapters are many, but how many are met is known on the device only.  All of them met, us, rank 16 / 64,
// lora.cu against lora_rows.cu: 512 rows of 48 adapters 26 / 34 against 43 / 55, of 16 26 / 34 against 26 / 33; 768 of 48 38 / 52
// against 44 / 55, 1000 of 48 50 / 68 against 45 / 56; 300 rows of 4 adapters 24 / 33 against 19 / 24.  So the rule goes by the pool, which
// bounds them, for the worst that it can meet: of a pool of 200 all met 54 / 81 against 124 / 150, 64 met 24 / 37 against 51 / 65, 16 met 26 / 34
// against 26 / 33; where a call of 512 rows meets one of them, it loses 26 / 34 against 21 / 26.
inline bool lora_few(int64_t m, int n_adapters) { return m <= kLoraFewRows || (m <= 2 * kLoraFewRows && n_adapters >= 16); }
int launch_lora(const LoraArgs& a, const DeviceInfo& dev, void* stream);
// Scratch of the many-row form for h's parts, and its launches.
size_t lora_rows_bytes(int n_adapters, int max_rank, int64_t m, const DeviceInfo& dev);
int launch_lora_rows(const LoraArgs& a, const DeviceInfo& dev, void* parts, void* stream);

}  // namespace qg
