// Router workspace layout (host and device).
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace qg {

constexpr int kMaxExperts = 512;
constexpr int kMaxTopk = 16;
constexpr int kRouteTile = 192;  // pairs per grouped-prefill tile (the tensor-core N)

// Group table entry (8 ints) of active expert z (ascending experts): expert, first grouped
// position, pair count, 0, then the tokens of its first kGroupRows pairs.
constexpr int kGroupRows = 4;
constexpr int kGroupInts = 8;
// Pairs one CTA routes in the decode chain's gate/up launch (T <= 4 tokens, k <= 16).
constexpr int kBlockRoutePairs = 64;

// Tokens that one block of the large router's top-k takes: whole rounds of its eight warps, some 512 blocks at most; and
// that one of its placing blocks takes: whole blocks of those, no more pairs than it has threads.
constexpr int kRouteBlock = 1024;
__host__ __device__ inline int route_block_tokens(int64_t T, int k) {
  const int64_t even = ((T + 511) / 512 + 7) / 8 * 8, most = kRouteBlock / k / 8 * 8;
  return (int)(even < most ? even : most);
}
__host__ __device__ inline int route_place_tokens(int64_t T, int k) {
  const int tb = route_block_tokens(T, k);
  return kRouteBlock / k / tb * tb;
}

struct RouteLayout {
  size_t meta, counts, offsets, active, pair_list, pair_pos, tiles, groups, zidx, block_counts, total;
  int64_t max_tiles, nblocks;
};

__host__ __device__ inline RouteLayout route_layout(int64_t T, int E, int k) {
  RouteLayout L;
  const int64_t P = T * k;
  const int tb = route_block_tokens(T, k);
  L.nblocks = (T + tb - 1) / tb;
  L.max_tiles = (P + kRouteTile - 1) / kRouteTile + E;
  size_t o = 0;
  auto take = [&o](size_t bytes) {
    const size_t at = o;
    o += (bytes + 255) & ~(size_t)255;
    return at;
  };
  L.meta = take(64);                      // [0] active experts, [1] tiles
  L.counts = take((size_t)E * 4);
  L.offsets = take((size_t)(E + 1) * 4);
  L.active = take((size_t)E * 4);
  L.pair_list = take((size_t)P * 4);      // grouped position -> pair t*k + j
  L.pair_pos = take((size_t)P * 4);       // pair -> grouped position
  L.tiles = take((size_t)L.max_tiles * 12);  // (expert, first position, count)
  L.groups = take((size_t)E * kGroupInts * 4);  // group table, one entry per active expert
  L.zidx = take((size_t)E * 4);                 // expert -> its index in the active list
  // Blocks grow from 8 tokens every 4096, so more tokens can have fewer of them: room for the most that any fewer tokens have
  // (512 from 4096 tokens on; past the largest block they only become more), as one workspace serves them all.
  const int64_t rounds = (T + 7) / 8, most = rounds < 512 ? rounds : 512;
  L.block_counts = take((size_t)(L.nblocks > most ? L.nblocks : most) * E * 4);
  L.total = o;
  return L;
}

struct RouteView {
  int* meta;
  int* counts;
  int* offsets;
  int* active;
  int* pair_list;
  int* pair_pos;
  int* tiles;
  int* groups;
  int* zidx;
  int* block_counts;  // [block][expert]: pairs, then pairs in the blocks before
};

// A qg_route_rule as the kernels take it.
struct RouteRule {
  int sigmoid, renormalise;
  int n_groups, topk_groups, group_best;
  int group_lanes;     // lanes that look through one group: 32 / n_groups rounded down to a power of two
  uint32_t group_mul;  // ceil(2^20 / experts a group): e * group_mul >> 20 is the group of e < 512
  int values;          // the choice goes by scores and bias; 0: by the logits, in the same order
  float scale;
  const float* bias;
};

RouteView route_view(void* ws, int64_t T, int E, int k);
int launch_route(const float* logits, int64_t T, int E, int k, int32_t* ids, float* wts, void* ws, void* stream);
int launch_route_by(const RouteRule& rule, const float* logits, int64_t T, int E, int k, int32_t* ids, float* wts, void* ws,
                    void* stream);

}  // namespace qg
