// How bitnest_prefix_attention cuts its work into parts (shared by its kernels).
#pragma once

#include "launch.h"

namespace bitnest {
namespace pattn {

constexpr int kSms = 148;
constexpr int kTcRows = 256, kTcTokens = 128;  // of a unit on the tcgen05 path
constexpr int64_t kTcMinRows = 64;

struct Plan {
  int G;                // query heads of a KV head
  // the prefix on the tensor cores' tcgen05 path: units of (256 rows of a KV
  // head, 128 tokens), dealt to the CTAs in equal runs
  bool tc;
  int tc_groups;        // row groups of a KV head
  int tc_tiles;         // token tiles of the prefix
  int64_t tc_units;
  int tc_ctas;
  // the prefix on mma.sync (few rows): CTAs of (KV head, row group, tokens)
  int row_warps;        // row tiles of a CTA (its other warps split tokens)
  int p_groups, p_len;
  int64_t p_ctas;
  int p_splits;         // parts of a row's prefix, at most
  // own tokens: CTAs of (sequence, KV head, row tile, tokens)
  int o_tiles, o_splits, o_len;
  int64_t o_ctas;
};

// The CTA that unit u belongs to: CTA c has units floor(c U / n) .. floor((c + 1) U / n) - 1.
__host__ __device__ inline int64_t tc_cta_of(const Plan &p, int64_t u) {
  return ((u + 1) * p.tc_ctas - 1) / p.tc_units;
}
// Parts of the rows of `item` = KV head * tc_groups + row group.
__host__ __device__ inline int tc_parts(const Plan &p, int64_t item) {
  return (int)(tc_cta_of(p, (item + 1) * p.tc_tiles - 1) - tc_cta_of(p, item * p.tc_tiles)) + 1;
}

cudaError_t launch_prefix_tc(const PrefixAttnArgs &a, const Plan &p, float *part_lse,
                             float *part_o, cudaStream_t st);

}  // namespace pattn
}  // namespace bitnest
