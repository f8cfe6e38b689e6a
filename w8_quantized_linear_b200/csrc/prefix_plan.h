// How bitnest_prefix_attention cuts its work into parts (shared by its kernels).
#pragma once

#include "launch.h"

namespace bitnest {
namespace pattn {

constexpr int kSms = 148;
constexpr int kTcTile = 128, kTcTokens = 128;  // rows of an MMA tile, tokens of a unit on the tcgen05 path
// The tcgen05 path from 64 rows of a KV head on, but for little work: with one
// KV head, 512 tokens and 64 rows the mma.sync path takes 9.7 us against 9.9, with
// 256 rows 11.2 against 11.0; at 64 rows and 2048 tokens 11.2 against 10.2, with 8
// KV heads 14.5 against 12.1, and at 8192 tokens 30 against 20 (join included).
constexpr int64_t kTcMinRows = 64, kTcMinTiles = 512;  // ... tiles of 16 rows x 16 tokens

struct Plan {
  int G, lgG;           // query heads of a KV head, and their logarithm
  // the prefix on the tensor cores' tcgen05 path: units of (tc_rows rows of a KV
  // head, 128 tokens), dealt to the CTAs in runs; tc_rows is 256, or 128 where
  // that still gives each CTA one unit (11.0 us instead of 14.6 at 256 rows, 512
  // tokens and one KV head)
  bool tc;
  int tc_rows;
  int tc_groups;        // row groups of a KV head
  int tc_tiles;         // token tiles of the prefix
  int tc_units, tc_run, tc_ctas;
  // the prefix on mma.sync (few rows): CTAs of (KV head, row group, tokens)
  int row_warps;        // row tiles of a CTA (its other warps split tokens)
  int p_groups, p_len, p_ctas;
  int p_splits;         // parts of a row's prefix, at most
  // own tokens: CTAs of (sequence, KV head, row tile, tokens)
  int o_tiles, o_splits, o_len, o_ctas;
};

// Parts of the rows of `item` = KV head * tc_groups + row group: one for each
// CTA that has units of it (CTA c has units c * tc_run .. (c + 1) * tc_run - 1).
__host__ __device__ inline int tc_first_cta(const Plan &p, int item) {
  return item * p.tc_tiles / p.tc_run;
}
__host__ __device__ inline int tc_parts(const Plan &p, int item) {
  return ((item + 1) * p.tc_tiles - 1) / p.tc_run - tc_first_cta(p, item) + 1;
}

cudaError_t launch_prefix_tc(const PrefixAttnArgs &a, const Plan &p, float *part_lse,
                             float *part_o, cudaStream_t st);

}  // namespace pattn
}  // namespace bitnest
