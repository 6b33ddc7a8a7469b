// kv_plan.h -- what the 8-bit cache's calls and the attention over a cache and
// drafts check and derive from their arguments on the host.
#pragma once

#include <cstdint>

#include "lse_merge.h"

namespace lsem {

// 8-bit cache, write and read back: check the arguments (`write`: quantize).
int check_kv_args(const lse_merge_kv_args& a, bool write);

// Attention over a cache and drafts: validated geometry.
struct TreePlan {
    int G;             // query heads per KV head
    int rows;          // query rows of one (sequence, KV head): T * G
    int shards;        // R, and one more for the drafts: as many partials per row as any call of
                       // these sizes has (more than 16 rows over a 16-bit cache: R, or none for R = 1)
    int64_t ws_l_off;  // workspace: partial o [B, T, Hq, shards, D] fp32, then lse [B, T, Hq, shards]
    int64_t ws_bytes;  // 0 for one shard without drafts, which writes the result itself
};
int tree_workspace(int B, int T, int Hq, int D, int R, bool drafts, TreePlan* plan);
int make_tree_plan(const lse_merge_tree_args& a, TreePlan* plan);
int tree_default_splits(int B, int T, int Hq, int Hkv, int L, int D, int sms);

}  // namespace lsem
