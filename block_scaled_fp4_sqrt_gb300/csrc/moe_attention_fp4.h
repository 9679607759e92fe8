// The paged attention's form for MXFP4 caches (moe_attention_fp4.cu), as moe_paged_attention sees it.
#pragma once

#include "moe_attention_common.cuh"

namespace moe {

int attention_fp4_tile_rows(int head_dim, int64_t rows);  // rows of a row tile for this many rows a kv head
int attention_fp4_blocks(int head_dim, int tile_rows);    // blocks an SM runs
int attention_fp4_lanes(int n_kv_heads);                // kv heads that as many blocks read side by side
size_t attention_fp4_groups(int n_kv_heads, int blocks);   // groups of blocks whose parts are joined in two steps
cudaError_t launch_attention_fp4(const AttnParams& p, int num_sms, cudaStream_t s);

}  // namespace moe
