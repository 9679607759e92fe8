// The paged attention's form for MXFP4 caches (moe_attention_fp4.cu), as moe_paged_attention sees it.
#pragma once

#include "moe_attention_common.cuh"

namespace moe {

int attention_fp4_tile_rows(int64_t rows);              // rows of a row tile for this many rows a kv head
int attention_fp4_blocks(int head_dim, int tile_rows);  // blocks an SM runs
cudaError_t launch_attention_fp4(const AttnParams& p, int num_sms, cudaStream_t s);

}  // namespace moe
