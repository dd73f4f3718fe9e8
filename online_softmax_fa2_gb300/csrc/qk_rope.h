// qk_rope.h -- launchers of qk_rope.cu (arguments validated by the caller, paged_api.cu).
#pragma once

#include "attn_more.h"

namespace attn {

attn_status_t launch_qk_norm_rope(const attn_qk_norm_rope_params_t &p, cudaStream_t s);
// part: one row of d floats for each of rope_bwd_blocks() blocks.
attn_status_t launch_qk_norm_rope_bwd(const attn_qk_norm_rope_bwd_params_t &p, float *part, cudaStream_t s);
// Blocks of the backward, at most.
int rope_bwd_blocks();
attn_status_t launch_paged_append(const attn_paged_append_params_t &p, cudaStream_t s);

}  // namespace attn
