// paged.h -- launcher of the attention over a paged cache (arguments validated by paged_api.cu).
#pragma once

#include "attn_internal.h"

namespace attn {

size_t paged_fwd_workspace(const attn_paged_fwd_params_t &p);
attn_status_t launch_paged_fwd(const attn_paged_fwd_params_t &p, void *workspace, cudaStream_t s);

}  // namespace attn
