// paged.h -- host side of the attention over a paged cache (arguments validated by paged_api.cu).
#pragma once

#include "attn_more.h"

namespace attn {
namespace paged {
struct Args;
}

size_t paged_fwd_workspace(const attn_paged_fwd_params_t &p);
attn_status_t launch_paged_fwd(const attn_paged_fwd_params_t &p, void *workspace, cudaStream_t s);

// The kernels (paged_rows.cu, paged_tc_sm103.cu); maps of the key and value pages with a box of min(page, box_keys) keys.
constexpr int kRowsBoxKeys = 64;
constexpr int rows_blocks(int64_t d) { return d == 64 ? 3 : 2; }  // CTAs an SM of the few-rows kernel
attn_status_t launch_paged_rows(const CUtensorMap &mk, const CUtensorMap &mv, const paged::Args &a, int d, int grid,
                                cudaStream_t s);
constexpr int kTcBoxKeys = 128;
attn_status_t launch_paged_tc(const CUtensorMap &mq, const CUtensorMap &mk, const CUtensorMap &mv, const paged::Args &a,
                              int d, int tiles, int tile_rows, int grid, bool cuts, cudaStream_t s);
// (tiles a block: 2 of up to 128 rows, or 1 of up to tile_rows, 64 or 128, with two CTAs an SM)

}  // namespace attn
