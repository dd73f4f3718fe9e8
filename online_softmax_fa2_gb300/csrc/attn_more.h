// attn_more.h -- what the operators around the attention share beside attn_internal.h.
#pragma once

#include "attn_internal.h"

namespace attn {

// Bit 2 of the device error word: a page, a position or a cu_q entry was out of range.
enum : uint32_t { kFlagBadIndex = 4u };

// Clears the calling thread's last error message (at the start of every entry point; attn_api.cu).
void clear_error();

}  // namespace attn
