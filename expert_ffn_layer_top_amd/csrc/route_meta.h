// What the two routers share: the block size of the row metadata and the kernels that turn per-block
// expert counts and ranks into counts, offsets, destination rows and row tokens.
#pragma once

#include "common.h"

namespace moe {

constexpr int kRouteBlock = 64;    // tokens per block (one bit each in a 64-bit mask)
constexpr int kMaxK = 16;
constexpr int kMaxE = 256;

// `hist` [ceil(T / 64)][E]: rows of each expert in each block of 64 tokens (overwritten); `dest`
// [T][k]: each row's rank among its block's rows of the same expert, replaced by its row in the
// expert buffers.  Writes counts, offsets, offsets_pad (if given) and row_token (if given).
int enqueue_route_metadata(const int32_t* topk_idx, int T, int E, int k, int32_t* counts, int32_t* offsets,
                           int32_t* offsets_pad, int pad, int32_t* dest, int32_t* row_token, int32_t* hist,
                           hipStream_t s);

}  // namespace moe
